"""Cases of the operators of a serving step: new tokens pooled into entries from a stream, entries
appended to the paged cache, and attention of a batch whose sequences share a long prefix.

kind "step"    new tokens of each sequence continue the pooling from a state, which is updated
kind "append"  rows normed, turned to their positions and put into slots of the paged cache, and read back
kind "share"   new tokens over entries that a group of sequences shares and each sequence's own

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits
(angles in 64), with ``own`` true through the framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DTYPE_CODE = {"bf16": 0, "fp16": 1, "fp32": 2}
FORMAT_CODE = {"bf16": 0, "e4m3": 1, "e2m1": 2}
GROUP = 32  # columns that share a scale byte
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases
def _step(name, seqs, tokens, ragged, ratio, coff, d, start, fork, page):
    c = dict(kind="step", seqs=seqs, tokens=tokens, ragged=ragged, ratio=ratio, coff=coff, d=d, start=start, fork=fork, page=page)
    return dict(c, name=name) if name else c


def _append(name, rows, heads, d, dtype, rot, at, layout, norm, first, step, pad, form, spare):
    c = dict(kind="append", rows=rows, heads=heads, d=d, dtype=dtype, rot=rot, at=at, layout=layout, norm=norm, first=first, step=step,
             pad=pad, form=form, spare=spare)
    return dict(c, name=name) if name else c


def _share(name, groups, seqs, tokens, ragged, q_heads, kv_heads, d, prefix, entries, ratio, page, form, sink):
    c = dict(kind="share", groups=groups, seqs=seqs, tokens=tokens, ragged=ragged, q_heads=q_heads, kv_heads=kv_heads, d=d, prefix=prefix,
             entries=entries, ratio=ratio, page=page, form=form, sink=sink)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step of 64 sequences, a quarter of which complete a block
        _step("step a batch by one token", 64, 1, False, 4, 2, 512, 9000, False, 64),
        # the same where blocks are long: few sequences complete one, and that one reads a long window
        _step("step long blocks by one token", 200, 1, False, 128, 2, 128, 30079, False, 64),
        # chunks of three prompts that go on where the last chunks ended, the headline pack's sizes
        _step("step prompts' chunks", 3, 8192, True, 4, 2, 512, 16390, False, 64),
        # long blocks of a chunk of four prompts, each the continuation of one shared beginning
        _step("step long blocks of chunks", 4, 16384, False, 128, 1, 512, 2000, True, 16),
        # the entries that a decoding batch completes in one step, some rows of the buffer unused
        _append("append a step", 64, 1, 512, "bf16", 64, 448, 1, True, 9000, 4, 40, "e4m3", 4096),
        # the entries of a long prompt's chunk
        _append("append a chunk", 24571, 1, 512, "bf16", 64, 448, 1, True, 3, 4, 0, "e4m3", 20000),
        # keys of grouped heads token by token, kept in 16 bits
        _append("append keys of grouped heads", 16384, 8, 128, "bf16", 128, 0, 0, False, 120000, 1, 0, "bf16", 3000),
        # index keys in 4 bits, made in 32 bits, only a part of the head turned
        _append("append index keys", 4099, 1, 128, "fp32", 64, 0, 0, True, 7, 4, 3, "e2m1", 500),
        # latency: four samples of one prompt
        _share("share from four samples", 1, 4, 1, False, 64, 1, 512, 2048, 64, 4, 64, "bf16", True),
        # a decoding batch behind one long system prompt, 8-bit entries
        _share("share a system prompt", 1, 64, 1, False, 64, 1, 512, 16384, 500, 4, 64, "e4m3", True),
        # grouped heads: few rows a sequence, so a tile of the prefix serves many sequences at once
        _share("share with grouped heads", 3, 120, 1, True, 16, 2, 128, 12000, 700, 1, 16, "bf16", False),
        # several samples of two prompts, each with a short draft of tokens that is checked at once
        _share("share from drafts", 2, 24, 5, True, 32, 4, 128, 20000, 300, 1, 64, "e4m3", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "append", "share"])
    if kind == "step":
        ratio = rng.choice([1, 2, 4, 4, 8, 16, 128, rng.randint(3, 40)])
        coff = rng.randint(1, 2)
        d = rng.choice([64, 128, 128, 512, 512, 8 * rng.randint(3, 70), rng.randint(9, 200)])
        single = rng.random() < 0.5
        seqs = _log(rng, 1, 256) if single else rng.randint(1, 8)
        most = max(2, 20_000_000 // (seqs * coff * d * (1 if d % 8 == 0 else 4)))
        tokens = rng.choice([1, 1, rng.randint(2, 5)]) if single else _log(rng, 6, min(16384, max(8, most)))
        return _step(None, seqs, tokens, rng.random() < 0.6, ratio, coff, d, rng.choice([0, _log(rng, 1, 100000)]), rng.random() < 0.3,
                     rng.choice([1, 16, 64, 64, rng.randint(2, 100)]))
    if kind == "append":
        form = rng.choice(["bf16", "e4m3", "e4m3", "e2m1"])
        d = rng.choice([64, 128, 512, 512, 32 * rng.randint(1, 20)]) if form != "bf16" else rng.choice([128, 512, rng.randint(20, 600)])
        heads = rng.choice([1, 1, 1, 2, 8, rng.randint(3, 9)])
        rows = _log(rng, 1, max(2, min(60000, (500_000 if form == "e2m1" else 12_000_000) // (heads * d))))
        rot = rng.choice([0, d // 2 * 2, min(64, d // 2 * 2), 2 * rng.randint(1, d // 2)])
        norm = rot == 0 or rng.random() < 0.7
        return _append(None, rows, heads, d, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rot, rng.choice([0, d - rot]), rng.randint(0, 1),
                       norm, rng.choice([0, _log(rng, 1, 1_000_000)]), rng.choice([1, 2, 4, 128]),
                       rng.choice([0, 0, min(rows - 1, rng.randint(1, 9))]), form, rng.randint(0, 5000))
    d = rng.choice([64, 128, 128, 256, 512, 512, 32 * rng.randint(2, 16)])
    kv_heads = rng.choice([1, 1, 1, 2, 4])
    group = rng.choice([1, 4, 8, 16, 64 // kv_heads, rng.randint(1, 20)])
    seqs = _log(rng, 1, 128)
    tokens = rng.choice([1, 1, 1, rng.randint(2, 8)])
    most = min(16384, 500_000_000 // (seqs * tokens * group * kv_heads), 60_000_000 // (kv_heads * d))
    entries = _log(rng, 2, max(3, min(800, most, 60_000_000 // (seqs * kv_heads * d))))
    ratio = rng.choice([0, 1, 4, 4, 2, 128])
    return _share(None, rng.randint(1, min(4, seqs)), seqs, tokens, rng.random() < 0.7, group * kv_heads, kv_heads, d,
                  _log(rng, min(128, most), max(2, most)), entries, ratio, rng.choice([1, 16, 64, 64, 128, rng.randint(2, 100)]),
                  rng.choice(["bf16", "bf16", "e4m3", "e2m1"]), rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs
def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _whole(v, kind=torch.int32):
    return torch.tensor(v, dtype=kind).cuda()


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _step_lengths(case):
    """New tokens and tokens so far, sequence by sequence: the case's own, whatever the seed."""
    rng = random.Random(case["start"] * 4096 + case["tokens"] * 8 + case["seqs"])
    n = [case["tokens"] if not case["ragged"] or b == 0 else rng.randint(0, case["tokens"]) for b in range(case["seqs"])]
    if case["fork"]:
        return n, [case["start"]] * case["seqs"]
    return n, [case["start"] if b == 0 else rng.randint(0, 2 * case["start"]) for b in range(case["seqs"])]


def _in_place(case):
    """Whether a state is updated where it lies, as in decoding; more tokens leave the old one whole, so that a pass can be run again."""
    return case["tokens"] == 1 and not case["fork"]


def _share_lengths(case):
    """Sequences of each group, and of each sequence the new tokens, own entries and first new token's position; the groups' prefixes."""
    rng = random.Random(case["prefix"] * 4096 + case["entries"] * 8 + case["tokens"])
    groups, seqs, ratio = case["groups"], case["seqs"], case["ratio"]
    cut = sorted(rng.sample(range(1, seqs), groups - 1)) if groups > 1 else []
    cut = [0] + cut + [seqs]
    prefix = [case["prefix"] if g == 0 else rng.randint(case["prefix"] // 2, case["prefix"]) for g in range(groups)]
    tokens = [case["tokens"] if not case["ragged"] or b == 0 else rng.randint(0, case["tokens"]) for b in range(seqs)]
    entries = [case["entries"] if b == 0 else rng.randint(0, case["entries"]) for b in range(seqs)]
    first = []
    for b in range(seqs):
        before = prefix[max(g for g in range(groups) if cut[g] <= b)]
        all_ = before + entries[b]
        p = max(0, all_ * ratio + (rng.randint(0, ratio - 1) if ratio else 0) - tokens[b])
        first.append(p)
        if ratio:
            entries[b] = max(0, min(all_, (p + tokens[b]) // ratio) - before)
    return cut, prefix, tokens, entries, first


def _frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * i / max(rot, 1))


def _turns(freq):
    """A position's turn of each pair in units of 2^-64 of a full one, as the entry points take it."""
    t = [int(round(v / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for v in freq.tolist()]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in t], dtype=torch.int64)


def _most(form):
    return 448.0 if form == "e4m3" else 6.0


def _quantise(x, form):
    """Rows [..., d] in 32 bits -> (values that the codes stand for, before the scale; the scales' exponents), per group."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    m, e = torch.frexp(g.abs().amax(-1, keepdim=True) / _most(form))
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    v = torch.ldexp(g, -e)
    _, b = torch.frexp(v)
    low, bits = (-6, 3) if form == "e4m3" else (0, 1)
    step = (b - 1).clamp(min=low) - bits
    return torch.ldexp(torch.round(torch.ldexp(v, -step)), step), e


def _pack(v, e, form, shape):
    """Codes and scale bytes as the cache holds them."""
    if form == "e4m3":
        data = v.reshape(shape).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = torch.searchsorted(torch.tensor(E2M1, device=v.device), v.abs().contiguous()).to(torch.uint8)
        a = (a | (torch.signbit(v).to(torch.uint8) << 3)).reshape(*shape[:-1], -1, 2)
        data = a[..., 0] | (a[..., 1] << 4)
    return data.contiguous(), (e + 127).to(torch.uint8).reshape(*shape[:-1], -1).contiguous()


def _values(data, scales, form):
    """What the cache's codes stand for, in 32 bits."""
    if form == "bf16":
        return data.float()
    if form == "e4m3":
        v = data.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=data.device)
        v = table[torch.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1).int()]
    s = torch.ldexp(torch.ones((), device=data.device), scales.int() - 127)
    return (v.reshape(*v.shape[:-1], -1, GROUP) * s[..., None]).reshape(v.shape)


def _pool(slots, heads, d, form, gen):
    """A cache whose every slot holds an entry of unit root mean square (a normed one)."""
    x = _normal((slots, heads, d), gen)
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    if form == "bf16":
        return x.bfloat16(), None
    return _pack(*_quantise(x, form), form, (slots, heads, d))


def _table(counts, page, most, order, at):
    """Pages of each sequence in a random order, from the pool's `order` on, and the next free place in it."""
    pages = [-(-n // page) for n in counts]
    table = torch.full((len(counts), max(1, -(-most // page))), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, at


def _prepare_step(s, gen):
    n, first = _step_lengths(s)
    seqs, ratio, coff, d, page = s["seqs"], s["ratio"], s["coff"], s["d"], s["page"]
    wide, window = coff * d, coff * ratio
    s["lens"], s["starts"] = n, first
    cu = _offsets(n)
    made = [(f + k) // ratio - f // ratio for f, k in zip(first, n)]
    s["total"], s["rows"] = sum(made), sum(made) + 3
    s["kv"], s["score"] = (_normal((max(cu[-1], 1), wide), gen).bfloat16() for _ in range(2))
    s["ape"] = 0.02 * _normal((ratio, wide), gen)
    s["cu"], s["first"] = _whole(cu), _whole(first)
    slots = torch.randperm(2 * seqs, generator=gen, device="cuda").to(torch.int32)
    s["from"], s["to"] = slots[:seqs].contiguous(), slots[seqs:].contiguous()
    if s["fork"]:
        s["from"] = s["from"][:1].expand(seqs).contiguous()
    elif _in_place(s):
        s["to"] = s["from"]
    s["kv_state"], s["score_state"] = (_normal((2 * seqs, window, wide), gen).bfloat16() for _ in range(2))
    held = [(f + k) // ratio for f, k in zip(first, n)]
    order = torch.randperm(sum(-(-h // page) for h in held) + 1, generator=gen, device="cuda").to(torch.int32)
    s["table"], _ = _table(held, page, max(held), order, 0)
    s["max_pages"] = s["table"].shape[1]
    s["out"] = torch.zeros(s["rows"], d, dtype=torch.bfloat16, device="cuda")
    s["positions"] = torch.zeros(s["rows"], dtype=torch.int32, device="cuda")
    s["slots"] = torch.zeros(s["rows"], dtype=torch.int64, device="cuda")
    s["entries"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")


def _prepare_append(s, gen):
    rows, heads, d, t, form = s["rows"], s["heads"], s["d"], DTYPES[s["dtype"]], s["form"]
    s["x"] = (_normal((rows, heads, d), gen) * (0.5 + _normal((rows, heads, 1), gen).abs())).to(t)
    s["weight"] = 1.0 + 0.1 * _normal((d,), gen) if s["norm"] else None
    live = rows - s["pad"]
    pos = s["first"] + s["step"] * torch.arange(rows, device="cuda", dtype=torch.int32)
    pos[live:] = -1
    s["pos"] = pos
    freq = _frequencies(s["rot"])
    s["turns"], s["freq"] = _turns(freq).cuda(), freq.cuda()
    s["num_slots"] = rows + s["spare"]
    s["slots"] = torch.randperm(s["num_slots"], generator=gen, device="cuda")[:rows].contiguous()
    s["slots"][live:] = -1
    wide = {"bf16": d, "e4m3": d, "e2m1": d // 2}[form]
    s["data"] = torch.zeros(s["num_slots"], heads, wide, dtype=torch.bfloat16 if form == "bf16" else torch.uint8, device="cuda")
    s["scales"] = None if form == "bf16" else torch.zeros(s["num_slots"], heads, d // GROUP, dtype=torch.uint8, device="cuda")
    s["y"] = torch.zeros(rows, heads, d, dtype=torch.bfloat16, device="cuda")


def _prepare_share(s, gen):
    cut, prefix, tokens, entries, first = _share_lengths(s)
    s["cuts"], s["pres"], s["lens"], s["ents"], s["starts"] = cut, prefix, tokens, entries, first
    page, heads, d = s["page"], s["q_heads"], s["d"]
    cu = _offsets(tokens)
    used = sum(-(-n // page) for n in prefix) + sum(-(-n // page) for n in entries)
    s["num_pages"] = used + 3
    order = torch.randperm(s["num_pages"], generator=gen, device="cuda").to(torch.int32)
    s["prefix_table"], at = _table(prefix, page, s["prefix"], order, 0)
    s["table"], _ = _table(entries, page, s["entries"], order, at)
    s["max_prefix_pages"], s["max_pages"] = s["prefix_table"].shape[1], s["table"].shape[1]
    s["data"], s["scales"] = _pool(s["num_pages"] * page, s["kv_heads"], d, s["form"], gen)
    s["total"] = cu[-1]
    q = _normal((cu[-1], heads, d), gen)
    s["q"] = (q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * 1.5).bfloat16()
    s["cu"], s["cut"], s["prefixes"], s["owns"], s["first"] = (_whole(v) for v in (cu, cut, prefix, entries, first))
    s["sinks"] = _normal((heads,), gen) if s["sink"] else None
    s["y"] = torch.zeros(cu[-1], heads, d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(cu[-1], heads, device="cuda")
    if own:  # the call's workspace
        import gated_pooling_gb300 as gp
        n = gp.csa_cache_attn_prefix_workspace_bytes(s["seqs"], s["groups"], cu[-1], heads, s["kv_heads"], d, s["max_pages"] * page,
                                                     s["max_prefix_pages"] * page)
        s["space"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    {"step": _prepare_step, "append": _prepare_append, "share": _prepare_share}[case["kind"]](s, gen)
    return s


# ------------------------------------------------------------------------ plain forms
def _plain_step(s):
    ratio, coff, d, page = s["ratio"], s["coff"], s["d"], s["page"]
    window, dev = coff * ratio, s["kv"].device
    first, cu = s["first"].long(), s["cu"].long()
    end = first + cu[1:] - cu[:-1]
    before, after = first // ratio, end // ratio
    made = torch.cumsum(after - before, 0)
    # the entries: sequence and block of each row, and its window's places among the new tokens and in the state
    rows = torch.arange(s["total"], device=dev)
    seq = torch.searchsorted(made, rows, right=True)
    block = after[seq] - made[seq] + rows
    at = torch.arange(ratio, device=dev)

    def half(values, state, which):
        pos = (block[:, None] - (1 if coff == 2 and which == 0 else 0)) * ratio + at
        old = pos < first[seq][:, None]
        cols = slice(which * d, which * d + d)
        new = values[torch.where(old, 0, pos - first[seq][:, None] + cu[seq][:, None]), cols]
        kept = state[s["from"][seq].long()[:, None], torch.where(old, pos, 0) % window, cols]
        return torch.where(old[..., None], kept, new).float(), pos >= 0

    halves = range(coff)
    k = [half(s["kv"], s["kv_state"], w) for w in halves]
    x = [half(s["score"], s["score_state"], w)[0] + s["ape"][None, :, w * d:w * d + d] for w in halves]
    x = torch.cat([torch.where(k[w][1][..., None], x[w], float("-inf")) for w in halves], 1)
    w = torch.exp(x - x.amax(1, keepdim=True))
    y = (w * torch.cat([v[0] for v in k], 1)).sum(1) / w.sum(1)
    s["out"][:s["total"]] = y.bfloat16()
    # where they go
    s["positions"].fill_(-1)
    s["slots"].fill_(-1)
    s["positions"][:s["total"]] = (block * ratio).int()
    s["slots"][:s["total"]] = s["table"][seq, block // page].long() * page + block % page
    s["entries"].copy_(after)
    # the state: each of its rows holds the last token of that place, in the columns that a later window reads
    j = torch.arange(window, device=dev)
    pos = end[:, None] - 1 - (end[:, None] - 1 - j) % window
    need = torch.stack([pos >= (after[:, None] - (coff - 1 - w)) * ratio for w in halves], -1) & (pos >= 0)[..., None]
    need = need.repeat_interleave(d, -1)
    old = pos < first[:, None]
    token = torch.where(old, 0, pos - first[:, None] + cu[:-1, None])
    source, to = s["from"].long(), s["to"].long()
    values = [torch.where(need, torch.where(old[..., None], state[source], new[token]), state[to])
              for new, state in ((s["kv"], s["kv_state"]), (s["score"], s["score_state"]))]
    s["kv_state"][to], s["score_state"][to] = values[0], values[1]
    return {"out": s["out"], "positions": s["positions"], "slots": s["slots"], "entries": s["entries"], "kv_state": s["kv_state"],
            "score_state": s["score_state"]}


def _plain_append(s):
    x = s["x"].float()
    if s["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    if s["rot"]:
        a = s["pos"].double()[:, None] * s["freq"][None, :]
        cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
        r = x[..., s["at"]:s["at"] + s["rot"]]
        u, v = (r[..., :s["rot"] // 2], r[..., s["rot"] // 2:]) if s["layout"] == 0 else (r[..., 0::2], r[..., 1::2])
        u, v = u * cos - v * sin, u * sin + v * cos
        r = torch.cat([u, v], -1) if s["layout"] == 0 else torch.stack([u, v], -1).flatten(-2)
        x = torch.cat([x[..., :s["at"]], r, x[..., s["at"] + s["rot"]:]], -1)
    live = s["rows"] - s["pad"]
    x, to = x[:live], s["slots"][:live]
    if s["form"] == "bf16":
        s["data"][to] = x.bfloat16()
        s["y"][:live] = s["data"][to]
    else:
        data, scales = _pack(*_quantise(x, s["form"]), s["form"], tuple(x.shape))
        s["data"][to] = data
        s["scales"][to] = scales
        s["y"][:live] = _values(s["data"][to], s["scales"][to], s["form"]).bfloat16()
    return s["y"]


def _entries(s, table, counts):
    """The entries that a table's sequences hold, in 32 bits, padded to the longest [sequences, heads, entries, d]; zeros behind."""
    e = torch.arange(table.shape[1] * s["page"], device=table.device)
    held = e[None, :] < counts[:, None]
    slot = torch.where(held, table[:, e // s["page"]].long() * s["page"] + e % s["page"], 0)
    k = _values(s["data"][slot], None if s["scales"] is None else s["scales"][slot], s["form"])
    return torch.where(held[:, :, None, None], k, 0.0).permute(0, 2, 1, 3).contiguous()


def _plain_share(s):
    """A prefix's products for all rows of its group at once, padded to the largest group; the own entries' sequence by sequence."""
    heads, kv, d, ratio, total = s["q_heads"], s["kv_heads"], s["d"], s["ratio"], s["total"]
    group, dev = heads // kv, s["q"].device
    cu, cut = s["cu"].long(), s["cut"].long()
    token = torch.arange(total, device=dev)
    seq = torch.searchsorted(cu[1:], token, right=True)
    part = torch.searchsorted(cut[1:], seq, right=True)
    pre, mine = _entries(s, s["prefix_table"], s["prefixes"]), _entries(s, s["table"], s["owns"])
    most_g = max(sum(s["lens"][a:b]) for a, b in zip(s["cuts"], s["cuts"][1:]))
    most_t = max(s["lens"])
    in_g, in_s = token - cu[cut[part]], token - cu[seq]

    def rows_of(values, which, place, n, most):
        """[total, kv, group, c] -> [n, kv, most * group, c]"""
        padded = torch.zeros(n, most, kv, group, values.shape[-1], device=dev)
        padded[which, place] = values
        return padded.permute(0, 2, 1, 3, 4).reshape(n, kv, most * group, -1)

    def back(values, which, place, n, most):
        return values.reshape(n, kv, most, group, -1).permute(0, 2, 1, 3, 4)[which, place]

    q = s["q"].float().reshape(total, kv, group, d)
    by_group, by_seq = (part, in_g, s["groups"], most_g), (seq, in_s, s["seqs"], most_t)
    x = torch.cat([back(rows_of(q, *by_group) @ pre.transpose(-1, -2), *by_group),
                   back(rows_of(q, *by_seq) @ mine.transpose(-1, -2), *by_seq)], -1) * (1.0 / math.sqrt(d))
    n_pre, before = pre.shape[2], s["prefixes"].long()[part]
    seen = before + s["owns"].long()[seq]
    if ratio:
        seen = torch.minimum(seen, (s["first"].long()[seq] + in_s + 1) // ratio)
    e = torch.arange(x.shape[-1], device=dev)
    hidden = torch.where(e < n_pre, e >= torch.minimum(before, seen)[:, None], before[:, None] + e - n_pre >= seen[:, None])
    x = x.masked_fill_(hidden[:, None, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].reshape(1, kv, group, 1)
        top = torch.maximum(top, sink)
    top = torch.where(torch.isinf(top), 0.0, top)
    x = x.sub_(top).exp_()
    z = x.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        z = z + torch.exp(sink - top)
    y = back(rows_of(x[..., :n_pre], *by_group) @ pre, *by_group) + back(rows_of(x[..., n_pre:], *by_seq) @ mine, *by_seq)
    y = torch.where(z > 0, y / z, 0.0).reshape(total, heads, d)
    return {"out": y.bfloat16(), "lse": (torch.log(z) + top).reshape(total, heads)}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import gated_pooling_gb300 as gp
    if s["kind"] == "step":
        gp.csa_compressor_step(s["kv"], s["score"], s["ape"], s["cu"], s["seqs"], s["ratio"], s["coff"], s["d"], s["kv"].shape[0],
                               s["first"], s["from"], s["to"], s["kv_state"].shape[0], s["kv_state"], s["score_state"], s["out"],
                               s["rows"], None, s["table"], s["max_pages"], s["page"], 0, s["positions"], s["slots"], s["entries"])
        return {"out": s["out"], "positions": s["positions"], "slots": s["slots"], "entries": s["entries"], "kv_state": s["kv_state"],
                "score_state": s["score_state"]}
    heads, d = s.get("q_heads") or s["heads"], s["d"]
    if s["kind"] == "append":
        form = FORMAT_CODE[s["form"]]
        gp.csa_cache_append(s["x"], DTYPE_CODE[s["dtype"]], s["rows"], heads, d, heads * d, d, s["weight"], int(s["norm"]), 1e-6, s["pos"],
                            s["turns"], s["rot"], s["at"], s["layout"], 1.0, s["slots"], s["num_slots"], form, s["data"], s["scales"])
        gp.csa_cache_read(s["data"], s["scales"], form, s["slots"], s["rows"], s["num_slots"], heads, d, s["y"], 0, heads * d, d)
        return s["y"]
    gp.csa_cache_attn_prefix(s["q"], heads * d, d, s["cu"], s["seqs"], s["total"], heads, s["kv_heads"], d, s["data"], s["scales"],
                             FORMAT_CODE[s["form"]], s["cut"], s["groups"], s["prefix_table"], s["max_prefix_pages"], s["prefixes"],
                             s["table"], s["max_pages"], s["num_pages"], s["page"], s["owns"], s["first"], s["ratio"], 1.0 / math.sqrt(d),
                             s["sinks"], s["y"], heads * d, d, s["lse"], s["space"], s["space"].numel())
    return {"out": s["y"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"step": _plain_step, "append": _plain_append, "share": _plain_share}[state["kind"]](state)


# -------------------------------------------------------------------------------- work
def _held(d, form):
    """Bytes of one entry of one head."""
    return {"bf16": 2.0 * d, "e4m3": d + d / GROUP, "e2m1": d / 2 + d / GROUP}[form]


def work(case):
    kind, d = case["kind"], case["d"]
    if kind == "step":
        ratio, coff = case["ratio"], case["coff"]
        n, first = _step_lengths(case)
        pairs = kept = made = 0  # (kv, score) pairs of d columns read of the new tokens, those that go into the state, entries
        old = set()              # state's pairs read, a forked state's once
        for b, (k, f) in enumerate(zip(n, first)):
            lo, hi = f // ratio, (f + k) // ratio
            made += hi - lo
            for half in range(coff):
                back = coff - 1 - half  # this half's tokens serve the block `back` behind their own
                if hi > lo:
                    start, stop = max(0, (lo - back) * ratio), (hi - back) * ratio
                    pairs += max(0, stop - max(start, f))
                    old.update((0 if case["fork"] else b, half, p) for p in range(start, min(stop, f)))
                keep = max(0, (hi - back) * ratio)
                kept += f + k - (max(keep, f) if _in_place(case) else keep)
                pairs += max(0, f + k - max(keep, f))
                if not _in_place(case):
                    old.update((0 if case["fork"] else b, half, p) for p in range(keep, f))
        return {"bytes": 4.0 * d * (pairs + len(old) + kept) + 2.0 * d * made + 4.0 * ratio * coff * d, "flops": 6.0 * made * ratio * coff * d}
    if kind == "append":
        n = (case["rows"] - case["pad"]) * case["heads"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]] * d
        return {"bytes": n * (size + 2 * _held(d, case["form"]) + 2 * d) + 20 * case["rows"], "flops": 16.0 * n * d}
    cut, prefix, tokens, entries, first = _share_lengths(case)
    ratio, cache, rows, seen = case["ratio"], 0, 0, 0
    for g, before in enumerate(prefix):
        cache += before if any(tokens[cut[g]:cut[g + 1]]) else 0
        for b in range(cut[g], cut[g + 1]):
            k, e = tokens[b], before + entries[b]
            cache += entries[b] if k else 0
            rows += k
            seen += sum(min(e, (first[b] + i + 1) // ratio) for i in range(k)) if ratio else k * e
    rows *= case["q_heads"]
    return {"bytes": cache * case["kv_heads"] * _held(d, case["form"]) + rows * (4 * d + 4), "flops": 4.0 * seen * case["q_heads"] * d}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_step(s):
    """Sequence by sequence: its tokens in order of position, from the first that the state has to hold."""
    ratio, coff, d, page = s["ratio"], s["coff"], s["d"], s["page"]
    window = coff * ratio
    out = torch.zeros(s["rows"], d, dtype=torch.float64, device="cuda")
    positions = torch.full((s["rows"],), -1, dtype=torch.int32)
    slots = torch.full((s["rows"],), -1, dtype=torch.int64)
    states = {k: s[k].double() for k in ("kv_state", "score_state")}
    source, to, table = s["from"].tolist(), s["to"].tolist(), s["table"].tolist()
    row = at = 0
    for b, (n, f) in enumerate(zip(s["lens"], s["starts"])):
        lo, hi = f // ratio, (f + n) // ratio
        base = max(0, lo - (coff - 1)) * ratio  # position of the first token in `line`
        line = {}
        for name, key in (("kv", "kv_state"), ("score", "score_state")):
            kept = s[key][source[b]][[p % window for p in range(base, f)]].double()
            line[name] = torch.cat([kept, s[name][at:at + n].double()])
        ape = s["ape"].double()
        if hi > lo:
            blocks = hi - lo
            grid = {k: v[lo * ratio - base:hi * ratio - base].reshape(blocks, ratio, -1) for k, v in line.items()}
            sides = [(grid["kv"][..., (coff - 1) * d:], grid["score"][..., (coff - 1) * d:] + ape[:, (coff - 1) * d:])]
            if coff == 2:
                k, x = (torch.zeros(blocks, ratio, d, dtype=torch.float64, device="cuda") for _ in range(2))
                x += float("-inf")
                have = min(blocks, (hi * ratio - base) // ratio - 1)  # blocks with a block before them
                if have:
                    start = (hi - have - 1) * ratio - base
                    k[blocks - have:] = line["kv"][start:start + have * ratio, :d].reshape(have, ratio, d)
                    x[blocks - have:] = line["score"][start:start + have * ratio, :d].reshape(have, ratio, d) + ape[:, :d]
                sides.insert(0, (k, x))
            k, x = (torch.cat([p[i] for p in sides], 1) for i in range(2))
            out[row:row + blocks] = torch.einsum("brd,brd->bd", torch.softmax(x, 1), k)
            for i in range(blocks):
                e = lo + i
                positions[row + i] = e * ratio
                slots[row + i] = table[b][e // page] * page + e % page
            row += blocks
        for half in range(coff):
            keep = max(0, (hi - (coff - 1 - half)) * ratio)
            if keep < f + n:
                where = [p % window for p in range(keep, f + n)]
                for name, key in (("kv", "kv_state"), ("score", "score_state")):
                    states[key][to[b], where, half * d:half * d + d] = line[name][keep - base:, half * d:half * d + d]
        at += n
    entries = torch.tensor([(f + n) // ratio for n, f in zip(s["lens"], s["starts"])], dtype=torch.int32)
    return {"out": out, "positions": positions, "slots": slots, "entries": entries, **states}


def _nearest(v, form):
    """Each value's nearest code value, a tie to the even code: by search in the table of all of them."""
    if form == "e4m3":
        table = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
    else:
        table = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    a = v.abs().contiguous()
    hi = torch.searchsorted(table, a).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(table[pick], v)


def _exact_append(s):
    """Each row's rotation as complex factors, each group's scale by its logarithm."""
    x = s["x"].double()
    if s["norm"]:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].double()
    if s["rot"]:
        turn = torch.polar(torch.ones_like(s["freq"]).expand(s["rows"], -1), s["pos"].double()[:, None] * s["freq"])[:, None]
        i = torch.arange(s["rot"] // 2, device=x.device)
        ia = s["at"] + (i if s["layout"] == 0 else 2 * i)
        ib = ia + (s["rot"] // 2 if s["layout"] == 0 else 1)
        z = torch.complex(x[..., ia], x[..., ib]) * turn
        x[..., ia], x[..., ib] = z.real, z.imag
    if s["form"] != "bf16":
        g = x.reshape(*x.shape[:-1], -1, GROUP)
        scale = torch.exp2(torch.ceil(torch.log2(g.abs().amax(-1, keepdim=True) / _most(s["form"]))).clamp(-127, 127))
        x = (_nearest(g / scale, s["form"]) * scale).reshape(x.shape)
    x[s["rows"] - s["pad"]:] = 0
    return x


def _exact_values(s, slots):
    """The entries in these slots."""
    rows = s["data"][slots]
    if s["form"] == "bf16":
        return rows.double()
    if s["form"] == "e4m3":
        v = torch.arange(256, device=rows.device).to(torch.uint8).view(torch.float8_e4m3fn).double()[rows.long()]
    else:
        pair = torch.empty(*rows.shape, 2, dtype=torch.float64, device=rows.device)
        table = torch.tensor([(-1.0 if c > 7 else 1.0) * E2M1[c % 8] for c in range(16)], dtype=torch.float64, device=rows.device)
        pair[..., 0], pair[..., 1] = table[(rows % 16).long()], table[(rows // 16).long()]
        v = pair.flatten(-2)
    return v * torch.exp2(s["scales"][slots].double() - 127.0).repeat_interleave(GROUP, -1)


def _exact_share(s):
    """Sequence by sequence over one list of its entries, the prefix's and its own, head by head of the cache."""
    out = torch.zeros(s["total"], s["q_heads"], s["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], s["q_heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    per, at, page = s["q_heads"] // s["kv_heads"], 0, s["page"]

    def slots(table, n):
        where = torch.arange(n, device="cuda")
        return table.long()[where // page] * page + where % page

    for g in range(s["groups"]):
        shared = _exact_values(s, slots(s["prefix_table"][g], s["pres"][g]))
        for b in range(s["cuts"][g], s["cuts"][g + 1]):
            n = s["lens"][b]
            if n == 0:
                continue
            kv = torch.cat([shared, _exact_values(s, slots(s["table"][b], s["ents"][b]))])
            e = kv.shape[0]
            lim = torch.full((n,), e, device="cuda")
            if s["ratio"]:
                lim = torch.minimum(lim, (s["starts"][b] + torch.arange(n, device="cuda") + 1) // s["ratio"])
            hidden = torch.arange(e, device="cuda")[None, None, :] >= lim[:, None, None]
            for h in range(s["kv_heads"]):
                hs = slice(h * per, (h + 1) * per)
                x = torch.einsum("tgd,ed->tge", s["q"][at:at + n, hs].double(), kv[:, h]) / math.sqrt(s["d"])
                x = torch.where(hidden, float("-inf"), x)
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][hs].double().reshape(1, per, 1).expand(n, per, 1)], -1)
                if x.shape[-1] == 0:
                    continue
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])[..., :e]
                out[at:at + n, hs] = torch.einsum("tge,ed->tgd", p, kv[:, h])
                lse[at:at + n, hs] = z
            at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "append": _exact_append, "share": _exact_share}[case["kind"]](s)
