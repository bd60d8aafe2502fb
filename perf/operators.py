"""Cases of the operators between a pooled entry and the attention that reads it.

kind "rotate"  norm of every head and rotation to the row's position, forward
kind "turn"    its gradients (input and norm weight)
kind "append"  rows quantised into slots of the paged cache, and read back
kind "gather"  rows of the cache read back
kind "attend"  new tokens over a paged cache whose entries are key and value at once

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
def _rotate(name, kind, rows, heads, d, dtype, rot, start, layout, norm, scaling, first, step, pad, slab):
    c = dict(kind=kind, rows=rows, heads=heads, d=d, dtype=dtype, rot=rot, start=start, layout=layout, norm=norm, scaling=scaling,
             first=first, step=step, pad=pad, slab=slab)
    return dict(c, name=name) if name else c


def _cache(name, kind, rows, heads, d, dtype, form, spare):
    c = dict(kind=kind, rows=rows, heads=heads, d=d, dtype=dtype, form=form, spare=spare)
    return dict(c, name=name) if name else c


def _attend(name, seqs, tokens, ragged, q_heads, kv_heads, d, entries, ratio, page, form, sink):
    c = dict(kind="attend", seqs=seqs, tokens=tokens, ragged=ragged, q_heads=q_heads, kv_heads=kv_heads, d=d, entries=entries,
             ratio=ratio, page=page, form=form, sink=sink)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the entries that a decoding batch of 16 sequences completes in one step
        _rotate("rotate a step's entries", "rotate", 16, 1, 512, "bf16", 64, 448, 1, True, "none", 9000, 37, 0, False),
        # the headline pack's entries (3 x 8192 tokens, ratio 4), positions one block apart, padded rows behind the last
        _rotate("rotate a pack's entries", "rotate", 6180, 1, 512, "bf16", 64, 448, 1, True, "linear", 3, 4, 36, False),
        # queries of a long prompt, read out of a wider projection, a long context's frequencies
        _rotate("rotate a prompt's queries", "rotate", 8192, 64, 128, "bf16", 128, 0, 0, True, "yarn", 120000, 1, 0, True),
        # training: gradients of the queries of 8192 tokens
        _rotate("turn back queries", "turn", 8192, 32, 128, "bf16", 128, 0, 0, True, "none", 0, 1, 0, False),
        # training in 32 bits: gradients of the headline pack's entries, the rotated part behind the rest
        _rotate("turn back entries in 32 bits", "turn", 6151, 1, 512, "fp32", 64, 448, 1, True, "yarn", 3, 4, 7, False),
        # one decoding step of 64 sequences writes its entries
        _cache("append a step", "append", 64, 1, 512, "bf16", "e4m3", 4096),
        # a chunk of a long prompt is written, and read back for the work that wants 16 bits
        _cache("append a chunk", "append", 24571, 1, 512, "bf16", "e4m3", 20000),
        # index keys of a long context kept in 4 bits
        _cache("gather index keys", "gather", 262139, 1, 128, "bf16", "e2m1", 100000),
        # latency of one sequence that decodes
        _attend("attend from one token", 1, 1, False, 64, 1, 512, 2048, 4, 64, "bf16", True),
        # a decoding batch over contexts of different lengths, 8-bit entries
        _attend("attend from a batch of tokens", 48, 1, False, 64, 1, 512, 8192, 4, 64, "e4m3", True),
        # chunks of three prompts over pooled entries
        _attend("attend from prompts' chunks", 3, 1024, True, 64, 1, 512, 4096, 4, 64, "bf16", True),
        # token-by-token entries, grouped heads, small pages
        _attend("attend with grouped heads", 2, 1500, True, 16, 2, 128, 6000, 1, 16, "e4m3", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "turn", "append", "gather", "attend", "attend"])
    if kind in ("rotate", "turn"):
        d = rng.choice([64, 128, 128, 512, 512, 8 * rng.randint(4, 64), rng.randint(33, 300)])
        heads = rng.choice([1, 1, 2, 8, rng.randint(3, 33), 64])
        rows = _log(rng, 1, max(2, min(40000, 50_000_000 // (heads * d))))
        rot = rng.choice([0, d // 2 * 2, min(64, d // 2 * 2), 2 * rng.randint(1, d // 2)])
        start = rng.choice([0, d - rot])
        norm = rot == 0 or rng.random() < 0.8
        return _rotate(None, kind, rows, heads, d, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rot, start, rng.randint(0, 1), norm,
                       rng.choice(["none", "linear", "yarn"]), rng.choice([0, _log(rng, 1, 1_000_000)]), rng.choice([1, 2, 4, 128]),
                       rng.choice([0, 0, min(rows - 1, rng.randint(1, 9))]), rng.random() < 0.3)
    if kind in ("append", "gather"):
        form = rng.choice(["bf16", "e4m3", "e4m3", "e2m1"])
        d = 32 * rng.randint(1, 20) if form != "bf16" else rng.choice([128, 512, rng.randint(20, 600)])
        heads = rng.choice([1, 1, 2, 8, rng.randint(3, 9)])
        rows = _log(rng, 1, max(2, min(300000, 30_000_000 // (heads * d))))
        return _cache(None, kind, rows, heads, d, rng.choice(["bf16", "bf16", "fp16", "fp32"]), form, rng.randint(0, 5000))
    single = rng.random() < 0.5
    d = rng.choice([64, 128, 128, 256, 512, 512, 32 * rng.randint(2, 16)])
    kv_heads = rng.choice([1, 1, 1, 2, 4])
    group = rng.choice([1, 4, 8, 16, 64 // kv_heads, rng.randint(1, 20)])
    seqs = _log(rng, 1, 64) if single else rng.randint(1, 6)
    tokens = rng.choice([1, 1, 1, rng.randint(2, 4)]) if single else _log(rng, 5, 2000)
    most = min(12000, 400_000_000 // (seqs * tokens * group * kv_heads), 80_000_000 // (seqs * kv_heads * d))
    ratio = rng.choice([0, 1, 4, 4, 2, 128])
    if not single and ratio == 0:
        ratio = rng.choice([0, 4])
    return _attend(None, seqs, tokens, rng.random() < 0.7, group * kv_heads, kv_heads, d, _log(rng, min(16, most), max(2, most)), ratio,
                   rng.choice([1, 16, 64, 64, 128, rng.randint(2, 100)]), rng.choice(["bf16", "bf16", "e4m3", "e2m1"]), rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs
def _frequencies(rot, scaling):
    """Frequencies in 64 bits and the amplitude: base 10000; linear: a quarter; yarn: 16 times a context of 4096."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        at = [rot * math.log(4096.0 / (n * 2.0 * math.pi)) / (2.0 * math.log(10000.0)) for n in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f / 16.0 * ramp + f * (1.0 - ramp), 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _turns(freq):
    """A position's turn of each pair in units of 2^-64 of a full one, as the entry points take it."""
    t = [int(round(v / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for v in freq.tolist()]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in t], dtype=torch.int64)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


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


def _empty_pool(slots, heads, d, form):
    if form == "bf16":
        return torch.zeros(slots, heads, d, dtype=torch.bfloat16, device="cuda"), None
    return (torch.zeros(slots, heads, d if form == "e4m3" else d // 2, dtype=torch.uint8, device="cuda"),
            torch.zeros(slots, heads, d // GROUP, dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    kind = case["kind"]
    if kind in ("rotate", "turn"):
        rows, heads, d, t = case["rows"], case["heads"], case["d"], DTYPES[case["dtype"]]
        wide = heads + 2 if case["slab"] else heads
        s["x"] = (_normal((rows, wide, d), gen) * (0.5 + _normal((rows, wide, 1), gen).abs())).to(t)[:, wide - heads:]
        if kind == "turn":
            s["dy"] = _normal((rows, wide, d), gen).to(t)[:, wide - heads:]
            s["dw"] = torch.zeros(d, device="cuda")
        s["weight"] = 1.0 + 0.1 * _normal((d,), gen) if case["norm"] else None
        pos = case["first"] + case["step"] * torch.arange(rows, device="cuda", dtype=torch.int32)
        if case["pad"]:
            pos[rows - case["pad"]:] = -1
        s["pos"] = pos
        s["freq"], s["amplitude"] = _frequencies(case["rot"], case["scaling"])
        s["turns"] = _turns(s["freq"]).cuda()
        s["freq"] = s["freq"].cuda()
        s["y"] = torch.zeros(rows, heads, d, dtype=t, device="cuda")
        if own and kind == "turn":
            import gated_pooling_gb300 as gp
            s["space"] = torch.empty(max(16, gp.csa_norm_rope_bwd_workspace_bytes(rows, heads, d)), dtype=torch.uint8, device="cuda")
    elif kind in ("append", "gather"):
        rows, heads, d, t = case["rows"], case["heads"], case["d"], DTYPES[case["dtype"]]
        slots = rows + case["spare"]
        s["num_slots"] = slots
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:rows].contiguous()
        if kind == "append":
            s["x"] = (_normal((rows, heads, d), gen) * torch.exp(_normal((rows, heads, 1), gen))).to(t)
            s["data"], s["scales"] = _empty_pool(slots, heads, d, case["form"])
        else:
            s["data"], s["scales"] = _pool(slots, heads, d, case["form"], gen)
        s["y"] = torch.zeros(rows, heads, d, dtype=t, device="cuda")
    else:
        seqs, ratio, page, heads = case["seqs"], case["ratio"], case["page"], case["q_heads"]
        tokens, entries, first = _lengths(case)
        s["lens"], s["ents"], s["starts"] = tokens, entries, first
        cu = [0]
        for n in tokens:
            cu.append(cu[-1] + n)
        pages = [-(-e // page) for e in entries]
        s["max_pages"] = max(1, -(-case["entries"] // page))
        s["num_pages"] = max(1, sum(pages) + 3)
        order = torch.randperm(s["num_pages"], generator=gen, device="cuda").to(torch.int32)
        table = torch.full((seqs, s["max_pages"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table
        s["data"], s["scales"] = _pool(s["num_pages"] * page, case["kv_heads"], case["d"], case["form"], gen)
        s["total"] = cu[-1]
        q = _normal((cu[-1], heads, case["d"]), gen)
        s["q"] = (q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * 1.5).bfloat16()
        s["cu"], s["entries_"], s["first"] = (torch.tensor(v, dtype=torch.int32).cuda() for v in (cu, entries, first))
        s["sinks"] = _normal((heads,), gen) if case["sink"] else None
        s["y"] = torch.zeros(cu[-1], heads, case["d"], dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(cu[-1], heads, device="cuda")
        if own:
            import gated_pooling_gb300 as gp
            n = gp.csa_cache_attn_workspace_bytes(seqs, cu[-1], heads, case["kv_heads"], case["d"], s["max_pages"] * page)
            s["space"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    return s


def _lengths(case):
    """New tokens, entries and the first new token's position, sequence by sequence: the case's own, whatever the seed."""
    rng = random.Random(case["entries"] * 4096 + case["tokens"])
    tokens = [case["tokens"] if not case["ragged"] or b == 0 else rng.randint(0, case["tokens"]) for b in range(case["seqs"])]
    entries = [case["entries"] if b == 0 else rng.randint(0 if case["ragged"] else min(1, case["entries"]), case["entries"])
               for b in range(case["seqs"])]
    ratio, first = case["ratio"], []
    for b, (n, e) in enumerate(zip(tokens, entries)):
        p = max(0, e * ratio + (rng.randint(0, ratio - 1) if ratio else 0) - n)
        first.append(p)
        if ratio:
            entries[b] = min(e, (p + n) // ratio)
    return tokens, entries, first


# ------------------------------------------------------------------------ plain forms
def _cos_sin(s, half):
    a = s["pos"].double()[:, None] * s["freq"][None, :]
    return [(f(a) * s["amplitude"]).to(half)[:, None, :] for f in (torch.cos, torch.sin)]


def _halves(x, s):
    """The two members of each pair in the rotated part."""
    r = x[..., s["start"]:s["start"] + s["rot"]]
    return (r[..., :s["rot"] // 2], r[..., s["rot"] // 2:]) if s["layout"] == 0 else (r[..., 0::2], r[..., 1::2])


def _joined(a, b, x, s):
    r = torch.cat([a, b], -1) if s["layout"] == 0 else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([x[..., :s["start"]], r, x[..., s["start"] + s["rot"]:]], -1)


def _plain_rotate(s):
    x = s["x"].float()
    if s["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * s["weight"]
    if s["rot"]:
        cos, sin = _cos_sin(s, torch.float32)
        a, b = _halves(x, s)
        x = _joined(a * cos - b * sin, a * sin + b * cos, x, s)
    return torch.where(s["pos"][:, None, None] >= 0, x, 0.0).to(s["x"].dtype)


def _plain_turn(s):
    live = s["pos"][:, None, None] >= 0
    x, g = s["x"].float(), torch.where(live, s["dy"].float(), 0.0)
    if s["rot"]:
        cos, sin = _cos_sin(s, torch.float32)
        a, b = _halves(g, s)
        g = _joined(a * cos + b * sin, b * cos - a * sin, g, s)
    if not s["norm"]:
        return {"dx": g.to(s["x"].dtype)}
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    n = x * r
    dw = (g * n).sum((0, 1))
    g = g * s["weight"]
    return {"dx": (r * (g - n * (g * n).mean(-1, keepdim=True))).to(s["x"].dtype), "dw": dw}


def _plain_append(s):
    x = s["x"].float()
    if s["form"] == "bf16":
        s["data"][s["slots"]] = x.bfloat16()
    else:
        data, scales = _pack(*_quantise(x, s["form"]), s["form"], tuple(x.shape))
        s["data"][s["slots"]] = data
        s["scales"][s["slots"]] = scales
    return _plain_gather(s)


def _plain_gather(s):
    scales = None if s["scales"] is None else s["scales"][s["slots"]]
    return _values(s["data"][s["slots"]], scales, s["form"]).to(s["y"].dtype)


def _plain_attend(s):
    """All sequences at once, padded to the longest."""
    seqs, heads, kv, d = s["seqs"], s["q_heads"], s["kv_heads"], s["d"]
    group, most_t, most_e = heads // kv, max(max(s["lens"]), 1), max(max(s["ents"]), 1)
    dev = s["q"].device
    n = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(most_t, device=dev)
    live = i[None, :] < n[:, None]
    rows = torch.where(live, s["cu"][:-1, None] + i[None, :], 0).long()
    q = s["q"].float()[rows].reshape(seqs, most_t, kv, group, d).permute(0, 2, 1, 3, 4).reshape(seqs, kv, most_t * group, d)
    e = torch.arange(most_e, device=dev)
    held = e[None, :] < s["entries_"][:, None]
    slot = torch.where(held, s["table"][:, e // s["page"]].long() * s["page"] + e % s["page"], 0)
    scales = None if s["scales"] is None else s["scales"][slot]
    k = _values(s["data"][slot], scales, s["form"])
    k = torch.where(held[:, :, None, None], k, 0.0).permute(0, 2, 1, 3).contiguous()
    seen = s["entries_"][:, None].expand(seqs, most_t)
    if s["ratio"]:
        seen = torch.minimum(seen, (s["first"][:, None] + i[None, :] + 1) // s["ratio"])
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).reshape(seqs, kv, most_t, group, most_e)
    x = x.masked_fill_((e[None, None, :] >= seen[:, :, None])[:, None, :, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].reshape(1, kv, 1, group, 1)
        top = torch.maximum(top, sink)
    top = torch.where(torch.isinf(top), 0.0, top)
    x = x.sub_(top).exp_()
    z = x.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        z = z + torch.exp(sink - top)
    y = torch.matmul(x.reshape(seqs, kv, most_t * group, most_e), k).reshape(seqs, kv, most_t, group, d)
    y = torch.where(z > 0, y / z, 0.0).permute(0, 2, 1, 3, 4).reshape(seqs, most_t, heads, d)
    lse = (torch.log(z) + top).permute(0, 2, 1, 3, 4).reshape(seqs, most_t, heads)
    return {"out": y[live].bfloat16(), "lse": lse[live]}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import gated_pooling_gb300 as gp
    kind = s["kind"]
    if kind == "rotate":
        gp.csa_norm_rope_fwd(s["x"], DTYPE_CODE[s["dtype"]], s["rows"], s["heads"], s["d"], s["x"].stride(0), s["x"].stride(1),
                             s["weight"], int(s["norm"]), 1e-6, s["pos"], s["turns"], s["rot"], s["start"], s["layout"], s["amplitude"],
                             s["y"], s["heads"] * s["d"], s["d"])
        return s["y"]
    if kind == "turn":
        gp.csa_norm_rope_bwd(s["x"], s["dy"], DTYPE_CODE[s["dtype"]], s["rows"], s["heads"], s["d"], s["x"].stride(0), s["x"].stride(1),
                             s["dy"].stride(0), s["dy"].stride(1), s["weight"], int(s["norm"]), 1e-6, s["pos"], s["turns"], s["rot"],
                             s["start"], s["layout"], s["amplitude"], s["y"], s["heads"] * s["d"], s["d"],
                             s["dw"] if s["norm"] else None, 0, s["space"], s["space"].numel())
        return {"dx": s["y"], "dw": s["dw"]} if s["norm"] else {"dx": s["y"]}
    if kind in ("append", "gather"):
        form, heads, d = FORMAT_CODE[s["form"]], s["heads"], s["d"]
        if kind == "append":
            gp.csa_cache_write(s["x"], DTYPE_CODE[s["dtype"]], s["rows"], heads, d, heads * d, d, s["slots"], s["num_slots"], form,
                               s["data"], s["scales"])
        gp.csa_cache_read(s["data"], s["scales"], form, s["slots"], s["rows"], s["num_slots"], heads, d, s["y"], DTYPE_CODE[s["dtype"]],
                          heads * d, d)
        return s["y"]
    heads, d = s["q_heads"], s["d"]
    gp.csa_cache_attn(s["q"], heads * d, d, s["cu"], s["seqs"], s["total"], heads, s["kv_heads"], d, s["data"], s["scales"],
                      FORMAT_CODE[s["form"]], s["table"], s["max_pages"], s["num_pages"], s["page"], s["entries_"], s["first"], s["ratio"],
                      1.0 / math.sqrt(d), s["sinks"], s["y"], heads * d, d, s["lse"], s["space"], s["space"].numel())
    return {"out": s["y"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "turn": _plain_turn, "append": _plain_append, "gather": _plain_gather,
            "attend": _plain_attend}[state["kind"]](state)


# -------------------------------------------------------------------------------- work
def _held(d, form):
    """Bytes of one entry of one head."""
    return {"bf16": 2.0 * d, "e4m3": d + d / GROUP, "e2m1": d / 2 + d / GROUP}[form]


def work(case):
    kind = case["kind"]
    if kind in ("rotate", "turn"):
        n = (case["rows"] - case["pad"]) * case["heads"] * case["d"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        passes = 2 if kind == "rotate" or not case["norm"] else 3
        return {"bytes": passes * n * size + 4 * case["rows"] + 4 * case["d"], "flops": (10 if kind == "rotate" else 20) * n}
    if kind in ("append", "gather"):
        n = case["rows"] * case["heads"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]] * case["d"]
        held = _held(case["d"], case["form"])
        return {"bytes": (2 if kind == "append" else 1) * n * (size + held) + 8 * case["rows"], "flops": 4 * n * case["d"]}
    ratio, cache, rows, seen = case["ratio"], 0, 0, 0
    for n, e, p in zip(*_lengths(case)):
        cache += e if n else 0
        rows += n
        seen += sum(min(e, (p + i + 1) // ratio) for i in range(n)) if ratio else n * e
    rows *= case["q_heads"]
    return {"bytes": cache * case["kv_heads"] * _held(case["d"], case["form"]) + rows * (4 * case["d"] + 4),
            "flops": 4.0 * seen * case["q_heads"] * case["d"]}


# ---------------------------------------------------------------- the definition in 64 bits
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


def _exact_cache(s):
    if s["kind"] == "append":
        x = s["x"].double()
        if s["form"] == "bf16":
            return x
        g = x.reshape(*x.shape[:-1], -1, GROUP)
        scale = torch.exp2(torch.ceil(torch.log2(g.abs().amax(-1, keepdim=True) / _most(s["form"]))).clamp(-127, 127))
        return (_nearest(g / scale, s["form"]) * scale).reshape(x.shape)
    rows = s["data"][s["slots"]]
    if s["form"] == "bf16":
        return rows.double()
    if s["form"] == "e4m3":
        v = torch.arange(256, device=rows.device).to(torch.uint8).view(torch.float8_e4m3fn).double()[rows.long()]
    else:
        pair = torch.empty(*rows.shape, 2, dtype=torch.float64, device=rows.device)
        table = torch.tensor([(-1.0 if c > 7 else 1.0) * E2M1[c % 8] for c in range(16)], dtype=torch.float64, device=rows.device)
        pair[..., 0], pair[..., 1] = table[(rows % 16).long()], table[(rows // 16).long()]
        v = pair.flatten(-2)
    return v * torch.exp2(s["scales"][s["slots"]].double() - 127.0).repeat_interleave(GROUP, -1)


def _exact_rows(s):
    """Forward or gradients with each row's rotation as complex factors."""
    x = s["x"].double()
    keep = (s["pos"] >= 0)[:, None, None]
    turn = torch.polar(torch.full_like(s["freq"], s["amplitude"]).expand(s["rows"], -1), s["pos"].double()[:, None] * s["freq"])[:, None]
    cols = torch.arange(s["rot"] // 2, device=x.device)
    ia = s["start"] + (cols if s["layout"] == 0 else 2 * cols)
    ib = ia + (s["rot"] // 2 if s["layout"] == 0 else 1)

    def turned(v, by):
        z = torch.complex(v[..., ia], v[..., ib]) * by
        v = v.clone()
        v[..., ia], v[..., ib] = z.real, z.imag
        return v

    rms = torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) if s["norm"] else None
    w = s["weight"].double() if s["norm"] else None
    if s["kind"] == "rotate":
        return turned(x / rms * w if s["norm"] else x, turn) * keep
    g = turned(s["dy"].double() * keep, turn.conj())
    if not s["norm"]:
        return {"dx": g}
    inner = (g * w * x).sum(-1, keepdim=True)
    return {"dx": g * w / rms - x * inner / (s["d"] * rms ** 3), "dw": torch.einsum("rhd,rhd->d", g, x / rms)}


def _exact_attend(s):
    """Sequence by sequence and head by head of the cache, the weights from the normalised exponentials."""
    out = torch.zeros(s["total"], s["q_heads"], s["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["total"], s["q_heads"]), float("-inf"), dtype=torch.float64, device="cuda")
    group, at = s["q_heads"] // s["kv_heads"], 0
    for b, n in enumerate(s["lens"]):
        e = s["ents"][b]
        where = torch.arange(e, device="cuda")
        slots = s["table"][b].long()[where // s["page"]] * s["page"] + where % s["page"]
        kv = _exact_cache({"kind": "gather", "form": s["form"], "data": s["data"], "scales": s["scales"], "slots": slots})
        for h in range(s["kv_heads"]):
            for t0 in range(0, n, 256):  # in pieces, for the memory
                t1 = min(n, t0 + 256)
                hs = slice(h * group, (h + 1) * group)
                lim = torch.full((t1 - t0,), e, device="cuda")
                if s["ratio"]:
                    lim = torch.minimum(lim, (s["starts"][b] + torch.arange(t0, t1, device="cuda") + 1) // s["ratio"])
                x = torch.einsum("tgd,ed->tge", s["q"][at + t0:at + t1, hs].double(), kv[:, h]) / math.sqrt(s["d"])
                x = torch.where(where[None, None, :] < lim[:, None, None], x, float("-inf"))
                if s["sinks"] is not None:
                    x = torch.cat([x, s["sinks"][hs].double().reshape(1, group, 1).expand(t1 - t0, group, 1)], -1)
                if x.shape[-1] == 0:
                    continue
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - torch.where(torch.isinf(z), 0.0, z)[..., None])[..., :e]
                out[at + t0:at + t1, hs] = torch.einsum("tge,ed->tgd", p, kv[:, h])
                lse[at + t0:at + t1, hs] = z
        at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("rotate", "turn"):
        return _exact_rows(s)
    return _exact_attend(s) if case["kind"] == "attend" else _exact_cache(s)
