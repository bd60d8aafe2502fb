"""A batch as it is served: prompts pooled and put into the cache, sequences that go on from a prompt's state and share
its entries, chunks first and then single tokens, each a pooling step, an append of what it completed and the
attention of its tokens, with every length, position and slot on the device; called one by one, and captured
once and replayed. Each operator is checked against 64-bit arithmetic on what the one before it left."""
import math

import pytest
import torch

from tests import operator_reference as R
from tests import serving_reference as V
from tests.test_gpu_append import check as check_append

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
PAGE = 16


class Batch:
    """Group i's sequences (group_of) have prompts[i] tokens in common."""

    def __init__(self, gp, prompts, group_of, more, ratio, coff, d, heads, fmt, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.gp, self.prompts, self.group_of, self.ratio, self.coff, self.d, self.heads, self.fmt = gp, prompts, group_of, ratio, coff, d, heads, fmt
        self.S, self.G, self.C, self.W = len(group_of), len(prompts), coff * d, coff * ratio
        total = max(prompts) + more
        self.kv, self.score = (torch.randn(self.S, total, self.C, generator=g).to(torch.bfloat16) for _ in range(2))
        for s, i in enumerate(group_of):
            for t in (self.kv, self.score):
                t[s, :prompts[i]] = t[group_of.index(i), :prompts[i]]
        self.ape = 0.3 * torch.randn(ratio, self.C, generator=g)
        self.weight = 1 + 0.1 * torch.randn(d, generator=g)
        self.rot = min(64, d)
        self.turns, self.amp = gp.csa_rope_table(self.rot, 10000.0, gp.CSA_ROPE_YARN, 16.0, 4096.0)
        self.sink = torch.randn(heads, generator=g)
        # states: a prompt's, then a sequence's; pages: a prompt's and a sequence's rows of two tables
        self.kv_state, self.score_state = (torch.zeros(self.G + self.S, self.W, self.C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.pages = [max(1, -(-(max(prompts) // ratio) // PAGE)), -(-(more // ratio + 1) // PAGE)]
        self.num = self.G * self.pages[0] + self.S * self.pages[1] + 1
        order = torch.randperm(self.num, generator=g).to(torch.int32)
        cut = self.G * self.pages[0]
        self.tables = [order[:cut].view(self.G, -1), order[cut:cut + self.S * self.pages[1]].view(self.S, -1)]
        self.dtables = [t.contiguous().cuda() for t in self.tables]
        slots = self.num * PAGE
        self.data = torch.full((slots, 1, {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt]), 0x2A, dtype=torch.uint8, device="cuda")
        self.scales = None if fmt == R.BF16 else torch.full((slots, 1, d // 32), 0x7E, dtype=torch.uint8, device="cuda")
        self.prefix_entries = torch.zeros(self.G, **I32)
        self.dape, self.dweight, self.dturns, self.dsink = (t.cuda() for t in (self.ape, self.weight, self.turns, self.sink))
        self.dgroups = torch.tensor(group_of, device="cuda")
        self.cuts = torch.tensor([group_of.index(i) for i in range(self.G)] + [self.S], **I32)
        self.done = [prompts[i] for i in group_of]  # tokens of each sequence so far
        self.gen = g

    def pooled(self, bufs, S, base, table, max_pages):
        """What a call's tokens complete, into the cache."""
        b, gp, d, slots = bufs, self.gp, self.d, self.num * PAGE
        gp.csa_compressor_step(b["kv"], b["score"], self.dape, b["cu"], S, self.ratio, self.coff, d, b["kv"].shape[0], b["first"],
                               b["source"], b["target"], self.G + self.S, self.kv_state, self.score_state, b["out"], b["out"].shape[0],
                               base, table, max_pages, PAGE, 0, b["positions"], b["slots"], b["entries"], b["err"])
        gp.csa_cache_append(b["out"], 0, b["out"].shape[0], 1, d, d, d, self.dweight, 1, 1e-6, b["positions"], self.dturns, self.rot,
                            d - self.rot, 1, self.amp, b["slots"], slots, self.fmt, self.data, self.scales, b["err"])

    def asked(self, b):
        """The call's tokens over their prompts' entries and their own."""
        S, T, H, d = self.S, b["kv"].shape[0], self.heads, self.d
        self.gp.csa_cache_attn_prefix(
            b["q"], H * d, d, b["cu"], S, T, H, 1, d, self.data, self.scales, self.fmt, self.cuts, self.G, self.dtables[0], self.pages[0],
            self.prefix_entries, self.dtables[1], self.pages[1], self.num, PAGE, b["entries"], b["first"], self.ratio, d ** -0.5, self.dsink,
            b["o"], H * d, d, b["lse"], b["ws"], b["ws"].numel(), b["err"])

    def buffers(self, S, tokens, source, target):
        rows, H, d = tokens // self.ratio + S + 1, self.heads, self.d
        ws = self.gp.csa_cache_attn_prefix_workspace_bytes(self.S, self.G, tokens, H, 1, d, self.pages[1] * PAGE, self.pages[0] * PAGE)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        return dict(kv=torch.zeros(tokens, self.C, **bf), score=torch.zeros(tokens, self.C, **bf), cu=torch.zeros(S + 1, **I32),
                    first=torch.zeros(S, **I32), source=torch.tensor(source, **I32), target=torch.tensor(target, **I32),
                    out=torch.zeros(rows, d, **bf), positions=torch.zeros(rows, **I32), slots=torch.zeros(rows, dtype=torch.int64, device="cuda"),
                    entries=torch.zeros(S, **I32), err=torch.zeros(1, **I32), q=torch.zeros(tokens, H, d, **bf), o=torch.zeros(tokens, H, d, **bf),
                    lse=torch.zeros(tokens, H, device="cuda"), ws=torch.zeros(ws, dtype=torch.uint8, device="cuda"))

    def fill(self, b, of, first, lens):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        for to, t in ((b["kv"], self.kv), (b["score"], self.score)):
            for i, s in enumerate(of):
                to[cu[i]:cu[i + 1]] = t[s, first[i]:first[i] + lens[i]].cuda()
        b["cu"].copy_(torch.tensor(cu))
        b["first"].copy_(torch.tensor(first))
        return cu

    def check_pooled(self, b, of, first, lens, was, table, base):
        assert int(b["err"]) == 0
        got, row = b["out"].double().cpu(), 0
        slots, positions = b["slots"].tolist(), b["positions"].tolist()
        for i, s in enumerate(of):
            for block in range(first[i] // self.ratio, (first[i] + lens[i]) // self.ratio):
                ref, bound = V.window_entry(self.kv[s], self.score[s], self.ape, block, self.ratio, self.coff, self.d)
                assert ((got[row] - ref).abs() <= bound).all()
                e = block - base[i]
                assert positions[row] == block * self.ratio and slots[row] == int(table[i, e // PAGE]) * PAGE + e % PAGE
                row += 1
        assert set(slots[row:]) <= {-1} and set(positions[row:]) <= {-1}
        check_append(b["out"].view(-1, 1, self.d), self.weight, 1, 1e-6, positions, self.turns, self.rot, self.d - self.rot, 1, self.amp,
                     slots, self.fmt, self.data, self.scales, was[0], was[1], self.num * PAGE)

    def was(self):
        return self.data.clone(), None if self.scales is None else self.scales.clone()

    def check_asked(self, b, cu, first, lens):
        if self.fmt == R.BF16:
            values = self.data.cpu().view(torch.bfloat16).double()
        else:
            values = R.dequantise(R.unpack(self.data.cpu(), self.fmt), self.scales.cpu().long(), self.fmt)
        lists = []
        for s, i in enumerate(self.group_of):
            shared = self.prompts[i] // self.ratio
            for t, row, n in ((self.tables[0], i, shared), (self.tables[1], s, (first[s] + lens[s]) // self.ratio - shared)):
                e = torch.arange(n)
                lists.append(t[row].long()[e // PAGE] * PAGE + e % PAGE)
        lists = [torch.cat(lists[k:k + 2]) for k in range(0, len(lists), 2)]
        table = torch.zeros(self.S, max([len(x) for x in lists] + [1]), dtype=torch.int64)
        for s, x in enumerate(lists):
            table[s, :len(x)] = x
        ref, rl, tol, ltol = R.attend(b["q"].cpu(), cu, values, table, 1, [len(x) for x in lists], first, self.ratio,
                                      self.d ** -0.5, self.sink)
        n = cu[-1]
        assert ((b["o"].double().cpu() - ref).abs() <= tol)[:n].all()
        fine = torch.isfinite(rl[:n])
        off = (b["lse"].double().cpu() - rl).abs()[:n]
        assert (off[fine] <= ltol[:n][fine]).all()

    def begin(self):
        of = [self.group_of.index(i) for i in range(self.G)]
        b = self.buffers(self.G, sum(self.prompts) + 1, [-1] * self.G, list(range(self.G)))
        self.fill(b, of, [0] * self.G, self.prompts)
        was = self.was()
        self.pooled(b, self.G, None, self.dtables[0], self.pages[0])
        self.prefix_entries.copy_(b["entries"])
        self.check_pooled(b, of, [0] * self.G, self.prompts, was, self.tables[0], [0] * self.G)
        assert self.prefix_entries.tolist() == [n // self.ratio for n in self.prompts]

    def call(self, b, lens, run):
        first = list(self.done)
        cu = self.fill(b, range(self.S), first, lens)
        b["q"].copy_(torch.randn(b["q"].shape, generator=self.gen))
        was = self.was()
        run()
        torch.cuda.synchronize()
        self.check_pooled(b, range(self.S), first, lens, was, self.tables[1], [self.prompts[i] // self.ratio for i in self.group_of])
        assert b["entries"].tolist() == [(f + n) // self.ratio - self.prompts[i] // self.ratio for f, n, i in zip(first, lens, self.group_of)]
        self.check_asked(b, cu, first, lens)
        self.done = [f + n for f, n in zip(first, lens)]


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("d,heads,ratio,coff", [(512, 64, 4, 2), (128, 16, 4, 2), (128, 8, 2, 1), (64, 4, 16, 1)])
def test_prompts_chunks_and_tokens(cuda_lib, fmt, d, heads, ratio, coff):
    """Chunks after the prompts, then single tokens, captured once and replayed until every sequence has
    completed blocks that reach into its state."""
    b = Batch(cuda_lib, [40 * ratio + 2, 3 * ratio - 1, ratio], [0, 0, 0, 1, 1, 2], 8 * ratio + 12, ratio, coff, d, heads, fmt, seed=d + ratio)
    b.begin()
    base = b.prefix_entries[b.dgroups].contiguous()
    own = [b.G + s for s in range(b.S)]

    def run(bufs):
        b.pooled(bufs, b.S, base, b.dtables[1], b.pages[1])
        b.asked(bufs)

    chunk = b.buffers(b.S, 5 * ratio + 24, [b.group_of[s] for s in range(b.S)], own)
    b.call(chunk, [5, ratio, 0, 1, 2 * ratio + 3, ratio - 1], lambda: run(chunk))
    chunk["source"].copy_(chunk["target"])
    b.call(chunk, [1, 0, 2 * ratio + 1, 2, 0, 1], lambda: run(chunk))

    one = b.buffers(b.S, b.S, own, own)
    b.call(one, [1] * b.S, lambda: run(one))
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        run(one)
    for _ in range(ratio + 3):
        b.call(one, [1] * b.S, graph.replay)


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 512), (4, 1, 64), (16, 2, 64), (128, 1, 128), (3, 2, 40)])
def test_stream_as_the_whole_pack(cuda_lib, ratio, coff, d):
    """Sequences pooled call by call give what csa_compressor_fwd gives for all of them at once, within both
    bounds."""
    g = torch.Generator().manual_seed(ratio)
    lens, C = [5 * ratio + 3, 2 * ratio, 9 * ratio + 1], coff * d
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    kv, score = (torch.randn(cu[-1], C, generator=g).to(torch.bfloat16) for _ in range(2))
    ape = 0.3 * torch.randn(ratio, C, generator=g)
    rows = sum(n // ratio for n in lens)
    whole = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    cuda_lib.csa_compressor_fwd(kv.cuda(), score.cuda(), ape.cuda(), torch.tensor(cu, **I32), len(lens), ratio, coff, d, cu[-1], whole, rows)
    kvs, scs = (torch.zeros(3, ratio * coff, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got, first, steps = [[] for _ in lens], [0] * 3, [1, ratio + 2, 1, 3 * ratio, 2, 9 * ratio]
    slot, err = torch.arange(3, **I32), torch.zeros(1, **I32)
    for n in steps:
        take = [min(n, m - f) for m, f in zip(lens, first)]
        tk, ts = (torch.cat([t[cu[s] + first[s]:cu[s] + first[s] + take[s]] for s in range(3)]).cuda() for t in (kv, score))
        c2 = [0, take[0], take[0] + take[1], sum(take)]
        made = [(f + k) // ratio - f // ratio for f, k in zip(first, take)]
        out = torch.zeros(sum(made) + 1, d, dtype=torch.bfloat16, device="cuda")
        cuda_lib.csa_compressor_step(tk, ts, ape.cuda(), torch.tensor(c2, **I32), 3, ratio, coff, d, max(1, sum(take)),
                                     torch.tensor(first, **I32), slot if any(first) else torch.full((3,), -1, **I32), slot, 3, kvs, scs, out,
                                     out.shape[0], None, None, 0, 1, 0, None, None, None, err)
        at = 0
        for s, m in enumerate(made):
            got[s].append(out[at:at + m].cpu())
            at += m
        first = [f + k for f, k in zip(first, take)]
    assert int(err) == 0 and first == lens
    whole, row = whole.cpu(), 0
    for s, parts in enumerate(got):
        for block, x in enumerate(torch.cat(parts)):
            ref, bound = V.window_entry(kv[cu[s]:], score[cu[s]:], ape, block, ratio, coff, d)
            assert ((x.double() - whole[row].double()).abs() <= 2 * bound).all()
            row += 1
    assert row == rows


def test_two_batches_at_once(cuda_lib):
    """Two captured batches, each with states, pages and a workspace of its own, replayed on two streams at the same
    time: the same bits as one after the other."""
    def make(seed):
        b = Batch(cuda_lib, [300, 64], [0] * 20 + [1] * 4, 80, 4, 2, 128, 16, R.E4M3, seed=seed)
        b.begin()
        base = b.prefix_entries[b.dgroups].contiguous()
        own = [b.G + s for s in range(b.S)]
        bufs = b.buffers(b.S, b.S * 3, [b.group_of[s] for s in range(b.S)], own)
        b.fill(bufs, range(b.S), list(b.done), [3] * b.S)
        bufs["q"].copy_(torch.randn(bufs["q"].shape, generator=b.gen))

        def run():
            b.pooled(bufs, b.S, base, b.dtables[1], b.pages[1])
            b.asked(bufs)
            bufs["first"] += 3
            bufs["source"].copy_(bufs["target"])
        return b, bufs, run

    kept = []
    for at_once in (False, True):
        pairs = [make(seed) for seed in (50, 51)]
        streams = [torch.cuda.Stream() for _ in pairs]
        graphs = []
        torch.cuda.synchronize()
        for (_, _, run), stream in zip(pairs, streams):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
                run()
            graphs.append(graph)
        torch.cuda.synchronize()
        for _ in range(20):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
                if not at_once:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        kept.append([t.clone() for b, bufs, _ in pairs for t in (b.data, b.kv_state, bufs["o"], bufs["lse"], bufs["out"], bufs["err"])])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*kept))
    assert int(kept[0][5]) == 0 and int(kept[0][11]) == 0


@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
def test_packed_call_replayed_on_other_lists(cuda_lib, fmt):
    """A captured call that packs its entries first, replayed on lists of other lengths than it was captured with."""
    from tests.test_gpu_attn_prefix import Case

    def make():
        return Case([(2000, [(5, 300)] * 60), (900, [(7, 90)] * 30)], 16, 1, 128, fmt, ratio=1, seed=60)
    one, two = make(), make()
    x, y = one.args(cuda_lib), two.args(cuda_lib)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            cuda_lib.csa_cache_attn_prefix(*y)
    torch.cuda.synchronize()
    new = dict(prefixes=[1290, 0], entries=[i * 3 for i in range(90)], first=[1500 + i for i in range(90)])
    for args in (x, y):
        args[16].copy_(torch.tensor(new["prefixes"]))
        args[21].copy_(torch.tensor(new["entries"][:60] + [e // 3 for e in new["entries"][60:]]))
        args[22].copy_(torch.tensor(new["first"]))
    cuda_lib.csa_cache_attn_prefix(*x)
    graph.replay()
    torch.cuda.synchronize()
    assert int(one.err) == 0 and torch.equal(one.out, two.out) and torch.equal(one.lse, two.lse)
    one.prefixes, one.first = new["prefixes"], new["first"]
    one.entries = new["entries"][:60] + [e // 3 for e in new["entries"][60:]]
    ref, _, tol, _ = one.reference()
    assert ((one.out.double().cpu() - ref).abs() <= tol)[:one.cu[-1]].all()
