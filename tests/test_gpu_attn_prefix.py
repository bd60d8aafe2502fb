"""Attention behind shared prefixes through the C ABI against the 64-bit reference over each sequence's whole list
of entries: formats, head layouts, groups that are empty, alone or many, prefixes and own entries from none to
many tiles, tokens that do not see all of a prefix, sequences without a token, every way that a tile comes in,
strides, values out of the ordinary, refusals on the device, a wait that runs out, graphs, and agreement with
csa_cache_attn."""
import math
import random

import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


class Case:
    """groups: [(prefix entries, [(new tokens, own entries), ...]), ...]; first "end": the last token sees all."""

    def __init__(self, groups, H, kv, d, fmt=R.BF16, page=16, ratio=0, first="end", sink=False, seed=0, lead=0, pad=2, sharp=1.0,
                 extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.H, self.kv, self.d, self.fmt, self.page, self.ratio = H, kv, d, fmt, page, ratio
        self.prefixes = [p for p, _ in groups]
        self.lens = [n for _, seqs in groups for n, _ in seqs]
        self.entries = [e for _, seqs in groups for _, e in seqs]
        self.cuts = [0]
        for _, seqs in groups:
            self.cuts.append(self.cuts[-1] + len(seqs))
        self.group_of = [i for i, (_, seqs) in enumerate(groups) for _ in seqs]
        self.S, self.G = len(self.lens), len(groups)
        self.cu = [lead]
        for n in self.lens:
            self.cu.append(self.cu[-1] + n)
        self.tokens = self.cu[-1] + pad
        if first == "end":
            first = [max(0, (self.prefixes[self.group_of[s]] + self.entries[s]) * max(ratio, 1) - self.lens[s]) for s in range(self.S)]
        self.first = first
        self.num_pages = sum(-(-n // page) for n in self.prefixes + self.entries) + extra_pages
        order = torch.randperm(self.num_pages, generator=g)
        at = 0
        self.tables = []
        for counts in (self.prefixes, self.entries):
            table = torch.full((max(len(counts), 1), max([-(-n // page) for n in counts] + [0]) + 1), -77, dtype=torch.int32)
            for s, n in enumerate(counts):
                k = -(-n // page)
                table[s, :k] = order[at:at + k]
                at += k
            self.tables.append(table)
        x = torch.randn(self.num_pages * page, kv, d, generator=g)
        if fmt == R.BF16:
            self.data, self.scales = x.to(torch.bfloat16), None
        else:
            codes, k = R.quantise(x.double(), fmt)
            self.data, self.scales = R.pack(codes, fmt), k.to(torch.uint8)
        self.q = (sharp * torch.randn(self.tokens, H, d, generator=g)).to(torch.bfloat16)
        self.sink = torch.randn(H, generator=g) if sink else None
        self.scale = 1.0 / math.sqrt(d)

    def values(self):
        if self.fmt == R.BF16:
            return self.data.double()
        return R.dequantise(R.unpack(self.data, self.fmt), self.scales.long(), self.fmt)

    def slots(self, table, n):
        e = torch.arange(n)
        return table.long()[e // self.page] * self.page + e % self.page

    def args(self, gp, slab=0, shift=0, ws=None):
        def dev(t):
            return None if t is None else t.cuda()

        def shifted(t):
            flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
            v = flat[shift:shift + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        T, H, d = self.tokens, self.H, self.d
        q = torch.zeros(T, H + slab, d, dtype=torch.bfloat16)
        q[:, slab:] = self.q
        q = shifted(q)[:, slab:]
        out = shifted(torch.full((T, H + slab, d), 7.0, dtype=torch.bfloat16))[:, slab:]
        lse, err = torch.full((T, H), 7.0, device="cuda"), torch.zeros(1, **I32)
        pre, own = (t.shape[1] for t in self.tables)
        if ws is None:
            n = gp.csa_cache_attn_prefix_workspace_bytes(self.S, self.G, T, H, self.kv, d, own * self.page, pre * self.page)
            assert n > 0
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        first = None if self.first is None else torch.tensor(self.first, **I32)
        self.out, self.lse, self.err = out, lse, err
        return (q, q.stride(0), q.stride(1), torch.tensor(self.cu, **I32), self.S, T, H, self.kv, d,
                shifted(self.data) if shift else dev(self.data), dev(self.scales), self.fmt, torch.tensor(self.cuts, **I32), self.G,
                dev(self.tables[0]), pre, torch.tensor(self.prefixes, **I32), dev(self.tables[1]), own, self.num_pages, self.page,
                torch.tensor(self.entries, **I32), first, self.ratio, self.scale, dev(self.sink), out, out.stride(0), out.stride(1), lse,
                ws, ws.numel(), err)

    def run(self, gp, **how):
        gp.csa_cache_attn_prefix(*self.args(gp, **how))
        torch.cuda.synchronize()
        return self.out, self.lse, int(self.err)

    def reference(self):
        """Each sequence's whole list, as slots of pages of one entry."""
        lists = [torch.cat([self.slots(self.tables[0][self.group_of[s]], self.prefixes[self.group_of[s]]),
                            self.slots(self.tables[1][s], self.entries[s])]) for s in range(self.S)]
        table = torch.zeros(self.S, max([len(x) for x in lists] + [1]), dtype=torch.int64)
        for s, x in enumerate(lists):
            table[s, :len(x)] = x
        return R.attend(self.q, self.cu, self.values(), table, 1, [len(x) for x in lists], self.first, self.ratio, self.scale, self.sink)

    def check(self, gp, **how):
        out, lse, err = self.run(gp, **how)
        assert err == 0, err
        ref, rl, tol, ltol = self.reference()
        a, b = self.cu[0], self.cu[-1]
        got, gl = out.double().cpu(), lse.double().cpu()
        bad = ~((got - ref).abs() <= tol)[a:b]
        assert not bad.any(), (int(bad.sum()), [x[0].item() for x in bad.nonzero(as_tuple=True)], float((got - ref).abs()[a:b].max()))
        fine = torch.isfinite(rl[a:b])
        assert torch.equal(gl[a:b][~fine], rl[a:b][~fine])
        assert ((gl - rl).abs()[a:b][fine] <= ltol[a:b][fine]).all()
        assert all((t == 7.0).all() for t in (got[:a], got[b:], gl[:a], gl[b:]))


SHAPES = [(64, 1, 512), (16, 1, 512), (1, 1, 128), (8, 2, 128), (12, 4, 64), (5, 1, 256), (128, 1, 128), (96, 1, 64), (6, 3, 40),
          (3, 1, 65), (2, 1, 1024), (4, 2, 320)]


@pytest.mark.parametrize("H,kv,d", SHAPES)
@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
def test_decoding(cuda_lib, H, kv, d, fmt):
    if fmt != R.BF16 and d % 32:
        pytest.skip("codes need groups of 32")
    Case([(200, [(1, 5), (1, 0), (1, 131), (1, 33)]), (0, [(1, 40)]), (128, []), (129, [(1, 0), (0, 7), (1, 2)])], H, kv, d, fmt,
         seed=H + d).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 128])
@pytest.mark.parametrize("H,kv,d", [(16, 2, 128), (64, 1, 512), (4, 1, 256)])
def test_pages_of_any_size(cuda_lib, fmt, page, H, kv, d):
    """Few rows (threads or copies fetch the tiles) and many (packed entries), tails inside pages and tiles."""
    Case([(300, [(1, 20), (2, 0), (1, 3)]), (77, [(1, 61)])], H, kv, d, fmt, page=page, sink=True, seed=page).check(cuda_lib)
    Case([(290, [(9, 20), (17, 1), (30, 64), (1, 5)]), (131, [(40, 9), (3, 30)])], H, kv, d, fmt, page=page, seed=page).check(cuda_lib)


@pytest.mark.parametrize("ratio", [1, 4, 128])
@pytest.mark.parametrize("H,kv,d", [(8, 1, 128), (64, 1, 512), (3, 1, 65), (2, 2, 64)])
def test_tokens_see_what_is_complete(cuda_lib, ratio, H, kv, d):
    """Prefixes that some, and that all tokens see in part, own entries that come into sight token by token."""
    groups = [(150, [(3, 4), (1, 0), (7, 3), (0, 9)]), (10, [(2, 140), (5, 1)])]
    Case(groups, H, kv, d, ratio=ratio, sink=True).check(cuda_lib)
    Case(groups, H, kv, d, ratio=ratio, first=None).check(cuda_lib)
    Case(groups, H, kv, d, ratio=ratio, first=[149 * ratio, 0, 150 * ratio - 2, 5, 9 * ratio, 2 ** 31 - 9]).check(cuda_lib)
    Case(groups, H, kv, d, ratio=ratio, first=[3, 140 * ratio, 0, 0, 5 * ratio, 0], sink=True, fmt=R.E4M3 if d % 32 == 0 else R.BF16).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
@pytest.mark.parametrize("H,kv,d", [(1, 1, 64), (4, 1, 128), (64, 1, 512), (2, 1, 256), (2, 1, 40)])
def test_many_sequences_in_a_unit(cuda_lib, fmt, H, kv, d):
    if fmt != R.BF16 and d % 32:
        pytest.skip("codes need groups of 32")
    rng = random.Random(H)
    for n in (70, 9):
        Case([(rng.choice([0, 100, 257]), [(rng.choice([0, 1, 1, 1, 2]), rng.choice([0, 1, 30, 129])) for _ in range(n)]) for _ in range(3)], H,
             kv, d, fmt, seed=n, lead=3).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d", [(64, 1, 512), (8, 1, 128), (8, 1, 256)])
def test_long_prefixes_are_shared_by_workers(cuda_lib, fmt, H, kv, d):
    """Units of many tiles, cut between workers in a prefix, in own entries and between them."""
    Case([(9000, [(1, 300), (1, 1000), (1, 0)]), (2500, [(1, 2000)])], H, kv, d, fmt, page=64, sink=True, seed=2).check(cuda_lib)
    Case([(5000, [(4, 10), (5, 400)] * 3)], H, kv, d, fmt, page=64, ratio=1, seed=3).check(cuda_lib)


@pytest.mark.parametrize("H,kv,d,slab,shift", [(8, 2, 128, 2, 0), (8, 1, 128, 1, 8), (4, 1, 64, 0, 1), (64, 1, 512, 3, 0)])
def test_strides_and_alignment(cuda_lib, H, kv, d, slab, shift):
    Case([(140, [(2, 30), (1, 3)]), (20, [(1, 9)])], H, kv, d).check(cuda_lib, slab=slab, shift=shift)


def test_a_group_for_each_sequence(cuda_lib):
    Case([(s * 7 % 50, [(s % 3, s % 11)]) for s in range(300)], 4, 1, 64, seed=5).check(cuda_lib)
    Case([(31, [(1, s % 4) for s in range(5000)])], 1, 1, 32, seed=6).check(cuda_lib)  # (more sequences than the plan holds in shared memory)


def test_scores_far_from_zero(cuda_lib):
    for sharp in (40.0, 1e4):
        Case([(260, [(1, 9), (1, 130), (2, 0)])], 8, 1, 128, sharp=sharp, seed=7).check(cuda_lib)


@pytest.mark.parametrize("H,kv,d", [(64, 1, 512), (16, 1, 128), (4, 1, 256), (6, 1, 72)])
@pytest.mark.parametrize("page", [16, 3])
def test_values_out_of_the_ordinary(cuda_lib, H, kv, d, page):
    """An own entry with a NaN reaches its own sequence's rows alone, whatever others share their tiles; one of
    a prefix reaches the tokens that see it; what nobody sees, in pages and behind them, reaches none."""
    def poisoned(group, index, own):
        c = Case([(200, [(1, 40), (1, 3), (2, 140)]), (140, [(1, 9), (1, 1)])], H, kv, d, page=page, seed=8, ratio=1)
        clean = c.run(cuda_lib)[0].clone()
        table, n = (c.tables[1], c.entries) if own else (c.tables[0], c.prefixes)
        slot = int(table[group, index // page]) * page + index % page
        c.data[slot, 0, d // 3] = math.nan if index % 2 else math.inf
        return c, clean, c.run(cuda_lib)
    for s, index in ((0, 39), (1, 2), (2, 0), (2, 131), (3, 8), (4, 0)):
        c, clean, (out, lse, err) = poisoned(s, index, True)
        assert err == 0
        hit = torch.zeros(c.tokens, dtype=torch.bool)
        hit[c.cu[s]:c.cu[s + 1]] = True
        if (s, index) == (2, 139):
            hit[c.cu[2]] = False
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all(), (s, index)
        assert torch.equal(out[~hit].cpu(), clean[~hit].cpu()), (s, index)
    for g, index in ((0, 5), (0, 199), (1, 139)):
        c, clean, (out, lse, err) = poisoned(g, index, False)
        hit = torch.zeros(c.tokens, dtype=torch.bool)
        hit[c.cu[c.cuts[g]]:c.cu[c.cuts[g + 1]]] = True
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit].cpu(), clean[~hit].cpu())
    c = Case([(200, [(1, 40), (1, 3), (2, 140)])], H, kv, d, page=page, seed=9, ratio=1, first=[120, 300, 190])
    clean = c.run(cuda_lib)[0].clone()
    c.data[int(c.tables[0][0, 199 // page]) * page + 199 % page] = math.nan  # seen from the second sequence alone
    c.data[int(c.tables[1][0, 0]) * page] = math.nan                        # seen from nowhere
    out = c.run(cuda_lib)[0]
    assert torch.isnan(out[1]).all() and torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])


WAYS = [(R.BF16, 16, 16, 2, 128, 0), (R.BF16, 3, 8, 1, 64, 0), (R.BF16, 16, 64, 1, 512, 0), (R.E4M3, 16, 16, 1, 128, 0), (R.E4M3, 16, 64, 1, 512, 0),
        (R.E4M3, 16, 64, 1, 128, 70), (R.FP4, 8, 4, 1, 256, 0), (R.BF16, 16, 4, 1, 65, 0)]
SOME = [(200, [(1, 40), (3, 140), (2, 0), (0, 3)]), (0, [(1, 0), (4, 130)]), (129, [(1, 1)] * 5)]


@pytest.mark.parametrize("fmt,page,H,kv,d,more", WAYS)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.3, 1e-30])
def test_scales_of_zero_and_below(cuda_lib, fmt, page, H, kv, d, more, scale):
    """A scale of 0 weighs all entries alike that a token sees, a negative one turns their order, a tiny one is no mask."""
    for sink in (False, True):
        c = Case(SOME + [(300, [(more, 90)])], H, kv, d, fmt, page=page, ratio=1, sink=sink, seed=61)
        c.scale = scale
        c.check(cuda_lib)


@pytest.mark.parametrize("fmt,page,H,kv,d,more", WAYS)
@pytest.mark.parametrize("long", [False, True])
def test_sinks_that_are_not_finite(cuda_lib, fmt, page, H, kv, d, more, long):
    """A sink of -inf is none, one of +inf takes all the weight (out 0, lse +inf), one of NaN makes NaN; in units by
    themselves and in ones that workers share."""
    groups = [(9000 if long else 200, SOME[0][1])] + SOME[1:] + [(300, [(more, 90)])]
    c, free, held = (Case(groups, H, kv, d, fmt, page=page, ratio=1, sink=True, seed=62) for _ in range(3))
    kind = torch.arange(H) % 4
    held.sink = torch.full((H,), 1.5)
    c.sink = torch.tensor([math.inf, math.nan, -math.inf, 1.5])[kind]
    free.sink = None
    out, lse, err = c.run(cuda_lib)
    assert err == 0
    n = c.cu[-1]
    out, lse = out.double().cpu()[:n], lse.double().cpu()[:n]
    sees = torch.isfinite(free.reference()[1][:n])  # (a token that sees nothing: out 0 and lse the sink)
    assert (out[:, kind == 0] == 0).all() and (lse[:, kind == 0] == math.inf).all()
    nan = kind == 1
    assert torch.isnan(lse[:, nan]).all() and torch.isnan(out[:, nan][sees[:, nan]]).all() and (out[:, nan][~sees[:, nan]] == 0).all()
    for k, like in ((2, free), (3, held)):
        ref, rl, tol, ltol = (x[:n][:, kind == k] for x in like.reference())
        assert ((out[:, kind == k] - ref).abs() <= tol).all()
        fine = torch.isfinite(rl)
        assert torch.equal(lse[:, kind == k][~fine], rl[~fine]) and ((lse[:, kind == k] - rl).abs()[fine] <= ltol[fine]).all()


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
@pytest.mark.parametrize("H,kv,d", [(64, 1, 512), (16, 1, 128), (6, 1, 72), (3, 1, 128), (4, 2, 256), (1, 1, 64), (2, 1, 65)])
@pytest.mark.parametrize("page,more", [(16, 0), (3, 0), (16, 60)])
def test_own_entries_that_later_tokens_alone_see(cuda_lib, fmt, H, kv, d, page, more):
    """A NaN or an infinity in an own entry that only a sequence's later tokens see, by the tile kernels' ways in
    (`more`: tokens of other sequences, for which entries are packed): those tokens are NaN in the heads that read it, and
    all others as they were, the same sequence's earlier ones in the same rows of a tile too."""
    if fmt != R.BF16 and d % 32:
        pytest.skip("codes need groups of 32")
    groups = [(200, [(1, 40), (5, 140), (3, 7)] + [(more, 300)] * (more > 0)), (0, [(4, 130)])]

    def case():
        return Case(groups, H, kv, d, fmt, page=page, seed=51, ratio=1, sink=True)
    clean, clean_lse, err = case().run(cuda_lib)
    assert err == 0
    clean, clean_lse = clean.cpu(), clean_lse.cpu()
    for s, back in ((1, 0), (1, 2), (1, 3), (2, 1), (len(groups[0][1]), 0), (len(groups[0][1]), 2)):
        c = case()
        index = c.entries[s] - 1 - back  # seen from the sequence's token lens[s] - 1 - back on
        slot, head = int(c.tables[1][s, index // page]) * page + index % page, kv - 1
        if fmt == R.BF16:
            c.data[slot, head, d // 3] = math.nan if back % 2 else -math.inf
        else:
            c.data[slot, head, d // 3] = 0x7F
        out, lse, err = c.run(cuda_lib)
        assert err == 0
        hit = torch.zeros(c.tokens, H, dtype=torch.bool)
        hit[c.cu[s] + c.lens[s] - 1 - back:c.cu[s + 1], head * (H // kv):] = True
        out, lse = out.cpu(), lse.cpu()
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all(), (s, back)
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit]), (s, back)


@pytest.mark.parametrize("d", [64, 65])
def test_device_refusals(cuda_lib, d):
    def case():
        return Case([(40, [(1, 9), (2, 3)]), (7, [(1, 0)])], 2, 1, d)
    for code, name, value in ((1, "cu", [0, 2, 1, 4]), (1, "cu", [0, 1, 3, 99]), (6, "entries", [9, -1, 0]), (6, "entries", [9, 999, 0]),
                              (9, "prefixes", [40, -1]), (9, "prefixes", [999, 7]), (9, "cuts", [0, 4, 3]), (9, "cuts", [1, 2, 3]),
                              (9, "cuts", [0, 2, 2]), (9, "cuts", [0, -1, 3])):
        c = case()
        c.tokens = 6
        c.q = c.q[:1].expand(6, -1, -1).contiguous()
        setattr(c, name, value)
        out, lse, err = c.run(cuda_lib)
        assert err == code and (out == 7).all() and (lse == 7).all(), (name, value, err)
    for which, at in ((0, (0, 2)), (1, (1, 0))):
        for bad in (-1, 10 ** 6):
            c = case()
            c.tables[which][at] = bad
            out, lse, err = c.run(cuda_lib)
            assert err == 7
            c2 = case()
            ref = c2.run(cuda_lib)[0]
            assert torch.equal(out[3], ref[3])  # the other group's


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
@pytest.mark.parametrize("H,kv,d", [(64, 1, 512), (8, 2, 128)])
def test_as_without_prefixes(cuda_lib, fmt, H, kv, d):
    """Prefixes of nothing: the same as csa_cache_attn, within both tolerances."""
    c = Case([(0, [(1, 90), (3, 300)]), (0, [(2, 129)])], H, kv, d, fmt, ratio=1, sink=True, seed=11)
    c.check(cuda_lib)
    out, lse, _ = c.run(cuda_lib)
    a = list(c.args(cuda_lib))
    ws = torch.empty(cuda_lib.csa_cache_attn_workspace_bytes(c.S, c.tokens, H, kv, d, a[18] * c.page), dtype=torch.uint8, device="cuda")
    cuda_lib.csa_cache_attn(*a[:12], *a[17:30], ws, ws.numel(), a[32])
    torch.cuda.synchronize()
    _, _, tol, ltol = c.reference()
    n = c.cu[-1]
    assert ((out - c.out).abs().double().cpu()[:n] <= 2 * tol[:n]).all() and ((lse - c.lse).abs().double().cpu()[:n] <= 2 * ltol[:n]).all()


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d,page", [(16, 2, 128, 16), (8, 1, 64, 4), (8, 1, 256, 16), (64, 1, 512, 4)])
def test_full_tables_and_exact_workspaces(cuda_lib, fmt, H, kv, d, page):
    """Chunks whose entries fill every table (and every place that the call may pack them in): right, by both entry
    points, and nothing behind a workspace of exactly the size that is asked for is touched."""
    def spare(n):
        ws = torch.full((n + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
        return ws, ws[:n]
    c = Case([(512, [(200, 256), (330, 256), (3, 256)]), (512, [(410, 256)])], H, kv, d, fmt, page=page, ratio=1, seed=21, lead=3)
    c.tables = [t[:, :-1].contiguous() for t in c.tables]  # (the tables are as wide as what they hold)
    n = cuda_lib.csa_cache_attn_prefix_workspace_bytes(c.S, c.G, c.tokens, H, kv, d, 256, 512)
    ws, view = spare(n)
    c.check(cuda_lib, ws=view)
    assert (ws[n:] == 0x5A).all()
    c = Case([(0, [(200, 384), (330, 384), (384, 384)])], H, kv, d, fmt, page=page, ratio=1, seed=22)
    c.tables = [c.tables[0], c.tables[1][:, :-1].contiguous()]
    a = list(c.args(cuda_lib))
    n = cuda_lib.csa_cache_attn_workspace_bytes(c.S, c.tokens, H, kv, d, 384)
    ws, view = spare(n)
    cuda_lib.csa_cache_attn(*a[:12], *a[17:30], view, n, a[32])
    torch.cuda.synchronize()
    assert (ws[n:] == 0x5A).all() and int(c.err) == 0
    ref, rl, tol, ltol = c.reference()
    end = c.cu[-1]
    assert ((c.out.double().cpu() - ref).abs() <= tol)[:end].all() and ((c.lse.double().cpu() - rl).abs() <= ltol)[:end].all()


@pytest.mark.parametrize("d", [128, 512])
def test_workspace_without_room_to_pack(cuda_lib, d):
    """bf16 in pages of a multiple of 8 needs what the query gives for no entries, and touches nothing behind it; codes and
    other pages are refused with that, and bf16 with less."""
    def case(fmt, page):
        return Case([(2048, [(1, 700)] * 40)], 64, 1, d, fmt, page=page, ratio=1, seed=41)
    c = case(R.BF16, 64)
    own, pre = c.tables[1].shape[1] * 64, c.tables[0].shape[1] * 64
    full = cuda_lib.csa_cache_attn_prefix_workspace_bytes(c.S, c.G, c.tokens, 64, 1, d, own, pre)
    n = cuda_lib.csa_cache_attn_prefix_workspace_bytes(c.S, c.G, c.tokens, 64, 1, d, 0, 0)
    assert n + (c.S * own + pre) * d * 2 <= full + (1 << 20)  # (the packed entries are what it lacks)
    ws = torch.full((n + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    c.check(cuda_lib, ws=ws[:n])
    assert (ws[n:] == 0x5A).all()
    for fmt, page in ((R.E4M3, 64), (R.BF16, 7)):
        c = case(fmt, page)
        with pytest.raises(cuda_lib.CsaError) as e:
            c.run(cuda_lib, ws=ws[:n])
        assert e.value.status == cuda_lib.CSA_ERR_WORKSPACE and (c.out == 7.0).all()
    with pytest.raises(cuda_lib.CsaError) as e:
        case(R.BF16, 64).run(cuda_lib, ws=ws[:n // 2])
    assert e.value.status == cuda_lib.CSA_ERR_WORKSPACE


def test_repeats_and_graph(cuda_lib):
    """The same bits from the same inputs; a captured call replayed on other lengths than it was captured with."""
    def make():
        return Case([(700, [(1, 90), (1, 30)]), (300, [(1, 129), (1, 16)])], 8, 1, 128, R.E4M3, ratio=1, sink=True, seed=12)
    c = make()
    a, b = c.run(cuda_lib), make().run(cuda_lib)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one, two = make(), make()
    x, y = one.args(cuda_lib), two.args(cuda_lib)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        cuda_lib.csa_cache_attn_prefix(*y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            cuda_lib.csa_cache_attn_prefix(*y)
    torch.cuda.synchronize()
    for args in (x, y):
        args[21].copy_(torch.tensor([80, 5, 100, 1]))   # entries
        args[16].copy_(torch.tensor([512, 77]))         # prefixes
        args[22].copy_(torch.tensor([600, 500, 90, 400]))  # first
    cuda_lib.csa_cache_attn_prefix(*x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(one.out, two.out) and torch.equal(one.lse, two.lse) and int(two.err) == 0
    one.entries, one.prefixes, one.first = [80, 5, 100, 1], [512, 77], [600, 500, 90, 400]
    ref, _, tol, _ = one.reference()
    assert ((one.out.double().cpu() - ref).abs() <= tol)[:4].all()


@pytest.mark.parametrize("H,kv", [(1, 1), (4, 2), (3, 1)])
def test_chunks_beside_single_tokens(cuda_lib, H, kv):
    """Few sequences in most blocks of 64 rows and many in some."""
    Case([(70, [(700, 30)] + [(1, i % 9) for i in range(60)]), (0, [(1, 3)] * 5), (200, [(0, 4)] * 70 + [(2, 140), (900, 9)])], H, kv, 64,
         page=8, ratio=1, seed=33, lead=1).check(cuda_lib)


@pytest.mark.parametrize("groups,seqs", [(16384, 1), (12300, 1300), (16384, 300), (16000, 700), (1, 4200), (1300, 16384)])
def test_most_groups_and_sequences(cuda_lib, groups, seqs):
    """Group and sequence lists of any size, most of the one empty or all of the other alone."""
    rng = random.Random(groups + seqs)
    some = sorted(rng.randrange(groups) for _ in range(seqs))
    lists = [[] for _ in range(groups)]
    for g in some:
        lists[g].append((1 if rng.random() < 0.9 else 0, rng.randrange(0, 20)))
    Case([(rng.randrange(0, 9) if x else 0, x) for x in lists], 2, 1, 64, page=8, seed=31).check(cuda_lib)


@pytest.mark.parametrize("fmt,lens", [(R.BF16, 1), (R.E4M3, 1), (R.E4M3, 40)])
def test_a_wait_that_runs_out(cuda_lib, fmt, lens):
    """A tile that never comes in: the call returns, reports it, leaves other rows alone, and the next one is right."""
    c = Case([(500, [(lens, 20), (lens, 3)])], 64, 1, 128, fmt, page=64, seed=13)
    before = c.run(cuda_lib)[0].clone()
    cuda_lib.csa_compressor_test_hooks(20000000, 0)
    try:
        out, _, err = c.run(cuda_lib)
        assert err == cuda_lib.CSA_DEVERR_TIMEOUT and (out[c.cu[-1]:] == 7).all()
    finally:
        cuda_lib.csa_compressor_test_hooks(0, -1)
    out, _, err = c.run(cuda_lib)
    assert err == 0 and torch.equal(out, before)


@pytest.mark.parametrize("d", [32, 48])
def test_long_lists(cuda_lib, d):
    """Prefixes whose entries' bytes pass 32 bits in the pool."""
    page, kv = 64, 4
    slots = (1 << 32) // (kv * d * 2) // page * page + 64 * page
    data = torch.zeros(slots, kv, d, dtype=torch.bfloat16, device="cuda")
    n = slots // page
    g = torch.Generator().manual_seed(14)
    far = torch.randn(2 * page, kv, d, generator=g).to(torch.bfloat16)
    data[-2 * page:] = far.cuda()
    table, own = torch.tensor([[n - 2, n - 1]], **I32), torch.tensor([[n - 1], [n - 2]], **I32)
    q = torch.randn(2, 8, d, generator=g).to(torch.bfloat16)
    out = torch.zeros(2, 8, d, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, **I32)
    t = lambda v: torch.tensor(v, **I32)  # noqa: E731
    ws = torch.empty(cuda_lib.csa_cache_attn_prefix_workspace_bytes(2, 1, 2, 8, kv, d, page, 2 * page), dtype=torch.uint8, device="cuda")
    cuda_lib.csa_cache_attn_prefix(q.cuda(), 8 * d, d, t([0, 1, 2]), 2, 2, 8, kv, d, data, None, 0, t([0, 2]), 1, table, 2, t([100]), own, 1, n,
                                   page, t([9, 64]), None, 0, 0.2, None, out, 8 * d, d, None, ws, ws.numel(), err)
    torch.cuda.synchronize()
    assert int(err) == 0
    lists = [torch.cat([torch.arange(100), torch.arange(page, page + 9)]), torch.cat([torch.arange(100), torch.arange(64)])]
    tab = torch.zeros(2, 164, dtype=torch.int64)
    for s, x in enumerate(lists):
        tab[s, :len(x)] = x
    ref, _, tol, _ = R.attend(q, [0, 1, 2], far.double(), tab, 1, [109, 164], None, 0, 0.2, None)
    assert ((out.double().cpu() - ref).abs() <= tol).all()
