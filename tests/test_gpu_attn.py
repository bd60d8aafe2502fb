"""Attention over the paged cache through the C ABI against the 64-bit reference: formats, head
layouts, lengths from none to many tiles, page sizes, masks that leave rows empty, sinks, strides,
non-finite values behind the mask, device-side refusals, graphs and repeated calls."""
import math

import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu


class Case:
    """One call's inputs on the CPU in the types they have, and the call."""

    def __init__(self, lens, entries, H, kv, d, fmt=R.BF16, page=16, ratio=1, first=None, sink=False, seed=0, lead=0,
                 pad=3, sharp=1.0, extra_pages=2):
        g = torch.Generator().manual_seed(seed)
        self.H, self.kv, self.d, self.fmt, self.page, self.ratio = H, kv, d, fmt, page, ratio
        self.S = len(lens)
        self.cu = [lead]
        for n in lens:
            self.cu.append(self.cu[-1] + n)
        self.tokens = self.cu[-1] + pad
        self.entries = list(entries)
        if first == "end":  # the last new token sees every entry
            first = [max(0, e * max(ratio, 1) - n) for n, e in zip(lens, entries)]
        self.first = first
        pages = [-(-e // page) for e in entries]
        self.max_pages = max(pages + [1]) + 1
        self.num_pages = sum(pages) + extra_pages
        order = torch.randperm(self.num_pages, generator=g)
        self.table = torch.full((self.S, self.max_pages), -77, dtype=torch.int32)
        at = 0
        for s, n in enumerate(pages):
            self.table[s, :n] = order[at:at + n]
            at += n
        slots = self.num_pages * page
        x = torch.randn(slots, kv, d, generator=g)
        if fmt == R.BF16:
            self.data, self.scales = x.to(torch.bfloat16), None
            self.values = self.data.double()
        else:
            codes, k = R.quantise(x.double(), fmt)
            self.data, self.scales = R.pack(codes, fmt), k.to(torch.uint8)
            self.values = R.dequantise(codes, k, fmt)
        self.q = (sharp * torch.randn(self.tokens, H, d, generator=g)).to(torch.bfloat16)
        self.sink = torch.randn(H, generator=g) if sink else None
        self.scale = 1.0 / math.sqrt(d)

    def run(self, gp, slab=0, shift=0, ws=None, keep=False):
        def dev(t):
            return None if t is None else t.cuda()
        T, H, d = self.tokens, self.H, self.d

        def shifted(t):
            flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
            v = flat[shift:shift + t.numel()].view(t.shape)
            v.copy_(t)
            return v
        q = torch.zeros(T, H + slab, d, dtype=torch.bfloat16)
        q[:, slab:] = self.q
        q = shifted(q)[:, slab:]
        out = shifted(torch.full((T, H + slab, d), 7.0, dtype=torch.bfloat16))[:, slab:]
        lse = torch.full((T, H), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if ws is None:
            n = gp.csa_cache_attn_workspace_bytes(self.S, T, H, self.kv, d, self.max_pages * self.page)
            assert n > 0
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        first = None if self.first is None else torch.tensor(self.first, **i32)
        args = (q, q.stride(0), q.stride(1), torch.tensor(self.cu, **i32), self.S, T, H, self.kv, d,
                shifted(self.data) if shift else dev(self.data), dev(self.scales), self.fmt, dev(self.table),
                self.max_pages, self.num_pages, self.page, torch.tensor(self.entries, **i32), first, self.ratio,
                self.scale, dev(self.sink), out, out.stride(0), out.stride(1), lse, ws, ws.numel(), err)
        gp.csa_cache_attn(*args)
        torch.cuda.synchronize()
        return (out, lse, int(err), args) if keep else (out, lse, int(err))

    def reference(self):
        return R.attend(self.q, self.cu, self.values, self.table, self.page, self.entries, self.first, self.ratio,
                        self.scale, self.sink)

    def check(self, gp, **how):
        out, lse, err = self.run(gp, **how)
        assert err == 0, err
        ref, rl, tol, ltol = self.reference()
        a, b = self.cu[0], self.cu[-1]
        got, gl = out.double().cpu(), lse.double().cpu()
        off = (got - ref).abs()[a:b]
        bad = ~(off <= tol[a:b])
        assert not bad.any(), (int(bad.sum()), [x[0].item() for x in bad.nonzero(as_tuple=True)], float(off.max()))
        fine = torch.isfinite(rl[a:b])
        assert torch.equal(gl[a:b][~fine], rl[a:b][~fine])  # -inf where nothing is seen and no sink
        assert ((gl - rl).abs()[a:b][fine] <= ltol[a:b][fine]).all()
        # rows of no sequence stay as they were
        rest = torch.cat([got[:a], got[b:]]), torch.cat([gl[:a], gl[b:]])
        assert all((t == 7.0).all() for t in rest)


SHAPES = [  # H, kv, d
    (64, 1, 512), (16, 1, 512), (1, 1, 128), (8, 2, 128), (12, 4, 64), (5, 1, 256), (128, 1, 128), (96, 1, 64),
    (6, 3, 40), (3, 1, 65), (2, 1, 1024), (4, 2, 320)]


@pytest.mark.parametrize("H,kv,d", SHAPES)
@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
def test_single_tokens(cuda_lib, H, kv, d, fmt):
    """A decoding batch: one token each (one sequence none), contexts of none to several tiles."""
    if fmt != R.BF16 and d % 32:
        pytest.skip("quantised formats take d in groups of 32")
    Case([1, 1, 0, 1, 1, 1], [700, 1, 40, 0, 128, 129], H, kv, d, fmt, first="end", sink=True, seed=d).check(cuda_lib)


@pytest.mark.parametrize("H,kv,d", SHAPES)
@pytest.mark.parametrize("ratio", [0, 1, 4, 128])
def test_chunks(cuda_lib, H, kv, d, ratio):
    """Chunks of new tokens: some from position 0, so that the first ones see nothing at larger ratios."""
    lens = [37, 0, 5, 70]
    entries = [n // max(ratio, 1) for n in lens] if ratio else [150, 7, 0, 300]
    first = [0, 0, 0, 0]
    if ratio:
        entries[2], first[2] = 190, 190 * ratio - 5
    Case(lens, entries, H, kv, d, ratio=ratio, first=first, seed=ratio + d, lead=2).check(cuda_lib)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 64, 100, 128, 256])
@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3])
def test_page_sizes(cuda_lib, page, fmt):
    Case([3, 1], [301, 258], 8, 2, 128, fmt, page=page, ratio=1, first="end", seed=page).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
def test_longer_chunk_512(cuda_lib, fmt):
    """Many row tiles over several entry tiles at the pooled entry's width, grouped heads, sinks."""
    Case([60, 21], [400, 130], 32, 2, 512, fmt, page=64, ratio=4, first="end", sink=True, seed=9).check(cuda_lib)


@pytest.mark.parametrize("entries", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 640])
@pytest.mark.parametrize("d", [128, 512])
def test_entry_counts(cuda_lib, entries, d):
    Case([2], [entries], 16, 1, d, ratio=0, seed=entries).check(cuda_lib)


@pytest.mark.parametrize("H,d", [(64, 512), (3, 65), (16, 128)])
def test_strides_and_alignment(cuda_lib, H, d):
    c = Case([9, 3], [140, 33], H, 1, d, ratio=1, first="end", seed=4)
    c.check(cuda_lib, slab=2)
    c.check(cuda_lib, shift=1)
    c.check(cuda_lib, slab=1, shift=8)


def test_sharp_and_growing_scores(cuda_lib):
    """Scores of tens that grow along the entries (the running maximum moves all the time), and a
    constant large offset."""
    for d in (128, 512):
        c = Case([2, 40], [500, 260], 16, 1, d, ratio=0, sharp=4.0, seed=3)
        ramp = torch.linspace(0.2, 3.0, c.values.shape[0])[torch.randperm(1).new_tensor(range(c.values.shape[0]))]
        c.data = (c.data.float() * ramp[:, None, None]).to(torch.bfloat16)
        c.values = c.data.double()
        c.check(cuda_lib)
        c.sink = torch.full((16,), 80.0)
        c.check(cuda_lib)
        c.sink = torch.full((16,), -200.0)
        c.check(cuda_lib)


@pytest.mark.parametrize("H,d", [(64, 512), (8, 128), (3, 65)])
def test_empty_rows(cuda_lib, H, d):
    """No entries at all, with and without a sink; tokens before the first complete block."""
    Case([4, 3], [0, 0], H, 1, d, ratio=0, seed=1).check(cuda_lib)
    Case([4, 3], [0, 5], H, 1, d, ratio=0, sink=True, seed=1).check(cuda_lib)
    Case([130, 6], [1, 0], H, 1, d, ratio=128, seed=1).check(cuda_lib)
    Case([5], [9], H, 1, d, ratio=1, first=[-40], sink=True, seed=1).check(cuda_lib)  # before the start: nothing


@pytest.mark.parametrize("H,d,fmt", [(64, 512, R.BF16), (8, 128, R.BF16), (3, 65, R.BF16), (16, 512, R.E4M3), (16, 128, R.FP4)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_entries_stay_behind_the_mask(cuda_lib, H, d, fmt, bad):
    """An entry with a NaN or infinity changes nothing for the tokens that do not see it, in the same
    tile and page, and slots of no sequence may hold anything."""
    c = Case([20], [40], H, 1, d, fmt, page=16, ratio=2, first=[55], seed=2)
    clean, lse, err = c.run(cuda_lib)
    assert err == 0
    ref = c.reference()[0]
    e = 33  # seen from position 67 on: by the tokens 12..19
    slot = int(c.table[0, e // c.page]) * c.page + e % c.page
    used = {int(c.table[0, i // c.page]) * c.page + i % c.page for i in range(40)}
    free = [s for s in range(c.num_pages * c.page) if s not in used]
    if fmt == R.BF16:
        c.data[slot, 0, d // 2] = bad
        c.data[free] = bad
    else:
        c.scales[slot, 0, 1] = 255
        c.scales[free] = 255
    got, glse, err = c.run(cuda_lib)
    assert err == 0
    assert torch.equal(got[:12], clean[:12]) and torch.equal(glse[:12], lse[:12])
    if not (bad == -float("inf") or bad == float("inf")):
        assert torch.isnan(got[12:20].float()).all()
    assert torch.isfinite(ref).all()


@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d,lens,page", [(64, 1, 512, [2], 16), (8, 2, 128, [3], 16), (8, 1, 96, [3], 5), (64, 1, 128, [9], 16)])
def test_every_code_and_scales_far_from_one(cuda_lib, fmt, H, kv, d, lens, page):
    """Random codes (all of them but NaN's) at scales from 2^-9 to 2^11, past the range in which one
    product with a bf16 factor widens them; then an e4m3 NaN code, which only its readers see."""
    c = Case(lens, [300], H, kv, d, fmt, page=page, ratio=0, seed=11)
    g = torch.Generator().manual_seed(12)
    slots = c.data.shape[0]
    codes = torch.randint(0, 256 if fmt == R.E4M3 else 16, (slots, kv, d), generator=g)
    if fmt == R.E4M3:
        codes[codes % 128 == 127] = 3
    k = torch.randint(118, 139, (slots, kv, d // 32), generator=g)
    c.data, c.scales = R.pack(codes, fmt), k.to(torch.uint8)
    c.values = R.dequantise(codes, k, fmt)
    c.scale = 1.0 / (float(c.values.abs().max()) * math.sqrt(d))
    c.check(cuda_lib)
    if fmt == R.E4M3:
        c.data[int(c.table[0, 0]) * page, 0, 5] = 0x7F
        out, _, err = c.run(cuda_lib)
        assert err == 0
        assert torch.isnan(out[:lens[0], :H // kv].float()).all() and torch.isfinite(out[:lens[0], H // kv:].float()).all()


def test_query_rows_are_apart(cuda_lib):
    for H, d in ((16, 512), (8, 128), (3, 65)):
        c = Case([12], [200], H, 1, d, ratio=1, first="end", seed=2)
        clean, lse, _ = c.run(cuda_lib)
        c.q[3, 1, 5], c.q[7, 2, 0] = float("nan"), float("inf")
        got, glse, _ = c.run(cuda_lib)
        rows = torch.ones(c.tokens, H, dtype=torch.bool)
        rows[3, 1] = rows[7, 2] = False
        assert torch.equal(got[rows], clean[rows]) and torch.equal(glse[rows.cuda()], lse[rows.cuda()])


@pytest.mark.parametrize("H,d", [(64, 512), (3, 65)])
def test_device_refusals(cuda_lib, H, d):
    gp = cuda_lib

    def fresh():
        return Case([4, 6], [40, 30], H, 1, d, ratio=1, first="end", seed=5)
    for cu, code in (([0, 6, 4], gp.CSA_DEVERR_CU_SEQLENS), ([-1, 4, 10], gp.CSA_DEVERR_CU_SEQLENS),
                     ([0, 4, 14], gp.CSA_DEVERR_CU_SEQLENS)):
        c = fresh()
        c.cu = cu
        out, lse, err = c.run(gp)
        assert err == code and (out == 7.0).all() and (lse == 7.0).all()
    for entries in ([-1, 3], [3, 16 * 5]):
        c = fresh()
        c.entries = entries
        out, lse, err = c.run(gp)
        assert err == gp.CSA_DEVERR_ENTRIES and (out == 7.0).all() and (lse == 7.0).all()
    for page in (-1, 10**9):
        c = fresh()
        good, _, _ = c.run(gp)
        c.table[0, 1] = page
        out, lse, err = c.run(gp)
        assert err == gp.CSA_DEVERR_PAGE
        assert torch.equal(out[4:10], good[4:10])  # the other sequence is untouched by it


@pytest.mark.parametrize("H,kv,d,lens", [(64, 1, 512, [1, 1, 1]), (64, 1, 512, [40, 25]), (8, 2, 128, [70, 1]), (3, 1, 65, [4])])
def test_repeats_and_graph(cuda_lib, H, kv, d, lens):
    """The same bits every time, with any workspace contents; and in a captured graph whose lengths
    and tables change between replays."""
    gp = cuda_lib
    a = Case(lens, [600] * len(lens), H, kv, d, ratio=1, first="end", sink=True, seed=5)
    out, lse, err, args = a.run(gp, keep=True)
    again, lse2, _ = a.run(gp)
    assert err == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        gp.csa_cache_attn(*args)
    b = Case(lens, [600] * len(lens), H, kv, d, ratio=1, first="end", sink=True, seed=6)
    b.entries = [max(0, 599 - 250 * i) for i in range(len(lens))]
    args[0].copy_(b.q)
    for at, src in ((9, b.data), (12, b.table), (16, torch.tensor(b.entries, dtype=torch.int32)), (20, b.sink)):
        args[at].copy_(src)
    args[21].fill_(7.0)
    args[24].fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    want, wl, _ = b.run(gp)
    assert torch.equal(args[21], want) and torch.equal(args[24], wl)


def test_offsets_past_32_bits(cuda_lib):
    """A pool of 4.3 GB whose last pages a sequence uses."""
    gp, d, page = cuda_lib, 512, 64
    pages = (1 << 32) // (page * d * 2) + 4
    data = torch.zeros(pages * page, 1, d, dtype=torch.bfloat16, device="cuda")
    c = Case([2], [100], 4, 1, d, page=page, ratio=0, seed=8)
    where = [pages - 1, pages - 2]
    for i, pg in enumerate(where):
        src = int(c.table[0, i]) * page
        data[pg * page:(pg + 1) * page] = c.data[src:src + page].cuda()
    out, lse, err, args = c.run(gp, keep=True)
    args = list(args)
    args[9], args[14] = data, pages
    args[12][0, :2] = torch.tensor(where, dtype=torch.int32)
    want = out.clone()
    args[21].fill_(0.0)
    gp.csa_cache_attn(*args)
    torch.cuda.synchronize()
    assert int(args[27]) == 0 and torch.equal(args[21][:2], want[:2])


def test_streams_apart(cuda_lib):
    """Two calls at once on two streams with workspaces of their own."""
    cases = [Case([1] * 4, [900] * 4, 64, 1, 512, ratio=0, seed=s) for s in (1, 2)]
    want = [c.run(cuda_lib)[0].clone() for c in cases]
    runs = [c.run(cuda_lib, keep=True) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for r in runs:
        r[3][21].fill_(0.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for r, s in zip(runs, streams):
            cuda_lib.csa_cache_attn(*r[3], stream=s)
    torch.cuda.synchronize()
    for r, w, c in zip(runs, want, cases):
        assert torch.equal(r[3][21][:c.cu[-1]], w[:c.cu[-1]])


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d,lens,entries,ratio", [
    (64, 1, 512, [70, 5, 0, 33], [530, 40, 9, 260], 4),   # units of 128 rows over several tiles, split over pairs
    (64, 1, 512, [9], [1500], 1),                         # few units: every unit in many pieces
    (16, 2, 128, [130, 3], [900, 400], 1),
    (8, 2, 256, [65, 64], [300, 129], 2),
    (20, 1, 192, [40], [700], 0),
    (24, 1, 64, [33, 90], [128, 1024], 1),
    (128, 1, 320, [3, 2], [257, 640], 0)])
def test_long_chunks(cuda_lib, fmt, H, kv, d, lens, entries, ratio):
    """Chunks long enough for packed entries and pairs of blocks, every format, odd row counts."""
    Case(lens, entries, H, kv, d, fmt, page=48, ratio=ratio, first="end", sink=True, seed=d + H).check(cuda_lib)


def test_many_sequences(cuda_lib):
    """The most sequences a call takes, most of them with a token and a few entries."""
    S = 16384
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 2, (S,), generator=g).tolist()
    entries = torch.randint(0, 6, (S,), generator=g).tolist()
    c = Case(lens, entries, 2, 1, 64, page=4, ratio=0, seed=3)
    out, lse, err = c.run(cuda_lib)
    assert err == 0
    some = [s for s in range(S) if lens[s]][::97] + [s for s in range(S) if lens[s]][-3:]
    for s in some:
        t, n = c.cu[s], entries[s]
        e = torch.arange(n)
        k = c.values[c.table[s].long()[e // 4] * 4 + e % 4, 0]
        x = c.q[t].double() @ k.T * c.scale
        want = torch.softmax(x, -1) @ k if n else torch.zeros(2, 64, dtype=torch.float64)
        # weights and output rounded to 16 bits (2^-8 each), scores of 64 fp32 products
        assert ((out[t].double().cpu() - want).abs() <= 2.1 * 2.0 ** -8 * (torch.softmax(x, -1) @ k.abs() if n else 1e-9)).all(), s


def test_a_table_much_larger_than_its_sequences(cuda_lib):
    """Chunks whose table could hold far more entries than there are."""
    c = Case([40, 30], [200, 90], 16, 1, 128, page=64, ratio=1, first="end", seed=6)
    wide = torch.full((2, 4000), -5, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table, c.max_pages = wide, 4000
    c.check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d", [(16, 1, 128), (8, 1, 256), (64, 1, 512)])
@pytest.mark.parametrize("entries", [[1030], [1500, 9], [3001, 0, 2500, 128, 129], [20500]])
def test_shares_of_long_contexts(cuda_lib, fmt, H, kv, d, entries):
    """One token over contexts that many workers share: units of two pieces to more than 32, the widest
    heads' entries by copies (short tables) and by threads (long ones)."""
    n = len(entries)
    Case([1] * n, entries, H, kv, d, fmt, page=64, ratio=0, sink=True, seed=sum(entries) + d).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d,lens", [(64, 1, 128, [5, 9]), (16, 2, 96, [60, 41, 3]), (32, 1, 256, [14, 0, 26]),
                                         (32, 1, 320, [13, 25])])
def test_packed_from_any_page(cuda_lib, fmt, H, kv, d, lens):
    """Chunks of enough rows to be packed, from pages that no tensor copy takes."""
    Case(lens, [430, 131, 255][:len(lens)], H, kv, d, fmt, page=9, ratio=1, first="end", sink=True,
         seed=H + d).check(cuda_lib)


@pytest.mark.parametrize("d", [128, 512])
def test_joins_of_pieces_that_see_nothing(cuda_lib, d):
    """Rows whose early positions hide most of a shared unit's entries, or all: some pieces, then every one, weigh
    nothing."""
    c = Case([40], [3000], 16, 1, d, page=64, ratio=1, first=[30], seed=d)
    c.check(cuda_lib)
    c = Case([40], [3000], 16, 1, d, page=64, ratio=1, first=[2950], seed=d)
    c.check(cuda_lib)
    c = Case([3, 2], [2600, 2600], 16, 1, d, page=64, ratio=64, first=[0, 70], sink=True, seed=d)
    c.check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,kv,d,page", [(64, 1, 512, 64), (64, 2, 256, 16), (128, 1, 128, 48), (64, 1, 512, 9),
                                         (64, 1, 256, 9), (128, 1, 128, 9)])
def test_many_units_of_chunks(cuda_lib, fmt, H, kv, d, page):
    """More units than workers, each worker going from one to the next: the next one's rows come while one's go."""
    Case([170, 1, 150, 0, 60], [430, 260, 129, 40, 1], H, kv, d, fmt, page=page, ratio=1, first="end", sink=True,
         seed=d + page).check(cuda_lib)


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("H,d,page", [(64, 512, 64), (20, 256, 16), (8, 128, 64), (64, 512, 3)])
def test_many_units_of_single_tokens(cuda_lib, fmt, H, d, page):
    """Several sequences to a worker, some of no entries, some of no token."""
    g = torch.Generator().manual_seed(d + H)
    S = 500
    lens = (torch.rand(S, generator=g) < 0.9).int().tolist()
    entries = torch.randint(0, 400, (S,), generator=g).tolist()
    entries[3] = entries[77] = 0
    Case(lens, entries, H, 1, d, fmt, page=page, ratio=0, sink=d == 256, seed=d).check(cuda_lib)
