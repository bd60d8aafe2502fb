"""Pooling of a stream through the C ABI against the 64-bit windows: calls of one and of many tokens, blocks that
begin in one call and end in another, every kernel, states kept in place, copied and forked, entries'
positions and slots, values out of the ordinary, refusals on the device, graphs."""
import math
import random
import time

import pytest
import torch

from tests import operator_reference as R
from tests import serving_reference as V

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


class Stream:
    """Sequences whose tokens come call by call, the state slots that they use, and what they have had."""

    def __init__(self, gp, S, ratio, coff, d, total, seed=0, shift=0, states=None, page=4):
        g = torch.Generator().manual_seed(seed)
        self.gp, self.S, self.ratio, self.coff, self.d, self.shift, self.page = gp, S, ratio, coff, d, shift, page
        C, W = coff * d, coff * ratio
        self.kv, self.score = (torch.randn(S, total, C, generator=g).to(torch.bfloat16) for _ in range(2))
        self.ape = 0.3 * torch.randn(ratio, C, generator=g)
        self.states = S + 2 if states is None else states
        self.kv_state, self.score_state = (self.dev(torch.full((self.states, W, C), float("nan"), dtype=torch.bfloat16))
                                           for _ in range(2))
        self.first = [0] * S
        self.slot = torch.randperm(self.states, generator=g)[:S].tolist()
        self.max_pages = max(1, -(-(total // ratio) // page))
        self.table = torch.randperm(S * self.max_pages, generator=g).reshape(S, -1).to(torch.int32)

    def dev(self, t):
        flat = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        v = flat[self.shift:self.shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    def call(self, lens, source=None, target=None, spare=3, pad=2, lead=0, base=None, offset=0):
        """One call, checked in full; the sequences have len more tokens after it."""
        source, target = self.slot if source is None else source, self.slot if target is None else target
        S, ratio, coff, d, page = self.S, self.ratio, self.coff, self.d, self.page
        cu = [lead]
        for n in lens:
            cu.append(cu[-1] + n)
        rows = sum((f + n) // ratio - f // ratio for f, n in zip(self.first, lens)) + spare
        kv, score = (torch.full((cu[-1] + pad, coff * d), float("nan"), dtype=torch.bfloat16) for _ in range(2))
        for s, n in enumerate(lens):
            for to, of in ((kv, self.kv), (score, self.score)):
                to[cu[s]:cu[s] + n] = of[s, self.first[s]:self.first[s] + n]
        before = [t.clone() for t in (self.kv_state, self.score_state)]
        out = self.dev(torch.full((rows, d), 7.0, dtype=torch.bfloat16))
        positions = torch.full((rows,), 77, **I32)
        slots = torch.full((rows,), 77, dtype=torch.int64, device="cuda")
        entries, err = torch.full((S,), 77, **I32), torch.zeros(1, **I32)
        dbase = None if base is None else torch.tensor(base, **I32)
        self.gp.csa_compressor_step(
            self.dev(kv), self.dev(score), self.ape.cuda() if not self.shift else self.dev(self.ape), torch.tensor(cu, **I32), S, ratio, coff, d,
            cu[-1] + pad, torch.tensor(self.first, **I32), torch.tensor(source, **I32), torch.tensor(target, **I32),
            self.states, self.kv_state, self.score_state, out, rows, dbase, self.table.cuda(), self.max_pages, page, offset,
            positions, slots, entries, err)
        torch.cuda.synchronize()
        assert int(err) == 0
        out, positions, slots = out.double().cpu(), positions.tolist(), slots.tolist()
        row, after = 0, [t.cpu().clone() for t in before]
        for s, n in enumerate(lens):
            f, mine = self.first[s], 0 if base is None else base[s]
            for b in range(f // ratio, (f + n) // ratio):
                ref, bound = V.window_entry(self.kv[s], self.score[s], self.ape, b, ratio, coff, d)
                off = (out[row] - ref).abs()
                assert (off <= bound).all(), (s, b, float((off / bound).max()))
                assert positions[row] == b * ratio + offset
                e = b - mine
                assert slots[row] == (int(self.table[s, e // page]) * page + e % page if e >= 0 else -1)
                row += 1
            assert int(entries[s]) == max(0, (f + n) // ratio - mine)
            if target[s] >= 0:
                at = V.held(f, n, ratio, coff, d)
                cols = torch.arange(coff * d).expand_as(at)
                for want, of in zip(after, (self.kv, self.score)):
                    want[target[s]] = torch.where(at >= 0, of[s][at.clamp(min=0), cols], want[target[s]])
            self.first[s] = f + n
        assert (out[row:] == 7.0).all() and positions[row:] == [-1] * spare and slots[row:] == [-1] * spare
        for want, got in zip(after, (self.kv_state, self.score_state)):
            assert torch.equal(want.view(torch.int16), got.cpu().view(torch.int16))


SHAPES = [(4, 2, 512), (4, 2, 64), (2, 2, 128), (1, 2, 64), (1, 1, 64), (2, 1, 40), (3, 1, 64), (4, 1, 128), (8, 1, 128),
          (8, 2, 64), (5, 2, 64), (3, 2, 552), (16, 1, 64), (128, 1, 64), (128, 2, 32), (40, 2, 24), (4, 2, 65), (1, 1, 7),
          (128, 2, 9), (2, 1, 13), (7, 1, 33), (4, 1, 5)]


@pytest.mark.parametrize("ratio,coff,d,shift", [(*s, 0) for s in SHAPES] + [(*s, 1) for s in SHAPES if s[2] in (64, 512)])
def test_calls_of_any_length(cuda_lib, ratio, coff, d, shift):
    rng = random.Random(ratio * 64 + d)
    st = Stream(cuda_lib, 5, ratio, coff, d, 8 * ratio + 40, seed=d, shift=shift)
    for i in range(6):
        most = [1, ratio, 2 * ratio + 3, 1, ratio + 1, 2][i]
        st.call([rng.randint(0, most) if i else most for _ in range(5)], spare=i % 3, lead=i, offset=i % ratio)


@pytest.mark.parametrize("ratio,coff,d,S", [(4, 2, 512, 40), (1, 1, 64, 40), (2, 2, 64, 130), (16, 2, 64, 40), (3, 1, 11, 33), (1, 2, 7, 9),
                                            (4, 1, 128, 512)])
def test_a_chunk_among_single_tokens(cuda_lib, ratio, coff, d, S):
    """Batches with room for 8 tokens a sequence, most of which one or two sequences have: their blocks are shared out."""
    most = 8 * S
    st = Stream(cuda_lib, S, ratio, coff, d, most + 4 * ratio, seed=S)
    lens = [1] * S
    lens[S // 3] = most - S - 10
    st.call(lens, pad=0, spare=2)
    lens = [0] * S
    lens[1], lens[S - 1], lens[S // 3] = most // 2 - 3, most // 2 - 20, 5
    st.call(lens, pad=0, lead=4)
    st.call([1] * S)


@pytest.mark.parametrize("ratio,coff,d,S", [(48, 1, 8, 512), (20, 2, 9, 300), (33, 1, 8, 513), (4, 2, 64, 256), (4, 2, 64, 257),
                                            (3, 2, 8, 250), (8, 1, 8, 60)])
def test_a_chunk_among_as_many_sequences_as_one_kernel_takes(cuda_lib, ratio, coff, d, S):
    """Both sides of the border between the kernels, for short windows and for long ones."""
    st = Stream(cuda_lib, S, ratio, coff, d, 8 * S + 2 * ratio, seed=S + 1)
    lens = [1] * S
    lens[S - 2] = 7 * S
    st.call(lens, pad=0, spare=1)
    lens = [0] * S
    lens[0], lens[S - 1], lens[S // 2] = 6 * S, 2 * ratio - 1, ratio + 1
    st.call(lens, pad=0, lead=1)
    st.call([s % 9 for s in range(S)], pad=0)


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 512), (4, 1, 64), (16, 2, 64), (2, 2, 64), (3, 2, 11)])
def test_single_tokens(cuda_lib, ratio, coff, d):
    st = Stream(cuda_lib, 7, ratio, coff, d, 5 * ratio + 6, seed=3)
    st.call([s for s in range(7)])  # every sequence at another place of its block
    for _ in range(3 * ratio - 1):
        st.call([1] * 7, spare=1)


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 512), (4, 1, 512), (128, 1, 64), (128, 2, 128), (1, 1, 512), (2, 1, 256)])
def test_long_chunks(cuda_lib, ratio, coff, d):
    st = Stream(cuda_lib, 3, ratio, coff, d, 1700, seed=4)
    st.call([5, 0, 700], spare=0)
    st.call([901, 333, 130], pad=0)
    st.call([1, 511, 0])


@pytest.mark.parametrize("S", [1, 300, 2000])
def test_many_sequences(cuda_lib, S):
    st = Stream(cuda_lib, S, 4, 2, 16, 12, seed=5)
    st.call([s % 5 for s in range(S)], spare=5)
    st.call([(s * 7) % 4 for s in range(S)], spare=0)
    st.call([1] * S, spare=0)


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 64), (4, 1, 64), (16, 2, 32), (3, 2, 5)])
def test_states_copied_and_forked(cuda_lib, ratio, coff, d):
    """Two prompts; then five sequences go on from the first one's state in states of their own, one without a
    token; a sequence that keeps nothing."""
    S = 6
    st = Stream(cuda_lib, S, ratio, coff, d, 6 * ratio, seed=6, states=2 * S)
    for t in (st.kv, st.score):
        t[1:5, :2 * ratio + 1] = t[0, :2 * ratio + 1]
    begun = 2 * ratio + 1
    st.call([begun, 0, 0, 0, 0, ratio], target=[0, -1, -1, -1, -1, 1], source=[-1] * S)
    st.first[1:5] = [begun] * 4
    st.call([1, ratio, 0, 2, ratio + 2, 1], source=[0] * 5 + [1], target=[5, 6, 7, 8, 9, 1])
    st.call([ratio] * 5 + [2], source=[5, 6, 7, 8, 9, 1], target=[5, 6, 7, 8, 9, 11])
    st.call([ratio - 1] * 5 + [2], source=[5, 6, 7, 8, 9, 11], target=[-1] * 6)


def test_prefix_entries_lie_elsewhere(cuda_lib):
    st = Stream(cuda_lib, 3, 4, 2, 64, 60, seed=7)
    st.call([21, 8, 30], base=[3, 0, 9])
    st.call([9, 8, 30], base=[3, 0, 9])


def test_calls_are_repeatable(cuda_lib):
    """The same bits from the same inputs, whatever lay in the outputs."""
    for ratio, coff, d in ((4, 2, 512), (128, 2, 64)):
        got = []
        for _ in range(2):
            st = Stream(cuda_lib, 4, ratio, coff, d, 700, seed=8)
            st.call([300, 7, 0, 129])
            st.call([200, 400, 1, 3])
            got.append((st.kv_state.clone(), st.score_state.clone()))
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*got))


def raw(gp, ratio=2, coff=1, d=8, cu=(0, 4), first=(0,), source=(0,), target=(0,), states=1, rows=4, kv=None, score=None, table=None,
        max_pages=0, page=1, base=None, capacity=None, nulls=False):
    """A small call whatever it holds; its outputs."""
    S = len(cu) - 1
    capacity = max(cu[-1], 0) if capacity is None else capacity
    C, W = coff * d, coff * ratio
    kv = torch.ones(capacity, C, dtype=torch.bfloat16, device="cuda") if kv is None else kv
    score = torch.zeros(capacity, C, dtype=torch.bfloat16, device="cuda") if score is None else score
    st = [torch.full((states, W, C), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.full((rows, d), 7.0, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.full((rows,), 77, **I32), torch.full((rows,), 77, dtype=torch.int64, device="cuda")
    entries, err = torch.full((max(S, 1),), 77, **I32), torch.zeros(1, **I32)
    t = lambda v: torch.tensor(v, **I32)  # noqa: E731
    gp.csa_compressor_step(kv, score, torch.zeros(ratio, C, device="cuda"), t(cu), S, ratio, coff, d, capacity, t(first), t(source),
                           t(target), states, *st, out, rows, None if base is None else t(base), None if table is None else t(table),
                           max_pages, page, 0, None if nulls else pos, None if nulls or table is None else slots,
                           None if nulls else entries, err)
    torch.cuda.synchronize()
    return int(err), out.cpu(), st, pos.tolist(), slots.tolist(), entries.tolist()


@pytest.mark.parametrize("code,how", [
    (1, dict(cu=(0, 5, 3), first=(0, 0), source=(0, 0), target=(0, 0), capacity=8)), (1, dict(cu=(0, 9), capacity=8)),
    (1, dict(cu=(-1, 3), capacity=8)), (2, dict(rows=1)), (8, dict(first=(-1,))), (8, dict(first=(2 ** 31 - 2,))),
    (8, dict(source=(1,))), (8, dict(target=(7,))), (8, dict(first=(3,), source=(-1,))),
    (8, dict(coff=2, first=(2,), source=(-1,))), (8, dict(cu=(0, 0), first=(3,), source=(-1,), rows=0, capacity=1)),
])
def test_device_refusals_leave_all_as_it_was(cuda_lib, code, how):
    err, out, st, pos, slots, entries = raw(cuda_lib, **how)
    assert err == code and (out == 7.0).all() and all((t == 5.0).all() for t in st)
    assert set(pos) <= {77} and set(entries) == {77}


@pytest.mark.parametrize("S", [2, 511, 512, 600])
def test_offsets_that_overlap_again_and_again(cuda_lib, S):
    """Each second sequence has all tokens of the call: refused, however many entries that makes."""
    cu = [8 * S * (s % 2) for s in range(S + 1)]
    err, out, st, pos, slots, entries = raw(cuda_lib, 1, 1, 4, cu, [0] * S, [-1] * S, [-1] * S, rows=8 * S, capacity=8 * S)
    assert err == 1 and (out == 7.0).all() and all((t == 5.0).all() for t in st) and set(pos) <= {77} and set(entries) == {77}


def test_calls_that_need_no_state(cuda_lib):
    assert raw(cuda_lib, first=(4,), source=(-1,))[0] == 0  # coff 1 at a block's beginning
    err, out, st, *_ = raw(cuda_lib, cu=(0, 3), source=(-1,), target=(-1,), states=0)
    assert err == 0 and (out[0] == 1.0).all() and (out[1:] == 7.0).all()
    assert raw(cuda_lib, cu=(0, 0), first=(3,), source=(-1,), target=(-1,), rows=2, capacity=1)[3] == [-1, -1]  # a padded sequence
    assert raw(cuda_lib, cu=(0,), first=(), source=(), target=(), rows=2, capacity=1)[3] == [-1, -1]  # no sequence at all
    assert raw(cuda_lib, nulls=True)[0] == 0


@pytest.mark.parametrize("ratio,coff,tokens", [(2, 1, 5), (2, 2, 5), (4, 1, 90), (16, 1, 5), (16, 2, 90), (2048, 1, 90), (1024, 2, 5)])
def test_last_positions(cuda_lib, ratio, coff, tokens):
    """The last tokens that positions reach: their blocks and what the state holds of them; and one more is refused."""
    end, d = 2 ** 31 - 4097, 8
    g = torch.Generator().manual_seed(11)
    kv, score = (torch.randn(tokens, coff * d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    first = end - tokens
    made = end // ratio - first // ratio
    err, out, st, pos, _, entries = raw(cuda_lib, ratio, coff, d, (0, tokens), (first,), rows=made + 1, kv=kv, score=score)
    assert err == 0 and entries == [end // ratio]
    assert pos == [(first // ratio + i) * ratio for i in range(made)] + [-1]
    full = torch.full((ratio * coff + tokens, coff * d), 5.0, dtype=torch.bfloat16)  # the state's positions, then the new ones
    full[-tokens:] = kv.cpu()
    sc = torch.full_like(full, 5.0)
    sc[-tokens:] = score.cpu()
    for i in range(made):
        x, k = [], []
        for p in range((first // ratio + i - coff + 1) * ratio, (first // ratio + i + 1) * ratio):
            half = 0 if coff == 1 or p < (first // ratio + i) * ratio else 1
            row = p - first + ratio * coff
            k.append(full[row, half * d:half * d + d].double())
            x.append(sc[row, half * d:half * d + d].double())
        x, k = torch.stack(x), torch.stack(k)
        ref = (torch.softmax(x, 0) * k).sum(0)
        assert ((out[i].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-4).all()  # (values and scores of 5: 150 U of them)
    W = ratio * coff
    for half in range(coff):
        keep = max(0, end // ratio - (coff - 1 - half)) * ratio
        for p in range(max(keep, first), end):
            for t, of in zip(st, (kv, score)):
                assert torch.equal(t[0, p % W, half * d:half * d + d], of[p - first, half * d:half * d + d])
    err, out, st, *_ = raw(cuda_lib, ratio, coff, d, (0, tokens), (first + 1,), rows=made + 1, kv=kv, score=score)
    assert err == 8 and all((t == 5.0).all() for t in st)


@pytest.mark.parametrize("ratio,coff,d", [(4, 2, 8), (16, 1, 4), (16, 2, 3)])
def test_most_sequences(cuda_lib, ratio, coff, d):
    """As many sequences as a call may have, whose numbers leave less room for tokens under way: the same bits as a
    quarter of them at a time."""
    S = 16384
    g = torch.Generator().manual_seed(12)
    lens = torch.randint(0, 2 * ratio, (S,), generator=g)
    first = torch.randint(0, 3 * ratio, (S,), generator=g).to(torch.int32)
    W, C = coff * ratio, coff * d
    kv, score = (torch.randn(int(lens.sum()), C, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ape = torch.randn(ratio, C, generator=g).cuda()
    states = [torch.randn(S, W, C, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    made = (first + lens) // ratio - first // ratio
    slot = torch.arange(S, **I32)

    def call(a, b, st):
        rows, t0, t1 = int(made[a:b].sum()), int(cu[a]), int(cu[b])
        out, pos, err = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, **I32), torch.zeros(1, **I32)
        cuda_lib.csa_compressor_step(kv[t0:t1].clone(), score[t0:t1].clone(), ape, (cu[a:b + 1] - t0).to(torch.int32).cuda(), b - a, ratio, coff, d,
                                     t1 - t0, first[a:b].cuda(), slot[a:b].clone(), slot[a:b].clone(), S, *st, out, rows, None, None, 0, 1, 0,
                                     pos, None, None, err)
        torch.cuda.synchronize()
        assert int(err) == 0
        return out, pos
    one, two = [t.clone() for t in states], [t.clone() for t in states]
    whole = call(0, S, one)
    parts = [call(a, a + S // 4, two) for a in range(0, S, S // 4)]
    assert torch.equal(whole[0], torch.cat([x[0] for x in parts])) and torch.equal(whole[1], torch.cat([x[1] for x in parts]))
    assert all(torch.equal(x, y) for x, y in zip(one, two))


def test_pages_that_are_missing(cuda_lib):
    err, out, _, pos, slots, entries = raw(cuda_lib, cu=(0, 8), rows=5, table=((3, -1),), max_pages=2, page=1)
    assert err == 7 and slots == [3, -1, -1, -1, -1] and pos == [0, 2, 4, 6, -1] and entries == [4] and (out[:4] == 1.0).all()
    err, _, _, _, slots, entries = raw(cuda_lib, cu=(0, 8), rows=4, table=((3, 9),), max_pages=2, page=1, base=(2,))
    assert err == 0 and slots == [-1, -1, 3, 9] and entries == [2]


@pytest.mark.parametrize("ratio,coff,d", [(4, 1, 8), (4, 1, 7), (32, 1, 8), (2, 1, 8)])
def test_values_out_of_the_ordinary(cuda_lib, ratio, coff, d):
    """A score of -inf weighs nothing, a window of nothing else is NaN, as are those with a score of +inf or
    NaN; a lowest score beside others weighs nothing."""
    g = torch.Generator().manual_seed(9)
    kv = torch.randn(5 * ratio, d, generator=g).to(torch.bfloat16)
    score = torch.randn(5 * ratio, d, generator=g).to(torch.bfloat16)
    score[1, :] = -math.inf
    score[ratio:2 * ratio, :] = -math.inf
    score[2 * ratio, :] = math.inf
    score[3 * ratio + 1, :] = math.nan
    score[4 * ratio:5 * ratio - 1, :] = -3.3895e38
    err, out, *_ = raw(cuda_lib, ratio, coff, d, (0, 5 * ratio), rows=5, kv=kv.cuda(), score=score.cuda())
    assert err == 0 and torch.isnan(out[1:4]).all()
    for b in (0, 4):
        x = score[b * ratio:(b + 1) * ratio].double()
        ref = (torch.softmax(x, 0) * kv[b * ratio:(b + 1) * ratio].double()).sum(0)
        assert ((out[b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5).all()  # (fp32: about 50 U of values of 4 at most)


@pytest.mark.parametrize("ratio,coff,d", [(4, 1, 8), (4, 1, 7), (32, 1, 8), (2, 2, 8), (16, 2, 4), (4, 2, 64)])
@pytest.mark.parametrize("S", [1, 40])
def test_scores_at_their_types_limits(cuda_lib, ratio, coff, d, S):
    """Windows whose scores are all the lowest value weigh their positions alike, the largest value takes the weight
    from all others, and beside the lowest one -inf still weighs nothing: by many tokens and by few a sequence."""
    g = torch.Generator().manual_seed(13)
    most = float(torch.finfo(torch.bfloat16).max)
    n = 5 * ratio
    kv, score = (torch.randn(S * n, coff * d, generator=g).to(torch.bfloat16).view(S, n, coff * d) for _ in range(2))
    score[:, :2 * ratio] = -most
    score[:, ratio] = -math.inf
    score[:, 3 * ratio - 1] = most
    score[:, 4 * ratio:] = most
    if S == 1:
        calls = [list(range(n))]
    else:  # two tokens a call
        calls = [list(range(a, min(a + 2, n))) for a in range(0, n, 2)]
    W, C = coff * ratio, coff * d
    states = [torch.zeros(S, W, C, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    own = torch.arange(S, **I32)
    got = [[] for _ in range(S)]
    for at in calls:
        rows = (at[-1] + 1) // ratio - at[0] // ratio
        out, err = torch.zeros(S * rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, **I32)
        cu = torch.arange(S + 1, **I32) * len(at)
        cuda_lib.csa_compressor_step(kv[:, at].contiguous().cuda(), score[:, at].contiguous().cuda(), torch.zeros(ratio, C, device="cuda"), cu, S,
                                     ratio, coff, d, S * len(at), torch.full((S,), at[0], **I32), own, own, S, *states, out, S * rows, dev_error=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        for s in range(S):
            got[s] += list(out.view(S, rows, d)[s].double().cpu())
    for s in range(S):
        assert len(got[s]) == 5
        for b in range(5):
            half = [(p, 0 if coff == 1 or p < b * ratio else d) for p in range(max(0, b - coff + 1) * ratio, (b + 1) * ratio)]
            x, k = (torch.stack([t[s, p, c:c + d].double() for p, c in half]) for t in (score, kv))
            w = torch.softmax(x, 0)
            ref = (w * k).sum(0)
            # (as window_entry's, but that the embedding is 0: a difference from the maximum is rounded, not its terms)
            away = torch.where(w > 0, x.amax(0) - x, 0.0)
            mass = R.U * ((2 * (10 + min(32, len(x))) + 16) * (w * k.abs()).sum(0) + 8 * (w * (k - ref).abs() * (away + 1)).sum(0))
            assert ((got[s][b] - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * mass).all(), (s, b)


@pytest.mark.parametrize("S", [4, 700])
@pytest.mark.parametrize("ratio,coff", [(2, 1), (2, 2)])
def test_states_that_sequences_meet_in(cuda_lib, S, ratio, coff):
    """A state that one sequence writes and another one writes or reads is reported, and all other sequences are as ever;
    what is only read, or named by a sequence that neither reads nor writes, may be named by any."""
    W = coff * ratio

    def call(change, first=W + 1, n=1):
        source, target, firsts, lens = [2 * s for s in range(S)], [2 * s + 1 for s in range(S)], [first] * S, [n] * S
        for s, how in change.items():
            source[s], target[s], firsts[s], lens[s] = (x if y is None else y for x, y in zip((source[s], target[s], firsts[s], lens[s]), how))
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        err, out, st, pos, *_ = raw(cuda_lib, ratio, coff, 8, cu, firsts, source, target, 2 * S, rows=S * (1 + n), capacity=cu[-1] + 1)
        return err, out, pos
    a, b = 1, S - 1
    fine, out, pos = call({})
    assert fine == 0
    for change in ({a: (2 * a, 2 * a, None, None), b: (2 * a, None, None, None)},         # goes on in place, and another forks from it
                   {a: (2 * a, 2 * b + 1, None, None)},                                   # two targets
                   {a: (2 * b + 1, None, None, None)},                                    # one's target is another's source
                   {a: (2 * b + 1, -1, None, None)},                                      # read alone
                   {a: (2 * b + 1, None, None, 0)},                                       # copied, without a token
                   {a: (2 * a, 5, None, None), b: (2 * b, 5, 0, 1), 2: (None, -1, None, None)}):  # one that begins, in another's
        err, got, at = call(change)
        assert err == 8, change
        if S > 4 and len(change) < 3 and all(x[3] is None for x in change.values()):
            rest = torch.tensor([s not in change and s != b for s in range(S)])
            assert torch.equal(got[:S][rest], out[:S][rest]) and at[:S] == pos[:S]
    for change in ({a: (0, None, None, None), b: (0, None, None, None), 2: (0, -1, None, None)},  # forks
                   {a: (7, 7, None, 0), b: (7, 7, None, 0), 2: (1, 1, None, 0)},                  # idle, whatever they name
                   {a: (2 * b + 1, None, 0, None)},                                               # nothing is read at a beginning
                   {a: (2 * b + 1, -1, None, 0)},                                                 # nor without a token or a target
                   {a: (-1, -1, 0, None), b: (-1, -1, 0, None)}):
        assert call(change)[0] == 0, change


@pytest.mark.parametrize("S", [2, 5, 16384])
def test_far_apart_states_are_not_taken_for_one(cuda_lib, S):
    """As many states as share a place in the lists that are looked at for states that meet; and a pair that does meet
    among them."""
    step = 2048 * S if S < 100 else 1024
    states, d = (S + 1) * step, 1
    kv, score = (torch.ones(S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = [torch.zeros(states, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err, out = torch.zeros(1, **I32), torch.zeros(S, d, dtype=torch.bfloat16, device="cuda")
    own = torch.arange(S, **I32) * step

    def call(target):
        cuda_lib.csa_compressor_step(kv, score, torch.zeros(1, d, device="cuda"), torch.arange(S + 1, **I32), S, 1, 1, d, S,
                                     torch.arange(S, **I32), own, target, states, *st, out, S, dev_error=err)
        torch.cuda.synchronize()
        return int(err)
    assert call(own) == 0 and (out == 1).all()
    other = own.clone()
    other[S - 1] = own[S // 3]
    assert call(other) == 8


def test_sizes_met_late_are_called_as_fast(cuda_lib):
    """What the library keeps of each size that it has met is found at once, however many there are: on the host, a call of
    a size met after ten thousand others takes about as long as the first one (half as long again, and a microsecond, for
    what else goes on; a list searched from its beginning takes four times as long)."""
    d, first, last = 2, 600, 11000
    kv, out = (torch.zeros(n, d, dtype=torch.bfloat16, device="cuda") for n in (9 * last, 1))
    ape, zero, none = torch.zeros(1, d, device="cuda"), torch.zeros(last + 1, **I32), torch.full((last,), -1, **I32)

    def call(S):  # (sequences without a token)
        cuda_lib.csa_compressor_step(kv, kv, ape, zero, S, 1, 1, d, 9 * S, zero, none, none, 0, None, None, out, 1)

    def host(S):
        best = math.inf
        for _ in range(30):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            for _ in range(20):
                call(S)
            best = min(best, time.perf_counter() - t0)
        return best / 20
    for S in range(first, last + 1):
        call(S)
        if S % 500 == 0:
            torch.cuda.synchronize()
    a, b = host(first), host(last)
    assert b < 1.5 * a + 1e-6, (a, b)


def test_graph_of_steps(cuda_lib):
    """A captured step that moves its own lengths on, replayed, against the calls one by one."""
    ratio, coff, d, S = 4, 2, 64, 3
    g = torch.Generator().manual_seed(10)
    steps = [torch.randn(S, coff * d, generator=g).to(torch.bfloat16).cuda() for _ in range(19)]
    ape = torch.randn(ratio, coff * d, generator=g).cuda()

    def make():
        c = dict(kv=torch.zeros(S, coff * d, dtype=torch.bfloat16, device="cuda"), first=torch.tensor([0, 1, 2], **I32),
                 own=torch.arange(S, **I32), cu=torch.arange(S + 1, **I32), err=torch.zeros(1, **I32),
                 out=torch.zeros(S, d, dtype=torch.bfloat16, device="cuda"), pos=torch.zeros(S, **I32))
        c["state"] = [torch.zeros(S, coff * ratio, coff * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        return c

    def step(c):
        cuda_lib.csa_compressor_step(c["kv"], c["kv"], ape, c["cu"], S, ratio, coff, d, S, c["first"], c["own"], c["own"], S,
                                     *c["state"], c["out"], S, None, None, 0, 1, 0, c["pos"], None, None, c["err"])
        c["first"] += 1

    one, two = make(), make()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(make())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(two)
    torch.cuda.synchronize()
    for x in steps:
        for c in (one, two):
            c["kv"].copy_(x)
        step(one)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("out", "pos", "first", "err"):
            assert torch.equal(one[k], two[k])
        assert int(one["err"]) == 0
    assert torch.equal(one["state"][0], two["state"][0])
