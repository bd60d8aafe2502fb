"""Cache attention where scores or entries leave the ordinary range, the tensor-core kernel in each of its
ways and the scalar one alike."""
import math

import pytest
import torch

from tests import operator_reference as R
from tests.test_gpu_attn import Case

pytestmark = pytest.mark.gpu

# H, kv, d, page, tokens: boxes, threads, boxes of one tile a block, packed (rows enough), threads at 512, scalar
WAYS = [(8, 1, 128, 16, 20), (8, 1, 128, 9, 20), (4, 1, 512, 16, 20), (64, 1, 512, 16, 20), (4, 1, 512, 9, 20),
        (16, 2, 256, 16, 20), (3, 1, 65, 16, 20), (2, 1, 1000, 16, 7)]


def slot_of(c, e):
    return int(c.table[0, e // c.page]) * c.page + e % c.page


def without(c, e, rows):
    """The reference over c's one sequence, with entry e left out for the tokens in `rows`: out, lse, bounds."""
    whole = c.reference()
    for t in rows:
        n = R.seen(c.first[0] + t, c.ratio, c.entries[0])
        rest = torch.tensor([[slot_of(c, k) for k in range(n) if k != e]], dtype=torch.int32)
        for to, part in zip(whole, R.attend(c.q[t:t + 1], [0, 1], c.values, rest, 1, [n - 1], None, 0, c.scale, c.sink)):
            to[t] = part[0]
    return whole


def singles(c):
    """The same tokens as sequences of one token each over the same entries."""
    n = c.cu[1]
    one = Case([1] * n, [1] * n, c.H, c.kv, c.d, page=c.page, ratio=c.ratio, first=[c.first[0] + i for i in range(n)])
    one.entries = c.entries * n
    one.max_pages, one.num_pages, one.table = c.max_pages, c.num_pages, c.table.repeat(n, 1)
    one.q, one.data, one.values, one.sink, one.scale = c.q, c.data, c.values, c.sink, c.scale
    return one


def agree(c, rows, want):
    """The tokens in `rows` of both calls are the reference's; returns what the others got."""
    ref, rl, tol, ltol = want
    rest = []
    for call in (c, singles(c)):
        out, lse, err = call.run(c.gp)
        out, lse = out.double().cpu()[:c.cu[1]], lse.double().cpu()[:c.cu[1]]
        dead = torch.isinf(rl[rows])
        assert err == 0 and ((out - ref[:c.cu[1]]).abs()[rows] <= tol[rows]).all()
        assert torch.equal(lse[rows][dead], rl[rows][dead])
        assert ((lse[rows] - rl[rows]).abs()[~dead] <= ltol[rows][~dead]).all()
        others = [i for i in range(c.cu[1]) if i not in rows]
        rest.append((out[others], lse[others]))
    return rest


# entries, the special one, and whether some tokens do not see it
PLACES = [(40, 33, True), (300, 33, False), (300, 290, True), (300, 33, True)]


def case(gp, way, place, sink):
    (H, kv, d, page, n), (entries, e, masked) = way, place
    ratio = 2 if masked else 0
    # (masked) token i sees the entry from the middle token on
    c = Case([n], [entries], H, kv, d, page=page, ratio=ratio, first=[2 * (e + 1) - 1 - n // 2], sink=sink, seed=e + d)
    c.gp = gp
    blind = [i for i in range(n) if R.seen(c.first[0] + i, ratio, entries) <= e]
    assert bool(blind) == masked and len(blind) < n
    return c, blind, [i for i in range(n) if i not in blind]


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("sink", [False, True])
def test_a_non_finite_entry_is_the_same_to_every_token_that_sees_it(cuda_lib, way, bad, place, sink):
    """NaN throughout, on whichever side of it the score falls, whether other rows of the tile see the entry or
    not, and whether the token comes in a chunk or by itself. The others see nothing of it."""
    c, blind, sees = case(cuda_lib, way, place, sink)
    slot = slot_of(c, place[1])
    c.data[slot, 0, c.d // 2] = bad
    want = c.reference()
    for out, lse in agree(c, blind, want):
        part = c.H // c.kv
        assert torch.isnan(out[:, :part]).all() and torch.isnan(lse[:, :part]).all()
        # the other cache head's entries are as they were
        assert ((out - want[0][sees]).abs()[:, part:] <= want[2][sees][:, part:]).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("place", PLACES)
def test_a_finite_entry_scored_past_fp32(cuda_lib, way, place):
    """A score below fp32's range weighs nothing: these rows are as if the entry were not there."""
    c, blind, sees = case(cuda_lib, way, place, True)
    c.q[:, :, 3] = -1e3
    c.data[:, :, 3] = 0
    c.values[:, :, 3] = 0
    slot = slot_of(c, place[1])
    c.data[slot, :, 3] = 3e38
    want = without(c, place[1], sees)
    agree(c, list(range(c.cu[1])), want)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("sink", [False, True])
def test_rows_that_score_everything_below_fp32(cuda_lib, way, sink):
    """They are rows that see nothing: out 0, lse the sink or -inf."""
    H, kv, d, page, n = way
    c = Case([n], [150], H, kv, d, page=page, ratio=0, sink=sink, seed=d)
    c.q[:, :, 3] = 1e3
    c.data[:, :, 3] = -3e38
    out, lse, err = c.run(cuda_lib)
    assert err == 0 and (out[:n] == 0).all()
    want = torch.full((n, H), -math.inf) if c.sink is None else c.sink.expand(n, H)
    assert torch.equal(lse[:n].cpu(), want)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("size", [1e7, 1e9, 1e11, 1e16, 1e28, 1e30, 1e33, 1e37])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("sink", [False, True])
def test_scores_far_from_zero(cuda_lib, way, size, sign, sink):
    """Every score finite and far from zero, a single exact product: the highest one has all the weight (out is
    its entry, the weight and the output rounded to 16 bits, 2^-8 each), and lse is its score or (far below
    zero) the sink. Its scale and the scale's way through log2 and back (two constants and two products)
    round it five times by half a step (U), the score's own product once by a whole one."""
    H, kv, d, page, n = way
    c = Case([n], [300], H, kv, d, page=page, ratio=0, sink=sink, seed=d + 1)
    c.q.zero_()
    c.q[:, :, 3] = math.sqrt(size)
    top = 170
    for e in range(300):
        c.data[slot_of(c, e), :, 3] = sign * math.sqrt(size) * (1 if e == top else 1 - sign * 0.5)
    out, lse, err = c.run(cuda_lib)
    score = c.q[0, 0, 3].double() * c.data[slot_of(c, top), 0, 3].double() * c.scale
    out, lse = out[:n].double().cpu(), lse[:n].double().cpu()
    assert err == 0
    if sink and sign < 0:
        assert (out == 0).all() and ((lse - c.sink).abs() <= 7 * R.U * c.sink.abs()).all()
    else:
        want = c.data[slot_of(c, top)].double().repeat_interleave(H // kv, 0).expand(n, H, d)
        assert ((out - want).abs() <= 2.01 * 2.0 ** -8 * want.abs()).all()
        assert ((lse - score).abs() <= 7 * R.U * score.abs()).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.3, 1e-45, 1e-30])
@pytest.mark.parametrize("place", PLACES)
def test_scales_of_zero_and_below(cuda_lib, way, scale, place):
    """A scale of 0 weighs every entry alike however large the products, a negative one turns their order, and
    neither lets a masked entry through."""
    c, _, _ = case(cuda_lib, way, place, True)
    c.scale = scale
    if scale >= 0:
        c.q[:, :, 3] = 1e19
        sign = torch.sign(c.data[:, :, 3].float())
        c.data[:, :, 3] = (sign * 1e18).to(torch.bfloat16)
        c.values = c.data.double()
    agree(c, list(range(c.cu[1])), c.reference())


@pytest.mark.parametrize("way,lens,entries,first", [(w, [w[4], 3], [300, 40], [0, 60]) for w in WAYS] + [
    ((16, 1, 128, 64, 1), [1], [3001], [6001]), ((16, 1, 512, 64, 2), [2], [20500], [40999]),
    ((64, 1, 128, 9, 1), [1, 1], [1500, 3001], [2999, 6001])])
def test_sinks_that_are_not_finite(cuda_lib, way, lens, entries, first):
    """A sink of -inf is none, one of +inf takes all the weight (out 0, lse +inf), one of NaN makes NaN; a token
    that sees nothing gets out 0 and lse the sink, whatever it is. In units by themselves and joined ones."""
    H, kv, d, page, _ = way
    c = Case(lens, entries, H, kv, d, page=page, ratio=2, first=first, seed=d)
    free = c.reference()
    c.sink = torch.tensor([math.inf, math.nan, -math.inf, 1.5])[torch.arange(H) % 4]
    held = Case(lens, entries, H, kv, d, page=page, ratio=2, first=first, seed=d)
    held.sink = torch.where(torch.isfinite(c.sink), c.sink, torch.zeros(()))
    held = held.reference()
    out, lse, err = c.run(cuda_lib)
    out, lse, T = out.double().cpu(), lse.double().cpu(), c.cu[-1]
    assert err == 0
    blind = torch.isinf(free[1][:T]).any(1)  # (without a sink)
    assert blind[0] == (first[0] == 0) and not blind.all()
    assert (out[:T][blind] == 0).all()
    assert torch.equal(lse[:T][blind].nan_to_num(7.0, 8.0, 9.0), c.sink.double().nan_to_num(7.0, 8.0, 9.0).expand(int(blind.sum()), H))
    sees = ~blind
    for h in range(H):
        got, gl = out[:T, h][sees], lse[:T, h][sees]
        if c.sink[h] == math.inf:
            assert (got == 0).all() and (gl == math.inf).all()
        elif torch.isnan(c.sink[h]):
            assert torch.isnan(got).all() and torch.isnan(gl).all()
        else:
            ref, rl, tol, ltol = (t[:T, h][sees] for t in (free if c.sink[h] == -math.inf else held))
            assert ((got - ref).abs() <= tol).all() and ((gl - rl).abs() <= ltol).all()


@pytest.mark.parametrize("way", WAYS)
def test_a_row_whose_scores_are_all_nan(cuda_lib, way):
    """out and lse NaN, with a sink and without."""
    H, kv, d, page, n = way
    for sink in (False, True):
        c = Case([n], [20], H, kv, d, page=page, ratio=0, sink=sink, seed=d)
        c.q[1, 1, 0] = math.nan
        out, lse, err = c.run(cuda_lib)
        assert err == 0 and torch.isnan(out[1, 1]).all() and torch.isnan(lse[1, 1])
        assert int(torch.isnan(lse).sum()) == 1 and int(torch.isnan(out).any(-1).sum()) == 1
