"""Head norm and rotation through the C ABI against the 64-bit reference: both directions, types,
layouts, part of the head, strided and in-place tensors, rows left out, far positions, the
vector and the scalar kernel, streams, graphs and repeated calls."""
import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu


def make(rows, heads, d, dtype, seed, slab=0, shift=0, spread=True):
    """[rows, heads, d] on the GPU, optionally a slice of a wider slab or off its 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, heads + slab, d, generator=g)
    if spread:
        x = x * torch.exp(torch.randn(rows, heads + slab, 1, generator=g))
    flat = torch.empty(x.numel() + 16, dtype=dtype, device="cuda")
    v = flat[shift:shift + x.numel()].view(rows, heads + slab, d)
    v.copy_(x.to(dtype))
    return v[:, slab:]


def setup(gp, rows, heads, d, rot, first=0, step=1, skip=(), seed=0, weight=True, scaling=0):
    g = torch.Generator().manual_seed(seed + 1000)
    w = (1 + 0.3 * torch.randn(d, generator=g)) if weight else None
    pos = (first + step * torch.arange(rows, dtype=torch.int64)).to(torch.int32)
    for r in skip:
        pos[r] = -1 - r
    turns, amp = gp.csa_rope_table(rot, scaling=scaling, factor=8.0 if scaling else 1.0)
    return w, pos, turns, amp


def cuda(t):
    return None if t is None else t.cuda()


def run_fwd(gp, x, dtype, w, norm, eps, pos, turns, rot, start, layout, amp, y, stream=None):
    rows, heads, d = x.shape
    gp.csa_norm_rope_fwd(x, R.DTYPES.index(dtype), rows, heads, d, x.stride(0), x.stride(1), cuda(w), norm, eps,
                         cuda(pos), cuda(turns) if rot else None, rot, start, layout, amp, y, y.stride(0),
                         y.stride(1), stream=stream)
    torch.cuda.synchronize()


def run_bwd(gp, x, dy, dtype, w, norm, eps, pos, turns, rot, start, layout, amp, dx, dw=None, acc=0, ws=None):
    rows, heads, d = dy.shape
    if dw is not None and ws is None:
        ws = torch.full((gp.csa_norm_rope_bwd_workspace_bytes(rows, heads, d) // 4,), float("nan"), device="cuda")
    gp.csa_norm_rope_bwd(x, dy, R.DTYPES.index(dtype), rows, heads, d, *(x.stride()[:2] if x is not None else (0, 0)),
                         *dy.stride()[:2], cuda(w), norm, eps, cuda(pos), cuda(turns) if rot else None, rot, start,
                         layout, amp, dx, *dx.stride()[:2], dw, acc, ws, 0 if ws is None else ws.numel() * 4)
    torch.cuda.synchronize()


# rows, heads, d, dtype, rot, start, layout, norm, weight, first, step
CASES = [
    (5, 1, 512, 0, 64, 448, 1, 1, True, 0, 4),       # an entry: the last 64 columns
    (33, 2, 512, 0, 64, 0, 0, 1, True, 100, 1),      # the first ones, halves
    (7, 64, 128, 0, 128, 0, 0, 1, True, 5, 1),       # queries
    (9, 3, 128, 1, 128, 0, 1, 1, True, 0, 1),
    (9, 5, 128, 2, 64, 32, 0, 1, False, 0, 7),
    (4, 1, 64, 2, 32, 32, 1, 0, False, 3, 1),        # the rotation alone
    (4, 7, 256, 0, 256, 0, 0, 0, False, 2000000, 1),
    (3, 2, 128, 0, 0, 0, 0, 1, True, 0, 1),          # the norm alone
    (1, 1, 1, 2, 0, 0, 0, 1, True, 0, 1),
    (1, 1, 2, 2, 2, 0, 1, 1, True, 1, 1),
    (6, 2, 65, 0, 30, 35, 0, 1, True, 9, 1),         # odd sizes: the scalar kernel
    (6, 2, 72, 1, 72, 0, 1, 1, True, 9, 1),          # nine pieces of eight
    (6, 3, 80, 0, 48, 16, 0, 1, True, 9, 1),
    (5, 2, 96, 0, 32, 8, 0, 1, True, 9, 1),          # the rotated part in the middle
    (5, 2, 104, 2, 8, 48, 1, 1, True, 9, 1),
    (3, 1, 1024, 0, 1024, 0, 0, 1, True, 77, 3),
    (3, 2, 1000, 2, 512, 8, 1, 1, True, 77, 3),
    (2, 1, 768, 0, 16, 752, 0, 1, True, 77, 3),
    (300, 9, 128, 0, 128, 0, 0, 1, True, 0, 1),      # many blocks
    (2, 2, 128, 0, 128, 0, 0, 1, True, 2**31 - 3, 1),  # the farthest positions
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("how", ["plain", "slab", "inplace", "shifted"])
def test_forward(cuda_lib, case, how):
    rows, heads, d, t, rot, start, layout, norm, weight, first, step = case
    dtype, gp = R.DTYPES[t], cuda_lib
    x = make(rows, heads, d, dtype, 1, slab=2 if how == "slab" else 0, shift=1 if how == "shifted" else 0)
    w, pos, turns, amp = setup(gp, rows, heads, d, rot, first, step, skip=[1] if rows > 2 else [], weight=weight,
                               scaling=2 if rot >= 64 else 0)
    keep = x.clone()
    y = x if how == "inplace" else torch.full((rows, heads, d), 7.0, dtype=dtype, device="cuda")
    run_fwd(gp, x, dtype, w, norm, 1e-6, pos, turns, rot, start, layout, amp, y)
    ref, mass = R.norm_rope(keep.cpu(), w, norm, 1e-6, R.angles(pos.clamp(min=0), turns), rot, start, layout, amp)
    live = pos >= 0
    R.close(y[live.cuda()], ref[live], mass[live], d, dtype, case)
    left = keep if how == "inplace" else torch.full_like(keep, 7.0)
    assert torch.equal(y[~live.cuda()], left[~live.cuda()])  # rows left out stay as they were


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("how", ["plain", "slab", "inplace", "into x", "shifted"])
def test_backward(cuda_lib, case, how):
    rows, heads, d, t, rot, start, layout, norm, weight, first, step = case
    dtype, gp = R.DTYPES[t], cuda_lib
    slab, shift = (2 if how == "slab" else 0), (1 if how == "shifted" else 0)
    x, dy = make(rows, heads, d, dtype, 1, slab, shift), make(rows, heads, d, dtype, 2, slab, shift, False)
    w, pos, turns, amp = setup(gp, rows, heads, d, rot, first, step, skip=[1] if rows > 2 else [], weight=weight,
                               scaling=2 if rot >= 64 else 0)
    kx, kg = x.clone(), dy.clone()
    dx = {"inplace": dy, "into x": x}.get(how, torch.full((rows, heads, d), 7.0, dtype=dtype, device="cuda"))
    before = dx.clone()
    dw = torch.full((d,), 3.0, device="cuda") if norm else None
    run_bwd(gp, x if norm or how == "into x" else None, dy, dtype, w, norm, 1e-6, pos, turns, rot, start, layout, amp,
            dx, dw, acc=1)
    live = pos >= 0
    ref, mass, rw, mw = R.norm_rope_bwd(kx.cpu()[live], kg.cpu()[live], w, norm, 1e-6,
                                        R.angles(pos[live], turns), rot, start, layout, amp)
    R.close(dx[live.cuda()], ref, mass, d, dtype, case)
    assert torch.equal(dx[~live.cuda()], before[~live.cuda()])
    if norm:  # each term as exact as the bound says, at most 64 plain additions in a row, the rest compensated
        off = (dw.double().cpu() - 3.0 - rw).abs()
        bound = (R.rope_bound(d, dtype) + 70 * R.U) * (mw + 3.0)
        assert (off <= bound).all(), float((off / bound).max())


def test_gradients_follow_differences(cuda_lib):
    """The gradients against central differences of the forward itself, in fp32."""
    gp, dtype = cuda_lib, torch.float32
    rows, heads, d, rot = 3, 2, 64, 32
    x, dy = make(rows, heads, d, dtype, 5, spread=False), make(rows, heads, d, dtype, 6, spread=False)
    w, pos, turns, amp = setup(gp, rows, heads, d, rot, 11, 3, scaling=2)
    args = (1, 1e-3, pos, turns, rot, 16, 0, amp)
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    run_bwd(gp, x, dy, dtype, w, *args, dx, dw)

    def loss(x, w):
        y = torch.empty_like(x)
        run_fwd(gp, x, dtype, w, *args, y)
        return float((y.double() * dy.double()).sum())

    # steps of 2^-6: truncation below h^2 = 2.5e-4 times third derivatives of the order of one,
    # rounding 384 outputs of a few U each over 2 h: 384 * 4 * 2^-24 / 2^-5 = 3e-3
    h = 2.0 ** -6
    for base, grad, pair in ((x, dx, lambda v: (v, w)), (w.cuda(), dw, lambda v: (x, v))):
        for i in range(0, base.numel(), 37):
            up, down = base.clone(), base.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            slope = (loss(*pair(up)) - loss(*pair(down))) / (2 * h)
            assert abs(slope - float(grad.view(-1)[i])) < 1e-2


def test_weight_gradient_store_and_repeat(cuda_lib):
    """accumulate 0 overwrites, results repeat bit for bit, and no row at all gives zeros."""
    gp, dtype = cuda_lib, torch.bfloat16
    x, dy = make(700, 4, 128, dtype, 1), make(700, 4, 128, dtype, 2)
    w, pos, turns, amp = setup(gp, 700, 4, 128, 128)
    got = []
    for fill in (float("nan"), 1.0):
        dx, dw = torch.empty_like(x), torch.full((128,), fill, device="cuda")
        run_bwd(gp, x, dy, dtype, w, 1, 1e-6, pos, turns, 128, 0, 0, amp, dx, dw)
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    dw = torch.full((128,), 5.0, device="cuda")
    run_bwd(gp, x[:0], dy[:0], dtype, w, 1, 1e-6, pos[:0], turns, 128, 0, 0, amp, x[:0], dw)
    assert (dw == 0).all()
    dw.fill_(5.0)
    run_bwd(gp, x, dy, dtype, w, 1, 1e-6, torch.full_like(pos, -1), turns, 128, 0, 0, amp, torch.empty_like(x), dw)
    assert (dw == 0).all()
    dx = torch.empty_like(x)  # a frozen weight: no gradient of it, no workspace
    run_bwd(gp, x, dy, dtype, w, 1, 1e-6, pos, turns, 128, 0, 0, amp, dx)
    assert torch.equal(dx, got[0][0])


def test_rows_are_apart(cuda_lib):
    """A NaN or infinity in one row's head stays there."""
    gp, dtype = cuda_lib, torch.bfloat16
    for d, rot in ((128, 128), (65, 30)):
        x = make(6, 4, d, dtype, 1)
        w, pos, turns, amp = setup(gp, 6, 4, d, rot)
        clean, y = torch.empty_like(x), torch.empty_like(x)
        run_fwd(gp, x, dtype, w, 1, 1e-6, pos, turns, rot, 0, 0, amp, clean)
        x[2, 1, 3], x[4, 0, 0] = float("nan"), float("inf")
        run_fwd(gp, x, dtype, w, 1, 1e-6, pos, turns, rot, 0, 0, amp, y)
        same = (y == clean).all(-1)
        assert not same[2, 1] and not same[4, 0] and int((~same).sum()) == 2


def test_zero_rows_and_graph(cuda_lib):
    """A zero head gives zeros (eps > 0); a captured call replays on new contents, on its stream."""
    gp, dtype = cuda_lib, torch.bfloat16
    x = torch.zeros(4, 2, 128, dtype=dtype, device="cuda")
    w, pos, turns, amp = setup(gp, 4, 2, 128, 128)
    w, pos, turns = w.cuda(), pos.cuda(), turns.cuda()
    y, dx, dw = torch.ones_like(x), torch.ones_like(x), torch.ones(128, device="cuda")
    dy = make(4, 2, 128, dtype, 2)
    ws = torch.empty(gp.csa_norm_rope_bwd_workspace_bytes(4, 2, 128), dtype=torch.uint8, device="cuda")

    def calls():
        gp.csa_norm_rope_fwd(x, 0, 4, 2, 128, 256, 128, w, 1, 1e-6, pos, turns, 128, 0, 0, amp, y, 256, 128)
        gp.csa_norm_rope_bwd(x, dy, 0, 4, 2, 128, 256, 128, 256, 128, w, 1, 1e-6, pos, turns, 128, 0, 0, amp, dx, 256,
                             128, dw, 0, ws, ws.numel())

    calls()
    torch.cuda.synchronize()
    assert (y == 0).all() and (dw == 0).all() and torch.isfinite(dx).all()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    x.copy_(make(4, 2, 128, dtype, 7))
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone(), dx.clone(), dw.clone()
    for t in (y, dx, dw):
        t.fill_(9.0)
    calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw)))
