"""Calls that the documentation of the entry operators allows beside the usual ones: optional arguments left
out, no pages at all, inputs that repeat, the narrowest heads."""
import pytest
import torch

from tests import operator_reference as R
from tests.test_gpu_attn import Case

pytestmark = pytest.mark.gpu

WAYS = [(8, 1, 128, 16, R.BF16, 20), (8, 1, 128, 9, R.BF16, 20), (64, 1, 512, 16, R.E4M3, 3), (64, 1, 256, 9, R.FP4, 20),
        (3, 1, 65, 16, R.BF16, 20)]


@pytest.mark.parametrize("H,kv,d,page,fmt,n", WAYS)
def test_attention_without_optional_arguments(cuda_lib, H, kv, d, page, fmt, n):
    """No lse, no error word, no first position (the tokens stand at 0, 1, ...): the same bits as with them."""
    c = Case([n, 2], [300, 7], H, kv, d, fmt, page=page, ratio=1, first=[0, 0], seed=d)
    out, lse, err, args = c.run(cuda_lib, keep=True)
    assert err == 0
    want, args = out.clone(), list(args)
    args[17] = args[24] = args[27] = None
    out.fill_(7.0)
    cuda_lib.csa_cache_attn(*args)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.check(cuda_lib)


@pytest.mark.parametrize("H,kv,d,page,fmt,n", WAYS)
@pytest.mark.parametrize("sink", [False, True])
def test_attention_over_an_empty_pool(cuda_lib, H, kv, d, page, fmt, n, sink):
    """No page, no table, no data."""
    c = Case([n], [0], H, kv, d, fmt, page=page, ratio=0, sink=sink, seed=d)
    out, lse, err, args = c.run(cuda_lib, keep=True)
    args = list(args)
    args[9] = args[10] = args[12] = None
    args[13] = args[14] = 0
    for t in (out, lse):
        t.fill_(7.0)
    cuda_lib.csa_cache_attn(*args)
    torch.cuda.synchronize()
    assert int(args[27]) == 0 and (out[:n] == 0).all() and (out[n:] == 7.0).all()
    want = torch.full((n, H), -float("inf")) if c.sink is None else c.sink.expand(n, H)
    assert torch.equal(lse[:n].cpu(), want)


@pytest.mark.parametrize("H,kv,d,page,fmt,n", WAYS)
def test_attention_of_a_repeated_query(cuda_lib, H, kv, d, page, fmt, n):
    """One query row for all tokens and heads (strides of 0)."""
    c = Case([n], [300], H, kv, d, fmt, page=page, ratio=2, first=[400], seed=d)
    c.q[:] = c.q[0, 0].clone()
    out, lse, err, args = c.run(cuda_lib, keep=True)
    want, wl, args = out.clone(), lse.clone(), list(args)
    args[0], args[1], args[2] = c.q[0, 0].clone().cuda(), 0, 0
    for t in (out, lse):
        t.fill_(7.0)
    cuda_lib.csa_cache_attn(*args)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("d", [8, 16, 24, 1, 2])
@pytest.mark.parametrize("page", [16, 9])
def test_attention_of_narrow_heads(cuda_lib, d, page):
    Case([20, 1], [300, 129], 16, 2, d, page=page, ratio=1, first="end", sink=True, seed=d).check(cuda_lib)


@pytest.mark.parametrize("d", [128, 65])
def test_norm_without_positions(cuda_lib, d):
    """The norm alone needs no position and no table; forward and backward."""
    gp, g = cuda_lib, torch.Generator().manual_seed(d)
    x, dy = (torch.randn(9, 3, d, generator=g).cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn(d, generator=g)).cuda()
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(gp.csa_norm_rope_bwd_workspace_bytes(9, 3, d), dtype=torch.uint8, device="cuda")
    gp.csa_norm_rope_fwd(x, 2, 9, 3, d, 3 * d, d, w, 1, 1e-6, None, None, 0, 0, 0, 1.0, y, 3 * d, d)
    gp.csa_norm_rope_bwd(x, dy, 2, 9, 3, d, 3 * d, d, 3 * d, d, w, 1, 1e-6, None, None, 0, 0, 0, 1.0, dx, 3 * d, d, dw, 0,
                         ws, ws.numel())
    torch.cuda.synchronize()
    ang = torch.zeros(9, 0, dtype=torch.float64)
    ref, mass = R.norm_rope(x.cpu(), w.cpu(), 1, 1e-6, ang, 0, 0, 0, 1.0)
    R.close(y, ref, mass, d, torch.float32, "y")
    rx, mx, rw, mw = R.norm_rope_bwd(x.cpu(), dy.cpu(), w.cpu(), 1, 1e-6, ang, 0, 0, 0, 1.0)
    R.close(dx, rx, mx, d, torch.float32, "dx")
    # each term as exact as the bound says, at most 64 plain additions in a row, the rest compensated
    assert ((dw.double().cpu() - rw).abs() <= (R.rope_bound(d, torch.float32) + 70 * R.U) * mw).all()


@pytest.mark.parametrize("rot,layout", [(64, 0), (30, 1)])
def test_one_row_turned_to_many_positions(cuda_lib, rot, layout):
    """An input that repeats (a row stride of 0)."""
    gp, g, d = cuda_lib, torch.Generator().manual_seed(rot), 64
    x = torch.randn(2, d, generator=g).cuda()
    pos = torch.arange(0, 70, dtype=torch.int32) * 1000003
    turns, amp = gp.csa_rope_table(rot)
    y = torch.empty(70, 2, d, device="cuda")
    gp.csa_norm_rope_fwd(x, 2, 70, 2, d, 0, d, None, 1, 1e-6, pos.cuda(), turns.cuda(), rot, 0, layout, amp, y, 2 * d, d)
    torch.cuda.synchronize()
    ref, mass = R.norm_rope(x.cpu().expand(70, 2, d), None, 1, 1e-6, R.angles(pos, turns), rot, 0, layout, amp)
    R.close(y, ref, mass, d, torch.float32, "y")


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
def test_one_row_written_to_many_slots(cuda_lib, fmt):
    """An input that repeats (strides of 0), heads too."""
    gp, d, rows, heads = cuda_lib, 64, 5, 3
    x = torch.randn(d, device="cuda").to(torch.bfloat16)
    width = {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt]
    data = torch.zeros(8, heads, width, dtype=torch.uint8, device="cuda")
    scales = None if fmt == R.BF16 else torch.zeros(8, heads, d // 32, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([7, 0, 3, -1, 4], device="cuda")
    gp.csa_cache_write(x, 0, rows, heads, d, 0, 0, slots, 8, fmt, data, scales)
    out = torch.full((rows, heads, d), 7.0, device="cuda")
    gp.csa_cache_read(data, scales, fmt, slots, rows, 8, heads, d, out, 2, heads * d, d)
    torch.cuda.synchronize()
    want = x.double().cpu()
    if fmt != R.BF16:
        want = R.dequantise(*R.quantise(want[None], fmt), fmt)[0]
    keep = [0, 1, 2, 4]
    assert torch.equal(out.cpu()[keep].double(), want.expand(4, heads, d)) and (out[3] == 7.0).all()
    assert not data[[1, 2, 5, 6]].any()
