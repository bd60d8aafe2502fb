"""Rows normed, turned and put into the cache in one call, against the 64-bit form and the codes' definition:
types, formats, layouts, odd sizes, strides, both kernels, rows left out, bad slots, values out of the
ordinary, far slots and positions, graphs."""
import math

import pytest
import torch

from tests import operator_reference as R
from tests import serving_reference as V

pytestmark = pytest.mark.gpu
FORMATS = [R.BF16, R.E4M3, R.FP4]


def pool(num, heads, d, fmt, shift=0):
    width = {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt]
    data = torch.full((num * heads * width + 64,), 0x2A, dtype=torch.uint8, device="cuda")
    scales = None if fmt == R.BF16 else torch.full((num, heads, d // 32), 0x7E, dtype=torch.uint8, device="cuda")
    return data[shift:shift + num * heads * width].view(num, heads, width), scales


def append(gp, x, weight, norm, eps, pos, turns, rot, start, layout, amp, slots, num, fmt, data, scales):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows, heads, d = x.shape
    gp.csa_cache_append(x, R.DTYPES.index(x.dtype), rows, heads, d, x.stride(0), x.stride(1), weight, norm, eps, pos, turns, rot,
                        start, layout, amp, slots, num, fmt, data, scales, err)
    torch.cuda.synchronize()
    return int(err)


def check(x, weight, norm, eps, pos, turns, rot, start, layout, amp, slots, fmt, data, scales, was, scales_was, num):
    """Rows that are in against the reference, all other slots as they were."""
    live = [r for r in range(x.shape[0]) if (pos is None or pos[r] >= 0) and 0 <= slots[r] < num]
    ang = R.angles([0 if pos is None else int(pos[r]) for r in live], turns.tolist())
    want, off = V.append_values(x.cpu()[live], weight, norm, eps, ang, rot, start, layout, amp)
    at = [int(slots[r]) for r in live]
    data = data.cpu()
    if fmt == R.BF16:
        got = data[at].view(torch.bfloat16).double()
        half = R.HALF[torch.bfloat16]
        assert ((got - want).abs() <= half * want.abs() + (1 + half) * off + R.TINY[torch.bfloat16]).all()
    else:
        V.check_codes(R.unpack(data[at], fmt), scales.cpu()[at], fmt, want, off)
    rest = torch.ones(num, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(data[rest], was.cpu()[rest])
    assert scales is None or torch.equal(scales.cpu()[rest], scales_was.cpu()[rest])


CASES = [  # rows, heads, d, rot, start, slab, shift of x
    (1, 1, 512, 64, 448, 0, 0), (67, 1, 512, 64, 448, 0, 0), (33, 2, 128, 128, 0, 0, 0), (19, 3, 64, 32, 32, 1, 0),
    (5, 1, 96, 48, 16, 0, 0), (9, 2, 160, 16, 8, 0, 0), (7, 1, 32, 32, 0, 0, 0), (4, 2, 1024, 64, 0, 0, 0), (3, 1, 992, 16, 40, 0, 0),
    (40, 1, 128, 0, 0, 0, 0), (21, 2, 96, 34, 3, 0, 0), (6, 2, 128, 64, 0, 0, 1), (300, 8, 128, 64, 64, 0, 0), (700, 1, 512, 64, 448, 0, 0),
    (0, 1, 64, 0, 0, 0, 0)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("rows,heads,d,rot,start,slab,shift", CASES)
def test_append(cuda_lib, fmt, dtype, layout, rows, heads, d, rot, start, slab, shift):
    g = torch.Generator().manual_seed(rows + d + layout)
    flat = torch.zeros(rows * (heads + slab) * d + 16, dtype=dtype, device="cuda")
    x = flat[shift:shift + rows * (heads + slab) * d].view(rows, heads + slab, d)[:, slab:]
    x.copy_((torch.randn(rows, heads, d, generator=g) * torch.exp(torch.randn(rows, heads, 1, generator=g))).to(dtype))
    norm = int((rows + d) % 3 != 0)
    weight = 1 + 0.1 * torch.randn(d, generator=g) if norm and rows % 2 else None
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    num = rows + 30
    slots = torch.randperm(num, generator=g)[:rows]
    if rows > 3:
        pos[1], slots[3] = -1, -9
    turns, amp = cuda_lib.csa_rope_table(rot, 10000.0)
    amp = 1.25
    data, scales = pool(num, heads, d, fmt)
    was, scales_was = data.clone(), None if scales is None else scales.clone()
    err = append(cuda_lib, x, None if weight is None else weight.cuda(), norm, 1e-6, pos.cuda(), turns.cuda() if rot else None, rot,
                 start, layout, amp, slots.cuda(), num, fmt, data, scales)
    assert err == 0
    check(x, weight, norm, 1e-6, pos.tolist(), turns, rot, start, layout, amp, slots.tolist(), fmt, data, scales, was, scales_was, num)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,rot", [(45, 6), (128, 64), (7, 0)])
def test_odd_sizes_and_no_positions(cuda_lib, fmt, d, rot):
    if fmt != R.BF16 and d % 32:
        pytest.skip("codes need groups of 32")
    g = torch.Generator().manual_seed(d)
    x = torch.randn(11, 3, d, generator=g).cuda()
    pos = None if rot == 0 else torch.arange(11, dtype=torch.int32)
    turns, _ = cuda_lib.csa_rope_table(rot)
    slots = torch.arange(20, 31)
    data, scales = pool(40, 3, d, fmt, shift=2)  # (an unaligned pool: the scalar kernel)
    was, scales_was = data.clone(), None if scales is None else scales.clone()
    assert append(cuda_lib, x, None, 1, 1e-5, None if pos is None else pos.cuda(), turns.cuda() if rot else None, rot, 0, 0, 1.0,
                  slots.cuda(), 40, fmt, data, scales) == 0
    check(x, None, 1, 1e-5, None if pos is None else pos.tolist(), turns, rot, 0, 0, 1.0, slots.tolist(), fmt, data, scales, was,
          scales_was, 40)


@pytest.mark.parametrize("d", [128, 45])
def test_slots_past_the_pool(cuda_lib, d):
    x = torch.ones(6, 1, d, dtype=torch.bfloat16, device="cuda")
    data, _ = pool(4, 1, d, R.BF16)
    was = data.clone()
    slots = torch.tensor([0, 4, 1 << 40, 3, -1, -(1 << 40)], device="cuda")
    assert append(cuda_lib, x, None, 0, 0.0, None, None, 0, 0, 0, 1.0, slots, 4, R.BF16, data, None) == 5
    got = data.cpu().view(torch.bfloat16)
    assert (got[[0, 3]] == 1).all() and torch.equal(data[1:3], was[1:3])


@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
@pytest.mark.parametrize("shift", [0, 1])
def test_values_out_of_the_ordinary(cuda_lib, fmt, shift):
    """Without a norm: zeros, subnormals, ties, the largest value, infinities and NaN as csa_cache_write has them,
    code by code; with one, a NaN makes its row NaN, and an infinity the group that holds it (the other columns
    are divided by an infinite root: 0)."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 1, 64, generator=g)
    x[0] = 0
    x[1] *= 2.0 ** -140
    x[2, 0, :32] = torch.arange(32) / 4 - 3
    x[3, 0, 5] = 3.4e38
    x[4, 0, 40] = math.inf
    x[5, 0, 3] = math.nan
    x[6, 0, :32] = -0.0
    slots = torch.arange(9)
    data, scales = pool(9, 1, 64, fmt, shift)
    assert append(cuda_lib, x.cuda(), None, 0, 0.0, None, None, 0, 0, 0, 1.0, slots.cuda(), 9, fmt, data, scales) == 0
    codes, k = R.quantise(x.double(), fmt)
    assert torch.equal(scales.cpu().long(), k)
    fine = (k != 255).repeat_interleave(32, -1)
    assert torch.equal(R.unpack(data.cpu(), fmt)[fine], codes[fine])
    assert append(cuda_lib, x.cuda(), None, 1, 1e-6, None, None, 0, 0, 0, 1.0, slots.cuda(), 9, fmt, data, scales) == 0
    assert (scales.cpu()[5] == 255).all() and scales.cpu()[4, 0].tolist() == [0, 255]
    assert (R.unpack(data.cpu(), fmt)[4, 0, :32] % (128 if fmt == R.E4M3 else 8) == 0).all()
    assert (scales.cpu()[[0, 1, 2, 6, 7, 8]] != 255).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_far_slots_and_positions(cuda_lib, fmt):
    """Slots whose bytes pass 32 bits, positions near 2^31."""
    d, heads = 512, 8
    num = (1 << 32) // (heads * 256) + 4099 if fmt == R.FP4 else (1 << 32) // (heads * 512) + 4099
    width = {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt]
    data = torch.zeros(num, heads, width, dtype=torch.uint8, device="cuda")
    scales = None if fmt == R.BF16 else torch.zeros(num, heads, d // 32, dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(4)
    x = torch.randn(4, heads, d, generator=g).to(torch.bfloat16)
    slots, pos = [num - 1, 0, num - 4000, num // 2], [2 ** 31 - 1, 5, 2 ** 30 + 1, 0]
    turns, _ = cuda_lib.csa_rope_table(64)
    assert append(cuda_lib, x.cuda(), None, 1, 1e-6, torch.tensor(pos, dtype=torch.int32).cuda(), turns.cuda(), 64, 448, 1, 1.0,
                  torch.tensor(slots).cuda(), num, fmt, data, scales) == 0
    want, off = V.append_values(x, None, 1, 1e-6, R.angles(pos, turns.tolist()), 64, 448, 1, 1.0)
    got = data[slots].cpu()
    if fmt == R.BF16:
        assert ((got.view(torch.bfloat16).double() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * off).all()
    else:
        V.check_codes(R.unpack(got, fmt), scales[slots].cpu(), fmt, want, off)


def test_graph_and_repeats(cuda_lib):
    """A captured call on other rows than it was captured with; the same bits from the same inputs."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 1, 512, generator=g).to(torch.bfloat16).cuda()
    pos, slots = torch.arange(40, dtype=torch.int32).cuda(), torch.randperm(64, generator=g)[:40].cuda()
    turns, _ = cuda_lib.csa_rope_table(64)
    turns = turns.cuda()

    def call(data, scales):
        cuda_lib.csa_cache_append(x, 0, 40, 1, 512, 512, 512, None, 1, 1e-6, pos, turns, 64, 448, 1, 1.0, slots, 64, R.E4M3, data, scales)

    one, two = pool(64, 1, 512, R.E4M3), pool(64, 1, 512, R.E4M3)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call(*pool(64, 1, 512, R.E4M3))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call(*two)
    torch.cuda.synchronize()
    x.mul_(1.5)
    pos[7] = -1
    slots.copy_(slots.flip(0))
    call(*one)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_heads_up_to_the_last_number(cuda_lib):
    """2^31 - 1 rows' heads that repeat one row of x: the count goes on past 2^31 in no warp."""
    heads, d = 2 ** 31 - 1, 8
    x = torch.randn(1, 1, d).to(torch.bfloat16).cuda()
    data = torch.zeros(heads, d, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cuda_lib.csa_cache_append(x, 0, 1, heads, d, 0, 0, None, 0, 0.0, None, None, 0, 0, 0, 1.0, torch.zeros(1, dtype=torch.int64, device="cuda"),
                              1, R.BF16, data, None, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for at in range(0, heads, 1 << 28):
        assert (data[at:at + (1 << 28)].view(torch.int64) == x.view(torch.int64).view(1, 2)).all()
