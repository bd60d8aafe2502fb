"""Rows into the paged cache and back through the C ABI, against the formats' definition code by
code: every type and format, vector and scalar kernels, strides, rows left out, bad slots, zeros,
infinities and NaN, subnormals, ties, and slots whose byte offset passes 32 bits."""
import pytest
import torch

from tests import operator_reference as R

pytestmark = pytest.mark.gpu
FORMATS = [R.BF16, R.E4M3, R.FP4]


def pool(slots, heads, d, fmt, shift=0):
    """data and scales filled with a pattern."""
    width = {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt]
    raw = torch.full((slots * heads * width + 16,), 0x2A, dtype=torch.uint8, device="cuda")
    data = raw[shift:shift + slots * heads * width].view(slots, heads, width)
    scales = None
    if fmt != R.BF16:
        raw = torch.full((slots * heads * (d // 32) + 16,), 0x7F, dtype=torch.uint8, device="cuda")
        scales = raw[shift:shift + slots * heads * (d // 32)].view(slots, heads, d // 32)
    return data, scales


def strided(rows, heads, d, dtype, slab, shift):
    flat = torch.zeros(rows * (heads + slab) * d + 16, dtype=dtype, device="cuda")
    return flat[shift:shift + rows * (heads + slab) * d].view(rows, heads + slab, d)[:, slab:]


def write(gp, x, slots, num, fmt, data, scales):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows, heads, d = x.shape
    gp.csa_cache_write(x, R.DTYPES.index(x.dtype), rows, heads, d, x.stride(0), x.stride(1), slots, num, fmt, data,
                       scales, err)
    torch.cuda.synchronize()
    return int(err)


def read(gp, data, scales, fmt, slots, num, d, out):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows, heads, d = out.shape
    gp.csa_cache_read(data, scales, fmt, slots, rows, num, heads, d, out, R.DTYPES.index(out.dtype), out.stride(0),
                      out.stride(1), err)
    torch.cuda.synchronize()
    return int(err)


def stored(data, scales, fmt):
    """Values that the cache's bytes stand for, in 64 bits on the CPU."""
    if fmt == R.BF16:
        return data.cpu().view(torch.bfloat16).double()
    return R.dequantise(R.unpack(data.cpu(), fmt), scales.cpu().long(), fmt)


def rounded(v, dtype):
    """fp32 values (exact in it) rounded once to a type."""
    return v.float().to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", R.DTYPES)
@pytest.mark.parametrize("rows,heads,d,slab,shift", [
    (1, 1, 512, 0, 0), (67, 1, 512, 0, 0), (19, 3, 128, 0, 0), (33, 2, 96, 0, 0), (5, 1, 32, 0, 0), (9, 5, 64, 2, 0),
    (9, 2, 160, 0, 1), (4, 2, 640, 1, 1), (300, 8, 128, 0, 0), (0, 1, 128, 0, 0), (7, 2, 224, 0, 8)])
def test_write_and_read(cuda_lib, fmt, dtype, rows, heads, d, slab, shift):
    g = torch.Generator().manual_seed(rows + d)
    x = strided(rows, heads, d, dtype, slab, shift)
    x.copy_((torch.randn(rows, heads, d, generator=g) * torch.exp(2 * torch.randn(rows, heads, 1, generator=g))).to(dtype))
    num = rows + 40
    slots = torch.randperm(num, generator=g)[:rows].cuda()
    if rows > 3:
        slots[2] = -5
    data, scales = pool(num, heads, d, fmt, shift if fmt != R.BF16 else 2 * shift)
    was, scales_was = data.clone(), None if scales is None else scales.clone()
    assert write(cuda_lib, x, slots, num, fmt, data, scales) == 0
    live = slots.cpu() >= 0
    xd = x.double().cpu()[live]
    at = slots.cpu()[live]
    if fmt == R.BF16:
        assert torch.equal(data.cpu()[at].view(torch.int16), x[live.cuda()].to(torch.bfloat16).cpu().view(torch.int16))
    else:
        codes, k = R.quantise(xd, fmt)
        assert torch.equal(scales.cpu()[at].long(), k) and torch.equal(R.unpack(data.cpu()[at], fmt), codes)
    rest = torch.ones(num, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(data.cpu()[rest], was.cpu()[rest])  # every other slot as it was
    assert scales is None or torch.equal(scales.cpu()[rest], scales_was.cpu()[rest])
    for back in R.DTYPES:
        out = strided(rows, heads, d, back, slab, shift)
        out.fill_(7.0)
        assert read(cuda_lib, data, scales, fmt, slots, num, d, out) == 0
        assert torch.equal(out.cpu()[live], rounded(stored(data, scales, fmt)[at], back))
        assert (out.cpu()[~live] == 7.0).all()


@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
@pytest.mark.parametrize("shift", [0, 1])
def test_every_corner_of_the_scale(cuda_lib, fmt, shift):
    """Groups at every binade of fp32, at the largest value's border, ties, signs, zeros, subnormals."""
    most, rows = R.MOST[fmt], []
    table = R.code_values(fmt)[:127 if fmt == R.E4M3 else 8]
    ties = ((table[1:] + table[:-1]) / 2)
    g = torch.Generator().manual_seed(1)
    for e in range(-149, 128, 3):
        v = torch.randn(32, generator=g, dtype=torch.float64) * 2.0 ** e
        rows.append(v.float().clamp(-3e38, 3e38))
    for e in (-126, -20, 0, 7, 100):
        for top in (most, most * (1 + 2.0 ** -23), most * (1 - 2.0 ** -24), most / 2, most / 2 * (1 + 2.0 ** -23)):
            v = ties[torch.randint(0, len(ties), (32,), generator=g)] * (2 * torch.randint(0, 2, (32,), generator=g) - 1)
            v[5], v[6], v[7] = top, 0.0, -0.0
            rows.append((v * 2.0 ** e).float())
    rows += [torch.zeros(32), torch.full((32,), -0.0), torch.full((32,), 3.4028234663852886e38)]
    for bad in (float("inf"), -float("inf"), float("nan")):
        v = torch.ones(32)
        v[9] = bad
        rows.append(v)
    x = strided(1, len(rows), 32, torch.float32, 0, shift)
    x.copy_(torch.stack(rows)[None])
    data, scales = pool(1, len(rows), 32, fmt, shift)
    assert write(cuda_lib, x, torch.zeros(1, dtype=torch.int64, device="cuda"), 1, fmt, data, scales) == 0
    codes, k = R.quantise(x.double().cpu(), fmt)
    assert torch.equal(scales.cpu().long(), k)
    fine = (k != 255).repeat_interleave(32, -1)
    assert torch.equal(R.unpack(data.cpu(), fmt)[fine], codes[fine])
    out = torch.zeros(1, len(rows), 32, device="cuda")
    assert read(cuda_lib, data, scales, fmt, torch.zeros(1, dtype=torch.int64, device="cuda"), 1, 32, out) == 0
    want = stored(data, scales, fmt)
    assert torch.equal(torch.isnan(out).cpu(), ~fine) and torch.equal(out.cpu()[fine], want.float()[fine])
    assert int((~fine).sum()) == 3 * 32


@pytest.mark.parametrize("fmt", FORMATS)
def test_all_codes_read_back(cuda_lib, fmt):
    """Every code at several scales, in every type (a code's value rounds once)."""
    if fmt == R.BF16:
        codes = torch.arange(1 << 16, dtype=torch.int32).to(torch.uint16).view(torch.uint8).reshape(64, 1, -1)
        data, scales, d = codes.cuda(), None, 1024
    else:
        n = 256
        codes = torch.arange(n, dtype=torch.int64).to(torch.uint8).reshape(1, 1, n).repeat(64, 1, 1)
        data, d = codes.cuda(), n if fmt == R.E4M3 else 2 * n
        scales = torch.arange(64 * (d // 32), dtype=torch.int64).remainder(256).to(torch.uint8).reshape(64, 1, -1).cuda()
    slots = torch.arange(64, device="cuda").flip(0).contiguous()
    for dtype in R.DTYPES:
        out = torch.zeros(64, 1, d, dtype=dtype, device="cuda")
        assert read(cuda_lib, data, scales, fmt, slots, 64, d, out) == 0
        want = rounded(stored(data, scales, fmt), dtype).flip(0)
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(out).cpu(), nan) and torch.equal(out.cpu()[~nan], want[~nan])


def test_bad_slots(cuda_lib):
    """A slot past the pool is reported, its row left out, the others done."""
    for fmt, shift in ((R.BF16, 0), (R.E4M3, 0), (R.FP4, 0), (R.E4M3, 1)):
        x = strided(4, 2, 64, torch.bfloat16, 0, shift)
        x.copy_(torch.randn(4, 2, 64).to(torch.bfloat16))
        data, scales = pool(8, 2, 64, fmt, shift)
        was = data.clone()
        slots = torch.tensor([3, 8, 1 << 40, 0], device="cuda")
        assert write(cuda_lib, x, slots, 8, fmt, data, scales) == cuda_lib.CSA_DEVERR_SLOT
        changed = (data != was).flatten(1).any(1).cpu()
        assert changed.tolist() == [True, False, False, True, False, False, False, False]
        out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        assert read(cuda_lib, data, scales, fmt, slots, 8, 64, out) == cuda_lib.CSA_DEVERR_SLOT
        assert (out[1:3] == 7.0).all() and not (out[0] == 7.0).all() and not (out[3] == 7.0).all()


def test_offsets_past_32_bits(cuda_lib):
    """A pool of 4.3 GB: its last slots."""
    num, d = (1 << 32) // 512 + 64, 512
    data = torch.empty(num, 1, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(num, 1, d // 32, dtype=torch.uint8, device="cuda")
    x = torch.randn(3, 1, d, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([num - 1, num - 40, 5], device="cuda")
    assert write(cuda_lib, x, slots, num, R.E4M3, data, scales) == 0
    out = torch.empty_like(x)
    assert read(cuda_lib, data, scales, R.E4M3, slots, num, d, out) == 0
    codes, k = R.quantise(x.double().cpu(), R.E4M3)
    assert torch.equal(out.cpu(), R.dequantise(codes, k, R.E4M3).to(torch.bfloat16))


def test_same_slot_read_twice_and_graph(cuda_lib):
    x = torch.randn(16, 1, 128, device="cuda").to(torch.bfloat16)
    data, scales = pool(32, 1, 128, R.FP4)
    slots = torch.arange(16, device="cuda")
    again = torch.tensor([3, 3, 0, 15, 3], device="cuda")
    out = torch.zeros(5, 1, 128, dtype=torch.bfloat16, device="cuda")

    def calls():
        cuda_lib.csa_cache_write(x, 0, 16, 1, 128, 128, 128, slots, 32, R.FP4, data, scales)
        cuda_lib.csa_cache_read(data, scales, R.FP4, again, 5, 32, 1, 128, out, 0, 128, 128)

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        calls()
    x.copy_(torch.randn(16, 1, 128).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    codes, k = R.quantise(x.double().cpu(), R.FP4)
    assert torch.equal(out.cpu(), R.dequantise(codes, k, R.FP4).to(torch.bfloat16)[again.cpu()])
