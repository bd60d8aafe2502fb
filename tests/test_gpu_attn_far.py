"""Cache attention over pools whose last pages lie past 32 bits of bytes, in every way a tile comes in but
tensor copies of the pages (tests/test_gpu_attn.py has those): the same bits as from a small pool."""
import pytest
import torch

from tests import operator_reference as R
from tests.test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,H,kv,d,fmt,page,lens,ratio", [
    ("threads", 4, 1, 256, R.BF16, 9, [2], 0), ("threads at 512", 4, 1, 512, R.BF16, 9, [2], 0),
    ("threads, 8 bits", 4, 1, 128, R.E4M3, 16, [2], 0), ("helped, 8 bits", 4, 1, 512, R.E4M3, 16, [2], 0),
    ("threads, 4 bits", 4, 1, 512, R.FP4, 16, [2], 0), ("heads", 4, 2, 256, R.E4M3, 16, [2], 0),
    ("packed", 64, 1, 512, R.BF16, 16, [9], 1), ("packed, 8 bits", 64, 1, 512, R.E4M3, 9, [9], 1),
    ("scalar", 2, 1, 1000, R.BF16, 16, [2], 0), ("scalar, 8 bits", 2, 1, 544, R.E4M3, 16, [2], 0)])
def test_last_pages_of_a_large_pool(cuda_lib, name, H, kv, d, fmt, page, lens, ratio):
    gp = cuda_lib
    c = Case(lens, [150], H, kv, d, fmt, page=page, ratio=ratio, first="end", seed=8)
    out, lse, err, args = c.run(gp, keep=True)
    assert err == 0
    args = list(args)
    row = c.data[0].numel() * c.data.element_size()
    pages = (1 << 32) // (page * row) + 40
    data = torch.empty((pages * page,) + tuple(c.data.shape[1:]), dtype=c.data.dtype, device="cuda")
    scales = None if c.scales is None else torch.empty((pages * page,) + tuple(c.scales.shape[1:]), dtype=torch.uint8,
                                                       device="cuda")
    used = -(-150 // page)
    for i in range(used):
        src, to = int(c.table[0, i]) * page, (pages - 1 - i) * page
        data[to:to + page] = c.data[src:src + page].cuda()
        if scales is not None:
            scales[to:to + page] = c.scales[src:src + page].cuda()
    args[9], args[10], args[14] = data, scales, pages
    args[12][0, :used] = torch.tensor([pages - 1 - i for i in range(used)], dtype=torch.int32)
    want, wl = out.clone(), lse.clone()
    args[21].fill_(7.0)
    args[24].fill_(7.0)
    gp.csa_cache_attn(*args)
    torch.cuda.synchronize()
    assert int(args[27]) == 0 and torch.equal(args[21], want) and torch.equal(args[24], wl)
