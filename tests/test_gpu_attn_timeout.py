"""Bounded waits of the cache attention, exercised without any fault: the test hook shortens the bound to
about 10 ms and keeps the first block from filling one tile's place, so that the waits for it run
out. Checked for every way a tile comes in: the call returns with CSA_DEVERR_TIMEOUT, rows of no
sequence stay as they were, and the next call on the stream writes the bits of a normal one."""
import pytest
import torch

from tests import operator_reference as R
from tests.test_gpu_attn import Case

pytestmark = pytest.mark.gpu

WAIT_CYCLES = 20_000_000  # about 10 ms at GB300 clocks

CASES = {  # the first block's share has the withheld tile, the last ones some laps of the ring behind it too
    "threads, bf16": (dict(lens=[1], entries=[160_000], H=4, kv=1, d=128, page=9, ratio=0), [0, 1, 6]),
    "boxes": (dict(lens=[1], entries=[160_000], H=4, kv=1, d=128, page=64, ratio=0), [0, 1, 6]),
    "boxes, a tile a block": (dict(lens=[1], entries=[300], H=4, kv=1, d=512, page=64, ratio=0), [0]),
    "threads, 4 bits": (dict(lens=[1, 1], entries=[300, 40], H=4, kv=1, d=256, fmt=R.FP4, ratio=0), [0]),
    "threads helped, 8 bits": (dict(lens=[1], entries=[40_000], H=64, kv=1, d=512, fmt=R.E4M3, ratio=0), [0, 1]),
    "packed": (dict(lens=[40], entries=[6000], H=64, kv=1, d=128, fmt=R.E4M3, ratio=1, first="end"), [0, 1, 9]),
    "packed, one tile in the ring": (dict(lens=[40, 7], entries=[4000, 9], H=64, kv=1, d=512, page=64, ratio=1, first="end"),
                                     [0, 1, 3]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_wait_runs_out_and_call_returns(cuda_lib, name):
    gp, (how, tiles) = cuda_lib, CASES[name]
    c = Case(**how, seed=3, sink=True, lead=1)
    a, b = c.cu[0], c.cu[-1]
    out, lse, err = c.run(gp)
    assert err == 0
    for tile in tiles:
        gp.csa_compressor_test_hooks(WAIT_CYCLES, tile)
        try:
            got, glse, err = c.run(gp)
        finally:
            gp.csa_compressor_test_hooks(0, -1)
        assert err == gp.CSA_DEVERR_TIMEOUT, tile
        for t in (got, glse):
            assert (t[:a] == 7.0).all() and (t[b:] == 7.0).all()
        again, alse, err = c.run(gp)
        assert err == 0 and torch.equal(again, out) and torch.equal(alse, lse)


def test_a_shorter_bound_alone_changes_nothing(cuda_lib):
    c = Case([1, 40], [500, 700], 64, 1, 128, ratio=1, first="end", seed=4)
    out, lse, err = c.run(cuda_lib)
    cuda_lib.csa_compressor_test_hooks(WAIT_CYCLES, -1)
    try:
        got, glse, short = c.run(cuda_lib)
    finally:
        cuda_lib.csa_compressor_test_hooks(0, -1)
    assert err == 0 and short == 0 and torch.equal(got, out) and torch.equal(glse, lse)
