"""Host side of the serving step's entry points: every refusal, and the references against plain loops. CPU
only: each call is refused (or is an empty one) before any CUDA runtime call."""
import math

import pytest
import torch

import gated_pooling_gb300 as gp
from tests import operator_reference as R
from tests import serving_reference as V

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced
INVALID, UNSUPPORTED, WORKSPACE, OK = (gp.CSA_ERR_INVALID_VALUE, gp.CSA_ERR_UNSUPPORTED, gp.CSA_ERR_WORKSPACE, gp.CSA_OK)


@pytest.fixture(scope="module")
def lib():
    return gp.load()


# ------------------------------------------------------------------------------------- step
def step(lib, **over):
    a = dict(kv=FAKE, score=FAKE, ape=FAKE, cu=FAKE, S=2, ratio=4, coff=2, d=64, capacity=16, first=FAKE, source=FAKE, target=FAKE,
             states=4, kvs=FAKE, scs=FAKE, out=FAKE, rows=8, base=FAKE, table=FAKE, max_pages=4, page=16, offset=0, pos=FAKE, slots=FAKE,
             entries=FAKE, err=None)
    a.update(over)
    return lib.csa_compressor_step(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(S=-1), INVALID), (dict(ratio=0), INVALID), (dict(d=0), INVALID), (dict(capacity=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(states=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(page=0), INVALID), (dict(offset=-1), INVALID),
    (dict(offset=4), INVALID), (dict(coff=0), UNSUPPORTED), (dict(coff=3), UNSUPPORTED), (dict(S=20000), UNSUPPORTED),
    (dict(ratio=1025), UNSUPPORTED), (dict(ratio=2049, coff=1), UNSUPPORTED), (dict(d=1 << 20), UNSUPPORTED),
    (dict(capacity=1 << 25), UNSUPPORTED), (dict(rows=1 << 26), UNSUPPORTED), (dict(states=1 << 31), UNSUPPORTED),
    (dict(states=1 << 62), UNSUPPORTED), (dict(kv=None), INVALID), (dict(score=None), INVALID), (dict(ape=None), INVALID),
    (dict(cu=None), INVALID), (dict(first=None), INVALID), (dict(source=None), INVALID), (dict(target=None), INVALID),
    (dict(kvs=None), INVALID), (dict(scs=None), INVALID), (dict(out=None), INVALID), (dict(table=None), INVALID),
    (dict(kv=FAKE + 1), INVALID), (dict(score=FAKE + 1), INVALID), (dict(ape=FAKE + 2), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(first=FAKE + 2), INVALID), (dict(source=FAKE + 2), INVALID), (dict(target=FAKE + 2), INVALID), (dict(kvs=FAKE + 1), INVALID),
    (dict(scs=FAKE + 1), INVALID), (dict(out=FAKE + 1), INVALID), (dict(base=FAKE + 2), INVALID), (dict(table=FAKE + 2), INVALID),
    (dict(pos=FAKE + 2), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(entries=FAKE + 2), INVALID), (dict(err=FAKE + 1), INVALID),
    (dict(S=0, rows=0), OK), (dict(S=0, pos=None, slots=None), OK),
])
def test_step_refusals(lib, over, code):
    assert step(lib, **over) == code


# ----------------------------------------------------------------------------------- append
def append(lib, **over):
    a = dict(x=FAKE, dtype=0, rows=4, heads=2, d=64, xr=128, xh=64, w=FAKE, norm=1, eps=1e-6, pos=FAKE, turns=FAKE, rot=64, start=0,
             layout=0, amp=1.0, slots=FAKE, n=16, fmt=1, data=FAKE, scales=FAKE, err=None)
    a.update(over)
    return lib.csa_cache_append(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(d=0), INVALID), (dict(norm=2), INVALID), (dict(rot=63), INVALID),
    (dict(rot=-2), INVALID), (dict(rot=66), INVALID), (dict(start=2), INVALID), (dict(start=-1, rot=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(xr=-1), INVALID),
    (dict(xh=-1), INVALID), (dict(n=-1), INVALID), (dict(pos=None), INVALID), (dict(turns=None), INVALID), (dict(x=None), INVALID),
    (dict(slots=None), INVALID), (dict(data=None), INVALID), (dict(scales=None), INVALID), (dict(norm=0), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(x=FAKE + 2, dtype=2), INVALID), (dict(w=FAKE + 2), INVALID), (dict(pos=FAKE + 2), INVALID),
    (dict(turns=FAKE + 4), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(err=FAKE + 2), INVALID),
    (dict(data=FAKE + 1, fmt=0), INVALID), (dict(d=1056), UNSUPPORTED), (dict(rows=1 << 31, heads=1), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED),
    (dict(d=72), UNSUPPORTED), (dict(n=1 << 62), UNSUPPORTED),
    (dict(rows=0), OK), (dict(rows=0, x=None, slots=None, pos=None, turns=None), OK),
])
def test_append_refusals(lib, over, code):
    assert append(lib, **over) == code


# ------------------------------------------------------------------ attention behind prefixes
def attn(lib, **over):
    a = dict(q=FAKE, qr=128, qh=64, cu=FAKE, S=2, tokens=4, H=2, kv=1, d=64, data=FAKE, scales=FAKE, fmt=1, seqs=FAKE, G=1, ptable=FAKE,
             max_prefix=4, pentries=FAKE, table=FAKE, max_pages=4, num_pages=8, page=16, entries=FAKE, first=FAKE, ratio=4, scale=0.125,
             sink=FAKE, out=FAKE, outr=128, outh=64, lse=FAKE, ws=FAKE, nb=1 << 30, err=None)
    a.update(over)
    return lib.csa_cache_attn_prefix(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(S=-1), INVALID), (dict(tokens=-1), INVALID), (dict(H=0), INVALID), (dict(kv=0), INVALID), (dict(H=3, kv=2), INVALID),
    (dict(d=0), INVALID), (dict(G=-1), INVALID), (dict(G=0), INVALID), (dict(max_prefix=-1), INVALID), (dict(seqs=None), INVALID),
    (dict(ptable=None), INVALID), (dict(pentries=None), INVALID), (dict(seqs=FAKE + 2), INVALID), (dict(ptable=FAKE + 2), INVALID),
    (dict(pentries=FAKE + 2), INVALID), (dict(max_pages=-1), INVALID), (dict(num_pages=-1), INVALID), (dict(page=0), INVALID),
    (dict(ratio=-1), INVALID), (dict(qr=-1), INVALID), (dict(qh=-1), INVALID), (dict(outr=-1), INVALID), (dict(outh=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(cu=None), INVALID), (dict(entries=None), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(table=None), INVALID), (dict(data=None), INVALID),
    (dict(scales=None), INVALID), (dict(q=FAKE + 1), INVALID), (dict(out=FAKE + 1), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(table=FAKE + 2), INVALID), (dict(entries=FAKE + 2), INVALID), (dict(first=FAKE + 2), INVALID),
    (dict(sink=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(err=FAKE + 2), INVALID), (dict(ws=FAKE + 8), INVALID),
    (dict(data=FAKE + 1, fmt=0), INVALID), (dict(d=1025, fmt=0), UNSUPPORTED), (dict(d=72), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED),
    (dict(S=20000), UNSUPPORTED), (dict(G=20000), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED),
    (dict(max_pages=1 << 30), UNSUPPORTED), (dict(max_prefix=1 << 30), UNSUPPORTED),
    (dict(max_pages=1 << 26, max_prefix=1 << 26), UNSUPPORTED), (dict(num_pages=1 << 60), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(nb=8), WORKSPACE), (dict(S=0), OK), (dict(S=0, G=0, seqs=None, ptable=None, pentries=None), OK), (dict(tokens=0), OK),
    (dict(outh=63), INVALID), (dict(outr=127), INVALID), (dict(outr=0), INVALID), (dict(outr=64, outh=255), INVALID),
])
def test_attn_refusals(lib, over, code):
    assert attn(lib, **over) == code


def test_attn_workspace_query_refuses(lib):
    for bad in ((-1, 1, 1, 1, 1, 64, 16, 16), (1, 0, 1, 1, 1, 64, 16, 16), (1, -1, 1, 1, 1, 64, 16, 16), (1, 20000, 1, 1, 1, 64, 16, 16),
                (1, 1, 1, 1, 1, 64, -1, 16), (1, 1, 1, 1, 1, 64, 16, -1), (1, 1, 1, 1, 1, 64, 1 << 30, 1 << 30),
                (1, 1, 1, 3, 2, 64, 16, 16), (1, 1, 1, 1, 1, 1025, 16, 16)):
        assert gp.csa_cache_attn_prefix_workspace_bytes(*bad) == 0


# ------------------------------------------------------------- the references check themselves
@pytest.mark.parametrize("ratio,coff", [(1, 1), (1, 2), (3, 1), (4, 2)])
def test_held_elements_are_those_that_later_windows_read(ratio, coff):
    """By trying every later block: an element is held when its token is there and a window to come reads it."""
    d = 2
    for total in range(0, 5 * ratio):
        want = {}
        for b in range(total // ratio, total // ratio + 3):
            for p in range(max(0, (b - coff + 1) * ratio), (b + 1) * ratio):
                half = 0 if coff == 1 or p < b * ratio else 1
                if p < total:
                    want[p % (ratio * coff), half] = p
        got = V.held(0, total, ratio, coff, d)
        for r in range(ratio * coff):
            for half in range(coff):
                assert (got[r, half * d:half * d + d] == want.get((r, half), -1)).all()


def test_window_entry_of_equal_scores_is_the_mean():
    kv = torch.arange(16.0).reshape(8, 2).to(torch.bfloat16)
    zero, ape = torch.zeros(8, 2, dtype=torch.bfloat16), torch.zeros(4, 2)
    out, bound = V.window_entry(kv, zero, ape, 1, 4, 2, 1)
    assert abs(float(out[0]) - (0 + 2 + 4 + 6 + 9 + 11 + 13 + 15) / 8) < 1e-12 and float(bound[0]) < 2 * 2.0 ** -8 * 7.5


@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
def test_code_check_takes_the_quantiser_and_refuses_a_step_off(fmt):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 64, generator=g, dtype=torch.float64)
    codes, k = R.quantise(x, fmt)
    V.check_codes(codes, k, fmt, x, torch.zeros_like(x))
    for c, s in ((codes, k + 1), (codes, k - 1), (codes.clone(), k)):
        if s is k:
            mag = 126 if fmt == R.E4M3 else 7
            c[3, 5] += 2 if (int(c[3, 5]) & mag) < mag - 2 else -2
        with pytest.raises(AssertionError):
            V.check_codes(c, s, fmt, x, torch.zeros_like(x))


# ------------------------------------------------------------------------ calls from Python
def python_append(**over):
    a = dict(x=FAKE, dtype=0, rows=0, heads=2, d=64, x_row_stride=128, x_head_stride=64, weight=None, norm=1, eps=1e-6, positions=FAKE,
             turns=FAKE, rot_dim=64, rot_start=0, layout=0, amplitude=1.0, slots=FAKE, num_slots=16, format=1, data=FAKE, scales=FAKE,
             dev_error=None, stream=0)
    a.update(over)
    gp.csa_cache_append(**a)


def test_python_calls_marshal_and_raise(lib):
    t = torch.zeros(64)
    python_append()                        # addresses and None
    python_append(x=t, weight=t, slots=t)  # tensors
    python_append(norm=True, eps=0, amplitude=1)
    for over, code in ((dict(x=FAKE + 1), INVALID), (dict(d=72), UNSUPPORTED), (dict(weight=FAKE + 2), INVALID)):
        with pytest.raises(gp.CsaError) as e:
            python_append(**over)
        assert e.value.status == code and "csa_cache_append" in str(e.value)
    for over, kind in ((dict(heads=1 << 31), OverflowError), (dict(rows=1 << 63), OverflowError), (dict(x=-1), OverflowError),
                       (dict(x="x"), AttributeError), (dict(d=1.5), TypeError), (dict(eps="1"), TypeError)):
        with pytest.raises(kind):
            python_append(**over)


def test_python_calls_and_ctypes_share_one_library(lib):
    python_append()
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libcsa_compressor" in line}
    assert len(paths) == 1
