"""Host side of the norm-and-rotation, cache and cache-attention entry points: the frequency
table against its formulas, the header's constants, and every refusal. CPU only: each call
is refused (or is an empty one) before any CUDA runtime call."""
import math
import os
import re

import pytest
import torch

import gated_pooling_gb300 as gp
from tests import operator_reference as R

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced
INVALID, UNSUPPORTED, WORKSPACE, OK = (gp.CSA_ERR_INVALID_VALUE, gp.CSA_ERR_UNSUPPORTED,
                                       gp.CSA_ERR_WORKSPACE, gp.CSA_OK)


@pytest.fixture(scope="module")
def lib():
    return gp.load()


def test_constants_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "csa_compressor.h")).read()
    names = re.findall(r"#define (CSA_(?:DTYPE|ROPE|CACHE|MAX_HEAD|DEVERR)\w*) (\d+)", text)
    assert len(names) >= 18
    for name, value in names:
        assert getattr(gp, name) == int(value), name


# ------------------------------------------------------------------------------ the table
@pytest.mark.parametrize("rot", [2, 64, 128, 130])
@pytest.mark.parametrize("args", [dict(), dict(base=500000.0), dict(scaling=1, factor=4.0),
                                  dict(scaling=2, factor=16.0, original_length=4096.0),
                                  dict(scaling=2, factor=40.0, original_length=8192.0, beta_fast=16.0,
                                       beta_slow=2.0),
                                  dict(scaling=2, factor=2.0, original_length=8.0)])
def test_table(lib, rot, args):
    turns, amp = gp.csa_rope_table(rot, **args)
    freq, want_amp = R.frequencies(rot, args.get("base", 10000.0), args.get("scaling", 0),
                                   args.get("factor", 1.0), args.get("original_length", 4096.0),
                                   args.get("beta_fast", 32.0), args.get("beta_slow", 1.0))
    assert turns.shape == (rot // 2,) and abs(amp - want_amp) <= R.U * want_amp
    for t, f in zip(turns.tolist(), freq):
        # pow, log and the blend in 64 bits: a few steps of 2^-53 each; and the rounding to a
        # whole number of units, half a unit = 2^-65 of a turn = 2 pi 2^-65
        bound = 32 * 2.0 ** -53 * f + 2 * math.pi * 2.0 ** -65
        assert abs((t % (1 << 64)) / 2.0 ** 64 * 2 * math.pi - f) <= bound


def test_table_of_nothing(lib):
    turns, amp = gp.csa_rope_table(0)
    assert turns.numel() == 0 and amp == 1.0


@pytest.mark.parametrize("args,code", [
    ((3, 1e4, 0, 1, 1, 1, 1), INVALID), ((-2, 1e4, 0, 1, 1, 1, 1), INVALID),
    ((64, 1.0, 0, 1, 1, 1, 1), INVALID), ((64, math.nan, 0, 1, 1, 1, 1), INVALID),
    ((64, math.inf, 0, 1, 1, 1, 1), INVALID), ((64, 1e4, 1, 0.5, 1, 1, 1), INVALID),
    ((64, 1e4, 1, math.nan, 1, 1, 1), INVALID), ((64, 1e4, 2, 4, 0.5, 32, 1), INVALID),
    ((64, 1e4, 2, 4, 4096, 0, 1), INVALID), ((64, 1e4, 2, 4, 4096, 32, -1), INVALID),
    ((64, 1e4, 3, 1, 1, 1, 1), UNSUPPORTED), ((64, 1e4, -1, 1, 1, 1, 1), UNSUPPORTED),
    ((1026, 1e4, 0, 1, 1, 1, 1), UNSUPPORTED),
])
def test_table_refusals(lib, args, code):
    buf = torch.zeros(1024, dtype=torch.int64)
    assert lib.csa_rope_table(*args, buf.data_ptr(), None) == code


def test_table_needs_its_buffer(lib):
    assert lib.csa_rope_table(64, 1e4, 0, 1, 1, 1, 1, None, None) == INVALID


# --------------------------------------------------------------------- norm and rotation
def rope_fwd(lib, **over):
    a = dict(x=FAKE, dtype=0, rows=4, heads=2, d=64, xr=128, xh=64, w=FAKE, norm=1, eps=1e-6, pos=FAKE,
             turns=FAKE, rot=64, start=0, layout=0, amp=1.0, y=FAKE, yr=128, yh=64)
    a.update(over)
    return lib.csa_norm_rope_fwd(*a.values(), None)


def rope_bwd(lib, **over):
    a = dict(x=FAKE, dy=FAKE, dtype=0, rows=4, heads=2, d=64, xr=128, xh=64, gr=128, gh=64, w=FAKE, norm=1,
             eps=1e-6, pos=FAKE, turns=FAKE, rot=64, start=0, layout=0, amp=1.0, dx=FAKE, dr=128, dh=64,
             dw=FAKE, acc=0, ws=FAKE, nb=1 << 20)
    a.update(over)
    return lib.csa_norm_rope_bwd(*a.values(), None)


ROPE_BOTH = [
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(d=0), INVALID), (dict(norm=2), INVALID),
    (dict(rot=63), INVALID), (dict(rot=-2), INVALID), (dict(rot=66), INVALID), (dict(start=2), INVALID),
    (dict(start=-1, rot=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(xr=-1), INVALID), (dict(xh=-64), INVALID),
    (dict(pos=None), INVALID), (dict(turns=None), INVALID), (dict(x=None), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(x=FAKE + 2, dtype=2), INVALID), (dict(w=FAKE + 2), INVALID),
    (dict(pos=FAKE + 2), INVALID), (dict(turns=FAKE + 4), INVALID),
    (dict(d=1025), UNSUPPORTED), (dict(rows=1 << 31, heads=1), UNSUPPORTED),
    (dict(rows=1 << 26, heads=64), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(layout=2), UNSUPPORTED),
]


@pytest.mark.parametrize("over,code", ROPE_BOTH + [
    (dict(norm=0), INVALID),  # a weight without a norm
    (dict(y=None), INVALID), (dict(y=FAKE + 1), INVALID), (dict(yr=-1), INVALID), (dict(yh=-1), INVALID),
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None, pos=None, turns=None), OK),
    # outputs whose elements would share a place
    (dict(yh=63), INVALID), (dict(yr=127), INVALID), (dict(yr=0), INVALID), (dict(yh=0), INVALID),
    (dict(yr=64, yh=255), INVALID), (dict(yr=1 << 62, yh=63), INVALID),
])
def test_rope_fwd_refusals(lib, over, code):
    assert rope_fwd(lib, **over) == code


@pytest.mark.parametrize("over,code", ROPE_BOTH + [
    (dict(norm=0, w=None), INVALID),  # a weight's gradient without a norm
    (dict(norm=0, dw=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID),
    (dict(dy=FAKE + 1), INVALID), (dict(dx=FAKE + 1), INVALID), (dict(dw=FAKE + 2), INVALID),
    (dict(ws=FAKE + 8), INVALID), (dict(gr=-1), INVALID), (dict(gh=-1), INVALID), (dict(dr=-1), INVALID),
    (dict(dh=-1), INVALID), (dict(ws=None), WORKSPACE), (dict(nb=255), WORKSPACE),
    (dict(rows=0, dw=None), OK), (dict(rows=0, acc=1), OK),
    (dict(dh=63), INVALID), (dict(dr=127), INVALID), (dict(dr=0), INVALID), (dict(dr=64, dh=255), INVALID),
])
def test_rope_bwd_refusals(lib, over, code):
    assert rope_bwd(lib, **over) == code


def test_rope_workspace_query_refuses(lib):
    for bad in ((-1, 1, 64), (4, 0, 64), (4, 1, 0), (4, 1, 1025), (1 << 30, 4, 64)):
        assert gp.csa_norm_rope_bwd_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------------------------ cache
def cache_write(lib, **over):
    a = dict(x=FAKE, dtype=0, rows=4, heads=2, d=64, xr=128, xh=64, slots=FAKE, n=16, fmt=1, data=FAKE,
             scales=FAKE, err=None)
    a.update(over)
    return lib.csa_cache_write(*a.values(), None)


def cache_read(lib, **over):
    a = dict(data=FAKE, scales=FAKE, fmt=1, slots=FAKE, rows=4, n=16, heads=2, d=64, x=FAKE, dtype=0, xr=128,
             xh=64, err=None)
    a.update(over)
    return lib.csa_cache_read(*a.values(), None)


@pytest.mark.parametrize("call", [cache_write, cache_read])
@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), INVALID), (dict(heads=0), INVALID), (dict(d=0), INVALID), (dict(n=-1), INVALID),
    (dict(xr=-1), INVALID), (dict(xh=-1), INVALID), (dict(x=None), INVALID), (dict(slots=None), INVALID),
    (dict(data=None), INVALID), (dict(scales=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(x=FAKE + 2, dtype=2), INVALID), (dict(slots=FAKE + 4), INVALID), (dict(err=FAKE + 2), INVALID),
    (dict(data=FAKE + 1, fmt=0), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED),
    (dict(fmt=-1), UNSUPPORTED), (dict(d=48), UNSUPPORTED), (dict(d=80, fmt=2), UNSUPPORTED),
    (dict(n=1 << 62), UNSUPPORTED), (dict(rows=1 << 62), UNSUPPORTED), (dict(heads=1 << 30), UNSUPPORTED),
    (dict(rows=0), OK),
])
def test_cache_refusals(lib, call, over, code):
    assert call(lib, **over) == code


@pytest.mark.parametrize("over", [dict(xh=63), dict(xr=127), dict(xr=0), dict(xh=0), dict(xr=64, xh=255)])
def test_cache_read_refuses_overlapping_rows(lib, over):
    assert cache_read(lib, **over) == INVALID


# -------------------------------------------------------------------------------- attention
def attn(lib, **over):
    a = dict(q=FAKE, qr=128, qh=64, cu=FAKE, S=2, tokens=4, H=2, kv=1, d=64, data=FAKE, scales=FAKE, fmt=1,
             table=FAKE, max_pages=4, num_pages=8, page=16, entries=FAKE, first=FAKE, ratio=4, scale=0.125,
             sink=FAKE, out=FAKE, outr=128, outh=64, lse=FAKE, ws=FAKE, nb=1 << 30, err=None)
    a.update(over)
    return lib.csa_cache_attn(*a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(S=-1), INVALID), (dict(tokens=-1), INVALID), (dict(H=0), INVALID), (dict(kv=0), INVALID),
    (dict(H=3, kv=2), INVALID), (dict(d=0), INVALID), (dict(max_pages=-1), INVALID),
    (dict(num_pages=-1), INVALID), (dict(page=0), INVALID), (dict(ratio=-1), INVALID), (dict(qr=-1), INVALID),
    (dict(qh=-1), INVALID), (dict(outr=-1), INVALID), (dict(outh=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(cu=None), INVALID),
    (dict(entries=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(table=None), INVALID), (dict(data=None), INVALID), (dict(scales=None), INVALID),
    (dict(q=FAKE + 1), INVALID), (dict(out=FAKE + 1), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(table=FAKE + 2), INVALID), (dict(entries=FAKE + 2), INVALID), (dict(first=FAKE + 2), INVALID),
    (dict(sink=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(err=FAKE + 2), INVALID),
    (dict(ws=FAKE + 8), INVALID), (dict(data=FAKE + 1, fmt=0), INVALID), (dict(d=1025, fmt=0), UNSUPPORTED),
    (dict(d=72), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(S=20000), UNSUPPORTED),
    (dict(tokens=1 << 30), UNSUPPORTED), (dict(max_pages=1 << 30), UNSUPPORTED),
    (dict(num_pages=1 << 60), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nb=8), WORKSPACE),
    (dict(S=0), OK), (dict(tokens=0), OK), (dict(tokens=0, q=None, out=None), OK),
    (dict(outh=63), INVALID), (dict(outr=127), INVALID), (dict(outr=0), INVALID), (dict(outr=64, outh=255), INVALID),
])
def test_attn_refusals(lib, over, code):
    assert attn(lib, **over) == code


@pytest.mark.parametrize("tokens", [(1 << 31) - 1, (1 << 31) - 128, (1 << 31) - 256])
def test_attn_row_numbers_stay_in_32_bits(lib, tokens):
    """A unit's rows are numbered up to its end, 64 or 128 rows on from its first."""
    assert attn(lib, tokens=tokens, H=1, kv=1) == UNSUPPORTED
    assert gp.csa_cache_attn_workspace_bytes(2, tokens, 1, 1, 64, 64) == 0


def test_attn_workspace_query_refuses(lib):
    for bad in ((-1, 1, 1, 1, 64, 16), (1, -1, 1, 1, 64, 16), (1, 1, 3, 2, 64, 16), (1, 1, 1, 1, 0, 16),
                (1, 1, 1, 1, 1025, 16), (1, 1, 1, 1, 64, -1), (1, 1 << 30, 4, 1, 64, 16)):
        assert gp.csa_cache_attn_workspace_bytes(*bad) == 0


# ------------------------------------------------------------- the reference checks itself
@pytest.mark.parametrize("fmt", [R.E4M3, R.FP4])
def test_reference_codes_round_trip(fmt):
    table = R.code_values(fmt)
    finite = table[torch.isfinite(table)]
    x = torch.cat([finite, torch.zeros(-len(finite) % 32, dtype=torch.float64)]).reshape(1, -1)
    x[0, 0::32] = R.MOST[fmt]  # every group at scale one
    codes, k = R.quantise(x, fmt)
    assert (k == 127).all() and torch.equal(R.dequantise(codes, k, fmt), x)
    assert torch.equal(R.unpack(R.pack(codes, fmt), fmt), codes)


def test_reference_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(3, 2, 12, generator=g, dtype=torch.float64) for _ in range(2))
    w = 1 + 0.1 * torch.randn(12, generator=g, dtype=torch.float64)
    ang = torch.randn(3, 4, generator=g, dtype=torch.float64)
    args = (1, 1e-3, ang, 8, 2, 1, 1.25)

    def loss(x, w):
        return (R.norm_rope(x, w, *args)[0] * dy).sum()

    dx, _, dw, _ = R.norm_rope_bwd(x, dy, w, *args)
    h = 2.0 ** -20  # central differences: h^2 of truncation, 2^-53 / h of rounding, both below 1e-8
    for t, grad in ((x, dx), (w, dw)):
        for i in range(0, t.numel(), 5):
            up, down = t.clone(), t.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            pair = ((up, w), (down, w)) if t is x else ((x, up), (x, down))
            slope = (loss(*pair[0]) - loss(*pair[1])) / (2 * h)
            assert abs(slope - grad.view(-1)[i]) < 1e-7
