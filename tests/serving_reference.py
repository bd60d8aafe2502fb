"""Plain 64-bit forms of a serving step's operators, written from their formulas: entries of a stream of
tokens and the state that a later call reads, and rows normed, turned and put into cache codes."""
import math

import torch

from tests import operator_reference as R

U, TINY = R.U, R.TINY[torch.bfloat16]
NAN16 = 0x7FFF


def window_entry(kv, score, ape, block, ratio, coff, d):
    """The entry of a block of one sequence, whose tokens so far are kv, score [tokens, coff * d]: (value, bound).

    Bound in fp32: an exponent's argument t = score log2e + ape log2e - max takes two roundings of each
    product, one of the sum and one of the difference, 4 U (|x| + |max|) in all; exp2 is within 2^-22 = 4 U. The
    sums: 8 positions in a thread, a merge of two roundings, two exp2 and products for every 8 positions
    more than 256 share (at most 8 times), 32 parts. A weight's error enters with kv - out, the sums' with kv,
    in numerator and denominator alike."""
    lo = max(0, block - (coff - 1)) * ratio
    own = block * ratio
    k, x = [], []
    for p in range(lo, own + ratio):
        half = 0 if coff == 1 or p < own else 1
        cols = slice(half * d, half * d + d)
        k.append(kv[p, cols].double())
        x.append(score[p, cols].double() + ape[p % ratio, cols].double())
    k, x = torch.stack(k), torch.stack(x)
    top = x.amax(0)
    e = torch.exp(x - top)
    w = e / e.sum(0)
    out = (w * k).sum(0)
    args = torch.where(torch.isfinite(x), x.abs(), 0.0) + top.abs()
    sums = min(len(k), 8) + 10 * math.ceil(len(k) / 256) + min(32, math.ceil(len(k) / 8))
    terms = torch.where(w > 0, w, 0.0)
    mass = U * ((2 * sums + 16) * (terms * k.abs()).sum(0) + 8 * (terms * (k - out).abs() * (args + 1)).sum(0))
    half = 2.0 ** -8
    return out, half * out.abs() + (1 + half) * mass + TINY


def held(first, n, ratio, coff, d):
    """Which elements of a state, as [ratio * coff, coff * d] (position or -1), a sequence holds after n more tokens."""
    W, done = ratio * coff, (first + n) // ratio
    at = torch.full((W, coff * d), -1, dtype=torch.int64)
    for half in range(coff):
        keep = max(0, done - (coff - 1 - half)) * ratio
        for p in range(keep, first + n):
            at[p % W, half * d:half * d + d] = p
    return at


def append_values(x, weight, norm, eps, ang, rot, start, layout, amp):
    """The finished rows in 64 bits and how far fp32 arithmetic may be off (angles as for fp32 results)."""
    n, mass = R.norm_rope(x, weight, norm, eps, ang, rot, start, layout, amp)
    return n, R.rope_bound(x.shape[-1], torch.float32) * mass


def check_codes(codes, scales, fmt, value, off):
    """Codes and scale bytes [..., d], [..., d/32] against the values that they stand for: a scale is the
    smallest that reaches the group's largest magnitude, as known to `off`, and each code the nearest one."""
    g, o = (t.reshape(*t.shape[:-1], t.shape[-1] // 32, 32) for t in (value.abs(), off))
    low, high = (g - o).clamp(min=0).amax(-1), (g + o).amax(-1)
    k = scales.double()
    most = R.MOST[fmt] * torch.exp2(k - 127.0)
    assert (most >= low).all() and ((k == 0) | (most / 2 < high)).all()
    s = torch.exp2(k - 127.0).repeat_interleave(32, -1)
    got = R.dequantise(codes, scales.long(), fmt)
    # half a step of the code nearest to the value: 2^-4 or 2^-2 of it, or of the smallest normal code
    part, least = (2.0 ** -4, 2.0 ** -10) if fmt == R.E4M3 else (2.0 ** -2, 0.25)
    bound = torch.maximum((value.abs() + off) * part, s * least) + off
    assert ((got - value).abs() <= bound).all(), float(((got - value).abs() / bound).max())
