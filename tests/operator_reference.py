"""Plain 64-bit forms of the head norm with rotation, the cache formats and the attention over
the cache, written from their formulas, and the error bounds that fp32 kernels keep to.

U is half a step of fp32 (2^-24); HALF[dtype] half a step of each type, relative to the value.
"""
import math

import torch

U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]  # in the order of CSA_DTYPE_*
HALF = {t: torch.finfo(t).eps / 2 for t in DTYPES}
TINY = {t: torch.finfo(t).smallest_normal * HALF[t] for t in DTYPES}  # half a step below the normals
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BF16, E4M3, FP4 = 0, 1, 2
MOST = {E4M3: 448.0, FP4: 6.0}


# ------------------------------------------------------------------------ norm and rotation
def frequencies(rot, base=10000.0, scaling=0, factor=1.0, length=4096.0, fast=32.0, slow=1.0):
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == 1:
        return [v / factor for v in f], 1.0
    if scaling == 2:
        def at(b):
            return rot * math.log(length / (2 * math.pi * b)) / (2 * math.log(base))
        lo = min(max(math.floor(at(fast)), 0), rot - 1)
        hi = min(max(math.ceil(at(slow)), 0), rot - 1)
        out = []
        for i, v in enumerate(f):
            m = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            out.append(v / factor * m + v * (1 - m))
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def angles(pos, turns):
    """[rows, pairs] in radians, from the integers the entry points take: exact modulo a turn."""
    rows = [[((int(p) * (int(t) % (1 << 64))) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for t in turns]
            for p in pos]
    return torch.tensor(rows, dtype=torch.float64).reshape(len(pos), len(turns))


def pair_columns(rot, start, layout):
    i = torch.arange(rot // 2)
    a = start + (2 * i if layout else i)
    return a, a + (1 if layout else rot // 2)


def rotate(n, ang, rot, start, layout, amp, back=False):
    """n [rows, heads, d] turned (back: the transpose), and |a| + |b| of each column's pair."""
    a, b = pair_columns(rot, start, layout)
    c, s = (f(ang)[:, None] * amp for f in (torch.cos, torch.sin))
    if back:
        s = -s
    y, mass = n.clone(), n.abs()
    y[..., a], y[..., b] = n[..., a] * c - n[..., b] * s, n[..., a] * s + n[..., b] * c
    both = (n[..., a].abs() + n[..., b].abs()) * abs(amp)
    mass[..., a], mass[..., b] = both, both
    return y, mass


def norm_rope(x, weight, norm, eps, ang, rot, start, layout, amp):
    x = x.double()
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    return rotate(x, ang, rot, start, layout, amp)


def norm_rope_bwd(x, dy, weight, norm, eps, ang, rot, start, layout, amp):
    """(dx, its mass, dweight, its mass) for the rows given."""
    g, gm = rotate(dy.double(), ang, rot, start, layout, amp, back=True)
    if not norm:
        return g, gm, None, None
    x = x.double()
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    dx = r * (w * g - x * r * r * (w * g * x).mean(-1, keepdim=True))
    mass = r * ((w * gm).abs() + x.abs() * r * r * (w * gm * x).abs().mean(-1, keepdim=True))
    return dx, mass, (g * x * r).sum((0, 1)), (gm * (x * r).abs()).sum((0, 1))


def rope_bound(d, dtype):
    """Error of a value in fp32 against its mass (the magnitudes it is made of).

    A sum of d terms, at most d/8 of them one after another in a lane (2 roundings each with
    the product) and then 5 joins: (d/8 + 6) U. Forward the root halves it and adds the
    quotient, root, weight and rotation products: 8 U more. Backward r enters three times and
    the dot product is another such sum: three times that all in all. cos and sin of an angle
    that is exact to 2^-25 half turns (9.4e-8): within 3e-7 as CUDA's sincospif (2 steps), and
    within 1e-6 for the 16-bit types; they enter twice backward (dn, and dn in the dot)."""
    turn = 3e-7 if dtype == torch.float32 else 1e-6
    return 3 * ((d / 8 + 6) * U + 8 * U) + 2 * turn


def close(got, ref, mass, d, dtype, what):
    got = got.double().cpu()
    k = rope_bound(d, dtype)
    bound = HALF[dtype] * ref.abs() + (1 + HALF[dtype]) * k * mass + TINY[dtype]
    off = (got - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound.clamp(min=1e-300)).nan_to_num(9e9).max()))


# ------------------------------------------------------------------------------- cache codes
def code_values(fmt):
    """Value of every code, by code."""
    if fmt == E4M3:
        out = []
        for c in range(256):
            e, m = (c >> 3) & 15, c & 7
            v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
            out.append((-v if c & 128 else v) if c & 127 != 127 else math.nan)
        return torch.tensor(out, dtype=torch.float64)
    return torch.cat([E2M1, -E2M1])


def quantise(x, fmt):
    """x [..., d] (double) -> (codes [..., d] int64, scale bytes [..., d/32]), code by code."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = g.abs().amax(-1)
    k = torch.zeros(top.shape, dtype=torch.int64)
    for byte in range(1, 255):  # the smallest byte whose scale reaches the largest magnitude
        k = torch.where(top > MOST[fmt] * 2.0 ** (byte - 1 - 127), byte, k)
    bad = ~torch.isfinite(g).all(-1)
    k = torch.where(bad, 255, k)
    v = torch.where(bad[..., None], 0.0, g * torch.exp2(127.0 - k.double())[..., None])
    table = code_values(fmt)[:127 if fmt == E4M3 else 8]
    a = v.abs()
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    sign = torch.signbit(v).long() * (128 if fmt == E4M3 else 8)
    return (code + sign).reshape(x.shape), k


def dequantise(codes, k, fmt):
    v = code_values(fmt)[codes]
    s = torch.where(k == 255, math.nan, torch.exp2(k.double() - 127.0))
    return v * s.repeat_interleave(32, -1)


def pack(codes, fmt):
    if fmt == E4M3:
        return codes.to(torch.uint8)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def unpack(data, fmt):
    if fmt == E4M3:
        return data.long()
    return torch.stack([data.long() & 15, data.long() >> 4], -1).flatten(-2)


# --------------------------------------------------------------------------------- attention
def seen(pos, ratio, n):
    return n if ratio == 0 else max(0, min(n, (pos + 1) // ratio))


def attend(q, cu, values, table, page_size, entries, first, ratio, scale, sink):
    """out, lse, and the bounds of each, in 64 bits: a loop over tokens and cache heads.

    values [slots, kv_heads, d]: what the cache stands for. Bounds: a score is a sum of d
    products in fp32 (2 d U of their magnitudes, whatever the order, rounding or truncation),
    which every weight takes twice (its own and the denominator's); exp2 of an fp32 argument
    within 2^-22 and U of the argument's size; the denominator's sum, n U. The weights are
    rounded to 16 bits (2^-8), so is the output."""
    T, H, d = q.shape
    kv = values.shape[1]
    G = H // kv
    out = torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    if sink is not None:
        lse[:] = sink.double()
    for s in range(len(cu) - 1):
        n_all = int(entries[s])
        e = torch.arange(n_all)
        slots = table[s].long()[e // page_size] * page_size + e % page_size
        k_all = values[slots] if n_all else values[:0]
        for t in range(int(cu[s]), int(cu[s + 1])):
            pos = (0 if first is None else int(first[s])) + t - int(cu[s])
            n = seen(pos, ratio, n_all)
            for h in range(kv if n else 0):
                hs = slice(h * G, (h + 1) * G)
                qv, k = q[t, hs].double(), k_all[:n, h]
                x = qv @ k.T * scale
                ds = float((qv.abs() @ k.abs().T * abs(scale)).max()) * 2 * d * U
                every = x if sink is None else torch.cat([x, sink[hs, None].double()], 1)
                z = torch.logsumexp(every, -1)
                w = torch.exp(x - z[:, None])
                out[t, hs], lse[t, hs] = w @ k, z
                rel = 2 * ds + 2 * float(every.abs().max()) * 4 * U + 2.0 ** -21 + n * U
                half = 2.0 ** -8
                tol[t, hs] = (half + rel) * (1 + half) * (w @ k.abs()) + half * (w @ k).abs() + TINY[torch.bfloat16]
                ltol[t, hs] = rel + 4 * U * z.abs()
    return out, lse, tol, ltol
