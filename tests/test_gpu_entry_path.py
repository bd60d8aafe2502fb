"""The entry path as a user runs it: packs are pooled, the pooled entries normed and turned to their
positions, written into the paged cache in each of its formats, and new tokens' queries, normed and
turned too, attend to them; all on one stream without a wait. Each step is checked against 64-bit
arithmetic on what the step before it left, so that every tolerance is that step's own.
Training: the pooled entries' gradient goes back through the norm and the pooling."""
import numpy as np
import pytest
import torch

import oracle
import thd_synth as ts
from tests import gpu_harness as H
from tests import operator_reference as R
from tests.parity import compare_bf16, compare_dape

pytestmark = pytest.mark.gpu


def pooled_positions(gp, pack, dev, rows):
    """Position of each pooled row's block in its sequence, from the device's own index map: the
    block's first token, and -1 for rows behind the last block."""
    m = torch.empty(rows, 3, dtype=torch.int32, device="cuda")
    gp.csa_compressor_map_blocks(dev["cu_seqlens"], pack.S, pack.ratio, pack.capacity, rows, m)
    return torch.where(m[:, 1] < 0, -1, m[:, 1] * pack.ratio).to(torch.int32).contiguous(), m


@pytest.mark.parametrize("fmt", [R.BF16, R.E4M3, R.FP4])
@pytest.mark.parametrize("d,heads,ratio,coff", [(512, 64, 4, 2), (128, 16, 4, 2), (128, 8, 2, 1)])
def test_pool_norm_write_attend(cuda_lib, fmt, d, heads, ratio, coff):
    gp = cuda_lib
    pack = ts.make_custom([700, 3, 0, 301], ratio=ratio, coff=coff, d=d, pad_rows=5, seed=31)
    dev = H.device_pack(pack)
    total, rows, page, rot = pack.total_comp, pack.total_comp + 7, 64, min(64, d)
    g = torch.Generator().manual_seed(7)
    w, wq = 1 + 0.1 * torch.randn(d, generator=g), 1 + 0.1 * torch.randn(d, generator=g)
    turns, amp = gp.csa_rope_table(rot, 10000.0, gp.CSA_ROPE_YARN, 16.0, 4096.0)
    dw, dwq, dturns = w.cuda(), wq.cuda(), turns.cuda()
    lens = np.diff(pack.cu_seqlens)
    counts = [int(n) // ratio for n in lens]
    # pages in a shuffled order, and each pooled row's slot
    max_pages = max(1, -(-max(counts) // page))
    pages = [-(-c // page) for c in counts]
    order = torch.randperm(sum(pages) + 2, generator=g)
    table = torch.full((pack.S, max_pages), -1, dtype=torch.int32)
    slots, at = [], 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n].to(torch.int32)
        at += n
        slots += [int(table[s, e // page]) * page + e % page for e in range(counts[s])]
    slots = torch.tensor(slots + [-1] * (rows - total))
    num = (sum(pages) + 2) * page
    data = torch.zeros(num, 1, {R.BF16: 2 * d, R.E4M3: d, R.FP4: d // 2}[fmt], dtype=torch.uint8, device="cuda")
    scales = None if fmt == R.BF16 else torch.zeros(num, 1, d // 32, dtype=torch.uint8, device="cuda")
    # the sequences' last tokens ask: 9 and 1 and 2 of them, the third sequence is empty
    new = [9, 1, 0, 2]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    first = [max(0, int(n) - k) for n, k in zip(lens, new)]
    T = int(cu[-1])
    q0 = torch.randn(T, heads, d, generator=g).to(torch.bfloat16)
    qpos = torch.cat([torch.arange(f, f + k) for f, k in zip(first, new)]).to(torch.int32)
    i32 = dict(dtype=torch.int32, device="cuda")
    # --- everything on the stream
    pooled = torch.full((rows, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, **i32)
    dq, dqpos, dslots, dtable = q0.cuda(), qpos.cuda(), slots.cuda(), table.cuda()
    dcu, dcounts, dfirst = torch.tensor(cu, **i32), torch.tensor(counts, **i32), torch.tensor(first, **i32)
    entries, q = torch.empty_like(pooled), torch.empty_like(dq)
    out = torch.empty(T, heads, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, heads, device="cuda")
    n = gp.csa_cache_attn_workspace_bytes(pack.S, T, heads, 1, d, max_pages * page)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    gp.csa_compressor_fwd(dev["kv"], dev["score"], dev["ape"], dev["cu_seqlens"], pack.S, ratio, coff, d, pack.capacity,
                          pooled, rows, err)
    pos, _ = pooled_positions(gp, pack, dev, rows)
    gp.csa_norm_rope_fwd(pooled, 0, rows, 1, d, d, d, dw, 1, 1e-6, pos, dturns, rot, d - rot, 1, amp, entries, d, d)
    gp.csa_cache_write(entries, 0, rows, 1, d, d, d, dslots, num, fmt, data, scales, err)
    gp.csa_norm_rope_fwd(dq, 0, T, heads, d, heads * d, d, dwq, 1, 1e-6, dqpos, dturns, rot, d - rot, 1, amp, q, heads * d, d)
    gp.csa_cache_attn(q, heads * d, d, dcu, pack.S, T, heads, 1, d, data, scales, fmt, dtable, max_pages, num // page, page,
                      dcounts, dfirst, ratio, d ** -0.5, None, out, heads * d, d, lse, ws, n, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    # --- step by step
    ref = oracle.fwd_pack(pack, want_f64=True, want_err=True)
    rep = compare_bf16("pooled", ts.bf16_tensor_bits(pooled[:total, 0].contiguous()), ref["out"], ref["out_f64"], ref["out_err"])
    assert rep.fail == 0, str(rep)
    live = pos.cpu() >= 0
    assert int(live.sum()) == total
    where = torch.cat([torch.arange(c) * ratio for c in counts])
    assert torch.equal(pos.cpu()[live].long(), where)
    y, mass = R.norm_rope(pooled.cpu()[:total], w, 1, 1e-6, R.angles(where, turns), rot, d - rot, 1, amp)
    R.close(entries[:total], y, mass, d, torch.bfloat16, "entries")
    held = entries.cpu()[:total]
    if fmt == R.BF16:
        values = data.cpu().view(torch.bfloat16).double()
        assert torch.equal(data.cpu()[slots[:total]].view(torch.bfloat16), held)
    else:
        codes, k = R.quantise(held.double(), fmt)
        assert torch.equal(R.unpack(data.cpu()[slots[:total]], fmt), codes) and torch.equal(scales.cpu()[slots[:total]].long(), k)
        values = R.dequantise(R.unpack(data.cpu(), fmt), scales.cpu().long(), fmt)
    y, mass = R.norm_rope(q0, wq, 1, 1e-6, R.angles(qpos, turns), rot, d - rot, 1, amp)
    R.close(q, y, mass, d, torch.bfloat16, "queries")
    want, wl, tol, ltol = R.attend(q.cpu(), cu, values, table, page, counts, first, ratio, d ** -0.5, None)
    assert ((out.double().cpu() - want).abs() <= tol).all()
    fine = torch.isfinite(wl)
    assert torch.equal(lse.cpu()[~fine].double(), wl[~fine]) and ((lse.double().cpu() - wl).abs()[fine] <= ltol[fine]).all()


@pytest.mark.parametrize("d,ratio,coff", [(512, 4, 2), (64, 2, 1)])
def test_gradients_through_norm_and_pooling(cuda_lib, d, ratio, coff):
    """The entries' gradient back through norm and rotation into the pooling's backward: the padded
    rows behind the last block take no part in either."""
    gp = cuda_lib
    pack = ts.make_custom([130, 5, 77], ratio=ratio, coff=coff, d=d, pad_rows=3, seed=33)
    dev = H.device_pack(pack)
    total, rows, rot = pack.total_comp, pack.total_comp + 4, 64 if d == 512 else 32
    g = torch.Generator().manual_seed(8)
    w = 1 + 0.1 * torch.randn(d, generator=g)
    turns, amp = gp.csa_rope_table(rot)
    pooled = torch.full((rows, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    gp.csa_compressor_fwd(dev["kv"], dev["score"], dev["ape"], dev["cu_seqlens"], pack.S, ratio, coff, d, pack.capacity,
                          pooled, rows)
    pos, _ = pooled_positions(gp, pack, dev, rows)
    dy = torch.randn(rows, 1, d, generator=g).to(torch.bfloat16).cuda()
    dpooled = torch.full((rows, 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(d, device="cuda")
    ws = torch.empty(gp.csa_norm_rope_bwd_workspace_bytes(rows, 1, d), dtype=torch.uint8, device="cuda")
    gp.csa_norm_rope_bwd(pooled, dy, 0, rows, 1, d, d, d, d, d, w.cuda(), 1, 1e-6, pos, turns.cuda(), rot, 0, 0, amp, dpooled,
                         d, d, dw, 0, ws, ws.numel())
    got = H.run_bwd(gp, pack, dev, out_rows=rows, dout=dpooled.view(rows, d))
    assert got[3] == 0
    where = pos.cpu()[:total]
    dx, mass, rw, mw = R.norm_rope_bwd(pooled.cpu()[:total], dy.cpu()[:total], w, 1, 1e-6, R.angles(where, turns), rot, 0, 0, amp)
    R.close(dpooled[:total], dx, mass, d, torch.bfloat16, "dpooled")
    assert ((dw.double().cpu() - rw).abs() <= (R.rope_bound(d, torch.bfloat16) + 70 * R.U) * mw).all()
    assert torch.isnan(dpooled[total:].float()).all()  # left as they were, and not read
    dout = ts.bf16_tensor_bits(dpooled[:total, 0].contiguous())
    ref = oracle.bwd(pack.kv, pack.score, pack.ape, pack.cu_seqlens, dout, ratio, coff, d, pack.capacity, want_f64=True,
                     want_err=True)
    for r in (compare_bf16("dkv", got[0], ref["dkv"], ref["dkv_f64"], ref["dkv_err"]),
              compare_bf16("dscore", got[1], ref["dscore"], ref["dscore_f64"], ref["dscore_err"]),
              compare_dape(got[2], ref["dape_f64"], ref["dape_err"])):
        assert r.fail == 0, str(r)
