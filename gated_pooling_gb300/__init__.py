"""GB300 (sm_103a) CSA/HCA KV-compressor gated-softmax pooling over THD packs.

A thin ctypes binding of the C ABI in ``include/csa_compressor.h``: the functions
below have the C names and arguments, and only marshal them (tensor -> device
pointer, stream -> cudaStream_t). Every step of the pooling runs in the library's
CUDA kernels. There is no fallback: if the library is missing, loading raises.

Tensors are torch CUDA tensors (bf16 for kv/score/dout/out/dkv/dscore and the KPool
key/gate, fp32 for ape/dape, int32 for cu_seqlens, lead and the error word); PyTorch
only provides device memory and streams.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import build as _build

LIB_PATH = _build.LIB
_lib: Optional[ctypes.CDLL] = None

CSA_OK, CSA_ERR_INVALID_VALUE, CSA_ERR_UNSUPPORTED, CSA_ERR_WORKSPACE, CSA_ERR_CUDA = 0, 1, 2, 3, 4
CSA_DEVERR_CU_SEQLENS, CSA_DEVERR_OUT_ROWS, CSA_DEVERR_TIMEOUT, CSA_DEVERR_LEAD = 1, 2, 3, 4
CSA_DEVERR_SLOT, CSA_DEVERR_ENTRIES, CSA_DEVERR_PAGE = 5, 6, 7
CSA_DTYPE_BF16, CSA_DTYPE_FP16, CSA_DTYPE_FP32 = 0, 1, 2
CSA_ROPE_PLAIN, CSA_ROPE_LINEAR, CSA_ROPE_YARN = 0, 1, 2
CSA_ROPE_HALF, CSA_ROPE_INTERLEAVED = 0, 1
CSA_CACHE_BF16, CSA_CACHE_E4M3, CSA_CACHE_E2M1 = 0, 1, 2
CSA_MAX_HEAD_DIM, CSA_CACHE_GROUP = 1024, 32
CSA_TEST_MIN_WAIT_CYCLES = 1000000
CSA_KPOOL_MAX_POOL = 1024
EXPORTED = ("csa_status_string", "csa_last_error_string", "csa_compressor_total_comp", "csa_compressor_fwd",
            "csa_compressor_bwd_workspace_bytes", "csa_compressor_bwd",
            "csa_compressor_bwd_noalloc", "csa_compressor_test_hooks",
            "csa_compressor_map_blocks", "csa_kpool_total", "csa_kpool_fwd", "csa_rope_table",
            "csa_norm_rope_fwd", "csa_norm_rope_bwd_workspace_bytes", "csa_norm_rope_bwd",
            "csa_cache_write", "csa_cache_read", "csa_cache_attn_workspace_bytes", "csa_cache_attn")


class CsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Loads the CUDA library (building it first only if ``path`` is None and it is
    missing or stale). Raises if it cannot be loaded."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    if path is None:
        if not _build.up_to_date():
            _build.build()
        path = LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not found at {path}; run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.csa_status_string.restype = ctypes.c_char_p
    lib.csa_status_string.argtypes = [ctypes.c_int]
    lib.csa_last_error_string.restype = ctypes.c_char_p
    lib.csa_last_error_string.argtypes = []
    lib.csa_compressor_total_comp.restype = i64
    lib.csa_compressor_total_comp.argtypes = [vp, i32, i32]
    lib.csa_compressor_fwd.restype = ctypes.c_int
    lib.csa_compressor_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i64, vp, i64, vp, vp]
    lib.csa_compressor_bwd_workspace_bytes.restype = sz
    lib.csa_compressor_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i64]
    lib.csa_compressor_bwd.restype = ctypes.c_int
    lib.csa_compressor_bwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64, vp, vp,
                                       vp, i32, vp, sz, vp, vp]
    lib.csa_compressor_bwd_noalloc.restype = ctypes.c_int
    lib.csa_compressor_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i64, i64,
                                               vp, vp, vp, i32, vp, vp]
    lib.csa_compressor_test_hooks.restype = ctypes.c_int
    lib.csa_compressor_test_hooks.argtypes = [i64, i32]
    lib.csa_compressor_map_blocks.restype = ctypes.c_int
    lib.csa_compressor_map_blocks.argtypes = [vp, i32, i32, i64, i64, vp, vp, vp]
    lib.csa_kpool_total.restype = i64
    lib.csa_kpool_total.argtypes = [vp, vp, i32, i32]
    lib.csa_kpool_fwd.restype = ctypes.c_int
    lib.csa_kpool_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i64, vp, i64, i32, vp, vp]
    f32, f64 = ctypes.c_float, ctypes.c_double
    lib.csa_rope_table.restype = ctypes.c_int
    lib.csa_rope_table.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    lib.csa_norm_rope_fwd.restype = ctypes.c_int
    lib.csa_norm_rope_fwd.argtypes = [vp, i32, i64, i32, i32, i64, i64, vp, i32, f32, vp, vp, i32,
                                      i32, i32, f32, vp, i64, i64, vp]
    lib.csa_norm_rope_bwd_workspace_bytes.restype = sz
    lib.csa_norm_rope_bwd_workspace_bytes.argtypes = [i64, i32, i32]
    lib.csa_norm_rope_bwd.restype = ctypes.c_int
    lib.csa_norm_rope_bwd.argtypes = [vp, vp, i32, i64, i32, i32, i64, i64, i64, i64, vp, i32, f32,
                                      vp, vp, i32, i32, i32, f32, vp, i64, i64, vp, i32, vp, sz, vp]
    lib.csa_cache_write.restype = ctypes.c_int
    lib.csa_cache_write.argtypes = [vp, i32, i64, i32, i32, i64, i64, vp, i64, i32, vp, vp, vp, vp]
    lib.csa_cache_read.restype = ctypes.c_int
    lib.csa_cache_read.argtypes = [vp, vp, i32, vp, i64, i64, i32, i32, vp, i32, i64, i64, vp, vp]
    lib.csa_cache_attn_workspace_bytes.restype = sz
    lib.csa_cache_attn_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i64]
    lib.csa_cache_attn.restype = ctypes.c_int
    lib.csa_cache_attn.argtypes = [vp, i64, i64, vp, i32, i64, i32, i32, i32, vp, vp, i32, vp, i32,
                                   i64, i32, vp, vp, i32, f32, vp, vp, i64, i64, vp, vp, sz, vp, vp]
    if path == LIB_PATH:
        _lib = lib
    return lib


def _ptr(x) -> Optional[int]:
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_raw_stream = None


def _find_raw_stream():
    """The current stream's handle: torch's raw getter where it has one (0.1 us; making a Stream
    object for it takes 2.9 us, as long as the rest of a small call), else the public way."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if raw is not None and device is not None:
        torch.cuda.init()
        return lambda: raw(device())
    return lambda: torch.cuda.current_stream().cuda_stream


def _stream(stream) -> Optional[int]:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            _raw_stream = _find_raw_stream()
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str) -> None:
    if status:
        msg = load().csa_status_string(status).decode()
        if status == CSA_ERR_CUDA:
            msg += f" ({load().csa_last_error_string().decode()})"
        raise CsaError(status, f"{what}: {msg}")


def csa_status_string(status: int) -> str:
    return load().csa_status_string(status).decode()


def csa_last_error_string() -> str:
    return load().csa_last_error_string().decode()


def csa_compressor_total_comp(cu_seqlens_host, S: int, ratio: int) -> int:
    """``cu_seqlens_host``: a host int32 array (numpy, CPU tensor or ctypes pointer)."""
    import numpy as np
    if hasattr(cu_seqlens_host, "numpy"):
        cu_seqlens_host = cu_seqlens_host.numpy()
    arr = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    return int(load().csa_compressor_total_comp(arr.ctypes.data_as(ctypes.c_void_p), S, ratio))


def csa_compressor_fwd(kv, score, ape, cu_seqlens, S: int, ratio: int, coff: int, d: int,
                       capacity: int, out, out_rows: int, dev_error=None, stream=None) -> None:
    _check(load().csa_compressor_fwd(_ptr(kv), _ptr(score), _ptr(ape), _ptr(cu_seqlens), S,
                                     ratio, coff, d, capacity, _ptr(out), out_rows,
                                     _ptr(dev_error), _stream(stream)), "csa_compressor_fwd")


def csa_compressor_bwd_workspace_bytes(S: int, ratio: int, coff: int, d: int, capacity: int,
                                       out_rows: int) -> int:
    return int(load().csa_compressor_bwd_workspace_bytes(S, ratio, coff, d, capacity, out_rows))


def csa_compressor_bwd(kv, score, ape, cu_seqlens, dout, S: int, ratio: int, coff: int, d: int,
                       capacity: int, out_rows: int, dkv, dscore, dape, accumulate_dape: int,
                       workspace, workspace_bytes: int, dev_error=None, stream=None) -> None:
    _check(load().csa_compressor_bwd(_ptr(kv), _ptr(score), _ptr(ape), _ptr(cu_seqlens),
                                     _ptr(dout), S, ratio, coff, d, capacity, out_rows, _ptr(dkv),
                                     _ptr(dscore), _ptr(dape), int(accumulate_dape),
                                     _ptr(workspace), workspace_bytes, _ptr(dev_error),
                                     _stream(stream)), "csa_compressor_bwd")


def csa_compressor_bwd_noalloc(kv, score, ape, cu_seqlens, dout, S: int, ratio: int, coff: int,
                               d: int, capacity: int, out_rows: int, dkv, dscore, dape,
                               accumulate_dape: int, dev_error=None, stream=None) -> None:
    """Backward without a caller workspace, for callers that cannot allocate device
    memory; see include/csa_compressor.h for the shared scratch array's rules."""
    _check(load().csa_compressor_bwd_noalloc(_ptr(kv), _ptr(score), _ptr(ape), _ptr(cu_seqlens),
                                             _ptr(dout), S, ratio, coff, d, capacity, out_rows,
                                             _ptr(dkv), _ptr(dscore), _ptr(dape),
                                             int(accumulate_dape), _ptr(dev_error),
                                             _stream(stream)), "csa_compressor_bwd_noalloc")


def csa_compressor_test_hooks(wait_cycles: int, withhold_row: int) -> None:
    """Test hook: pipeline wait bound (0 = default) and the row whose copies the first
    CTA's producer withholds (-1 = off), for every later call."""
    _check(load().csa_compressor_test_hooks(int(wait_cycles), int(withhold_row)),
           "csa_compressor_test_hooks")


def csa_compressor_map_blocks(cu_seqlens, S: int, ratio: int, capacity: int, out_rows: int,
                              seg_blk_base, dev_error=None, stream=None) -> None:
    _check(load().csa_compressor_map_blocks(_ptr(cu_seqlens), S, ratio, capacity, out_rows,
                                            _ptr(seg_blk_base), _ptr(dev_error),
                                            _stream(stream)), "csa_compressor_map_blocks")


def csa_kpool_total(cu_seqlens_host, lead_host, S: int, pool: int) -> int:
    """Pool count from host int32 arrays (``lead_host`` may be None)."""
    import numpy as np
    def arr(x):
        if x is None:
            return None
        if hasattr(x, "numpy"):
            x = x.numpy()
        return np.ascontiguousarray(x, dtype=np.int32)
    cu, ld = arr(cu_seqlens_host), arr(lead_host)
    return int(load().csa_kpool_total(cu.ctypes.data_as(ctypes.c_void_p),
                                      None if ld is None else ld.ctypes.data_as(ctypes.c_void_p),
                                      S, pool))


def csa_kpool_fwd(key, gate, cu_seqlens, lead, S: int, pool: int, d: int, capacity: int, out,
                  out_rows: int, compress: int = 0, dev_error=None, stream=None) -> None:
    """KPool forward (the DSA indexer's key pooling); ``lead`` may be None."""
    _check(load().csa_kpool_fwd(_ptr(key), _ptr(gate), _ptr(cu_seqlens), _ptr(lead), S, pool, d,
                                capacity, _ptr(out), out_rows, int(compress), _ptr(dev_error),
                                _stream(stream)), "csa_kpool_fwd")



def csa_rope_table(rot_dim: int, base: float = 10000.0, scaling: int = CSA_ROPE_PLAIN,
                   factor: float = 1.0, original_length: float = 4096.0, beta_fast: float = 32.0,
                   beta_slow: float = 1.0):
    """``(turns, amplitude)``: a host int64 tensor [rot_dim / 2] holding the uint64 turns of
    each pair (move it to the GPU for the calls), and the amplitude to pass with it."""
    import torch
    turns = torch.zeros(max(rot_dim, 0) // 2, dtype=torch.int64)
    amplitude = ctypes.c_float(1.0)
    _check(load().csa_rope_table(rot_dim, base, scaling, factor, original_length, beta_fast,
                                 beta_slow, turns.data_ptr() or None, ctypes.byref(amplitude)),
           "csa_rope_table")
    return turns, amplitude.value


def csa_norm_rope_fwd(x, dtype: int, rows: int, heads: int, d: int, x_row_stride: int,
                      x_head_stride: int, weight, norm: int, eps: float, positions, turns,
                      rot_dim: int, rot_start: int, layout: int, amplitude: float, y,
                      y_row_stride: int, y_head_stride: int, stream=None) -> None:
    """Norm of every head and rotation to the row's position; strides in elements."""
    _check(load().csa_norm_rope_fwd(_ptr(x), dtype, rows, heads, d, x_row_stride, x_head_stride,
                                    _ptr(weight), int(norm), eps, _ptr(positions), _ptr(turns),
                                    rot_dim, rot_start, layout, amplitude, _ptr(y), y_row_stride,
                                    y_head_stride, _stream(stream)), "csa_norm_rope_fwd")


def csa_norm_rope_bwd_workspace_bytes(rows: int, heads: int, d: int) -> int:
    return int(load().csa_norm_rope_bwd_workspace_bytes(rows, heads, d))


def csa_norm_rope_bwd(x, dy, dtype: int, rows: int, heads: int, d: int, x_row_stride: int,
                      x_head_stride: int, dy_row_stride: int, dy_head_stride: int, weight,
                      norm: int, eps: float, positions, turns, rot_dim: int, rot_start: int,
                      layout: int, amplitude: float, dx, dx_row_stride: int, dx_head_stride: int,
                      dweight, accumulate_dweight: int, workspace, workspace_bytes: int,
                      stream=None) -> None:
    _check(load().csa_norm_rope_bwd(_ptr(x), _ptr(dy), dtype, rows, heads, d, x_row_stride,
                                    x_head_stride, dy_row_stride, dy_head_stride, _ptr(weight),
                                    int(norm), eps, _ptr(positions), _ptr(turns), rot_dim,
                                    rot_start, layout, amplitude, _ptr(dx), dx_row_stride,
                                    dx_head_stride, _ptr(dweight), int(accumulate_dweight),
                                    _ptr(workspace), workspace_bytes, _stream(stream)),
           "csa_norm_rope_bwd")


def csa_cache_write(x, dtype: int, rows: int, heads: int, d: int, x_row_stride: int,
                    x_head_stride: int, slots, num_slots: int, format: int, data, scales,
                    dev_error=None, stream=None) -> None:
    """Rows into slots of the paged cache, quantised as ``format`` says."""
    _check(load().csa_cache_write(_ptr(x), dtype, rows, heads, d, x_row_stride, x_head_stride,
                                  _ptr(slots), num_slots, format, _ptr(data), _ptr(scales),
                                  _ptr(dev_error), _stream(stream)), "csa_cache_write")


def csa_cache_read(data, scales, format: int, slots, rows: int, num_slots: int, heads: int, d: int,
                   out, dtype: int, out_row_stride: int, out_head_stride: int, dev_error=None,
                   stream=None) -> None:
    """Slots of the paged cache back into rows of ``dtype``."""
    _check(load().csa_cache_read(_ptr(data), _ptr(scales), format, _ptr(slots), rows, num_slots,
                                 heads, d, _ptr(out), dtype, out_row_stride, out_head_stride,
                                 _ptr(dev_error), _stream(stream)), "csa_cache_read")


def csa_cache_attn_workspace_bytes(S: int, tokens: int, q_heads: int, kv_heads: int, d: int,
                                   max_entries: int) -> int:
    return int(load().csa_cache_attn_workspace_bytes(S, tokens, q_heads, kv_heads, d, max_entries))


def csa_cache_attn(q, q_row_stride: int, q_head_stride: int, cu_seqlens, S: int, tokens: int,
                   q_heads: int, kv_heads: int, d: int, data, scales, format: int, page_table,
                   max_pages: int, num_pages: int, page_size: int, entries, first, ratio: int,
                   softmax_scale: float, sink, out, out_row_stride: int, out_head_stride: int,
                   lse, workspace, workspace_bytes: int, dev_error=None, stream=None) -> None:
    """New tokens over the paged cache, an entry being key and value at once."""
    _check(load().csa_cache_attn(_ptr(q), q_row_stride, q_head_stride, _ptr(cu_seqlens), S, tokens,
                                 q_heads, kv_heads, d, _ptr(data), _ptr(scales), format,
                                 _ptr(page_table), max_pages, num_pages, page_size, _ptr(entries),
                                 _ptr(first), ratio, softmax_scale, _ptr(sink), _ptr(out),
                                 out_row_stride, out_head_stride, _ptr(lse), _ptr(workspace),
                                 workspace_bytes, _ptr(dev_error), _stream(stream)),
           "csa_cache_attn")
