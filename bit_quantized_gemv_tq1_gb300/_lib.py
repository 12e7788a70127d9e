"""ctypes binding of libtq1 (include/tq1.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
CUDA tensors (or raw device addresses as ints) plus sizes; all computation
happens in the library's CUDA kernels.  There is no CPU path: if the
library is not built, or a tensor is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

_lock = threading.Lock()
_lib = None

TQ1_OK = 0
STATUS = {
    0: "TQ1_OK", -1: "TQ1_ERR_NULL", -2: "TQ1_ERR_SHAPE", -3: "TQ1_ERR_ALIGN", -4: "TQ1_ERR_UNSUPPORTED",
    -5: "TQ1_ERR_WORKSPACE", -6: "TQ1_ERR_CUDA", -7: "TQ1_ERR_TIMEOUT", -8: "TQ1_ERR_BAD_ID",
    -9: "TQ1_ERR_NO_PAGES",
}
BLOCK_BYTES = 54
Q8_BYTES = 36
TQ1_F32, TQ1_F16, TQ1_BF16 = 0, 1, 2


class KvCache(ctypes.Structure):
    """tq1_kv_cache; made by tq1_kv_cache(), which keeps the tensors alive."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_kv", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class KvBatch(ctypes.Structure):
    """tq1_kv_batch; made by tq1_kv_batch()."""
    _fields_ = [("page_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


class PagePool(ctypes.Structure):
    """tq1_page_pool; made by tq1_page_pool()."""
    _fields_ = [("base", ctypes.c_void_p), ("n_pools", ctypes.c_int64), ("pool_stride", ctypes.c_int64),
                ("page_bytes", ctypes.c_int64), ("n_pages", ctypes.c_int64), ("refs", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("n_seqs", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("page_size", ctypes.c_int64)]


class Tq1Error(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {STATUS.get(code, code)} ({library().tq1_status_string(code).decode()})"
        if code == -6:
            msg += f": {library().tq1_last_cuda_error().decode()}"
        super().__init__(msg)


def library_path() -> str:
    return _build.LIB


def library() -> ctypes.CDLL:
    """Load libtq1.so (must have been built by build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libtq1 is not built ({path} missing): run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        lib.tq1_status_string.restype = ctypes.c_char_p
        lib.tq1_status_string.argtypes = [ctypes.c_int]
        lib.tq1_version.restype = ctypes.c_char_p
        lib.tq1_version.argtypes = []
        lib.tq1_debug_inject_wait_timeout.restype = None
        lib.tq1_debug_inject_wait_timeout.argtypes = []
        lib.tq1_last_cuda_error.restype = ctypes.c_char_p
        lib.tq1_last_cuda_error.argtypes = []
        lib.tq1_blocks_bytes.restype = SZ
        lib.tq1_blocks_bytes.argtypes = [I64, I64]
        lib.tq2_blocks_bytes.restype = SZ
        lib.tq2_blocks_bytes.argtypes = [I64, I64]
        lib.tq2_quantize_rows.argtypes = [P, P, I64, I64, P]
        lib.tq2_mmv.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq2_mmv_partials.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq2_dequantize_rows.argtypes = [P, P, I64, I64, ctypes.c_int, P]
        lib.tq2_mmv_f32.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq2_mmv_add.argtypes = [P, P, P, P, I64, I64, I64, P]
        lib.tq2_mmv_id.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq2_mmv_id_slots.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq2_get_rows.argtypes = [P, P, I64, P, I64, I64, ctypes.c_int, P]
        lib.tq1_q8_1_bytes.restype = SZ
        lib.tq1_q8_1_bytes.argtypes = [I64, I64]
        lib.tq1_quantize_rows.argtypes = [P, P, I64, I64, P]
        lib.q8_1_quantize_acts.argtypes = [P, P, I64, I64, P]
        lib.tq1_mmv.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq1_mmv_partials.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq1_mmv_add.argtypes = [P, P, P, P, I64, I64, I64, P]
        lib.tq1_mmv_f32.argtypes = [P, P, P, I64, I64, I64, P]
        lib.tq1_mmv_id_workspace_size.restype = SZ
        lib.tq1_mmv_id_workspace_size.argtypes = [I64, I64, I64]
        lib.tq1_mmv_id.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq1_mmv_id_slots.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq1_mmv_id_noalloc.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P]
        lib.tq1_mmv_workspace_size.restype = SZ
        lib.tq1_mmv_workspace_size.argtypes = [I64, I64, I64]
        lib.tq1_mmv_ws.argtypes = [P, P, P, P, I64, I64, I64, P, SZ, P]
        lib.tq2_mmv_ws.argtypes = [P, P, P, P, I64, I64, I64, P, SZ, P]
        lib.tq1_mmv_id_partials.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq2_mmv_id_partials.argtypes = [P, I64, P, P, P, I64, I64, I64, I64, P, SZ, P]
        lib.tq1_dequantize_rows.argtypes = [P, P, I64, I64, ctypes.c_int, P]
        lib.tq1_get_rows.argtypes = [P, P, I64, P, I64, I64, ctypes.c_int, P]
        lib.tq1_sync_status.argtypes = [P]
        C, B, G, INT, F32, F64 = (ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch), ctypes.POINTER(PagePool),
                                  ctypes.c_int, ctypes.c_float, ctypes.c_double)
        lib.tq1_rope_freqs.argtypes = [P, I64, F64, F64, F64, F64, F64, P]
        lib.tq1_rope_append.argtypes = [C, B, P, I64, P, I64, P, I64, INT, P, I64, I64, P, I64, INT, F32, P, P]
        lib.tq1_paged_attn_workspace_size.restype = SZ
        lib.tq1_paged_attn_workspace_size.argtypes = [C, I64, I64, I64]
        lib.tq1_paged_attn.argtypes = [C, B, P, I64, I64, I64, F32, INT, I64, P, I64, INT, P, SZ, P]
        lib.tq1_pages_workspace_size.restype = SZ
        lib.tq1_pages_workspace_size.argtypes = [G]
        lib.tq1_pages_copy.argtypes = [G, P, P, I64, P]
        lib.tq1_pages_resize.argtypes = [G, P, P, I64, P, SZ, P]
        lib.tq1_pages_fork.argtypes = [G, P, P, I64, P, SZ, P]
        lib.tq1_pages_compact.argtypes = [G, P, SZ, P]
        for name in ("tq1_quantize_rows", "q8_1_quantize_acts", "tq1_mmv", "tq1_mmv_add", "tq1_mmv_f32",
                     "tq1_mmv_partials", "tq1_mmv_id", "tq1_mmv_id_slots", "tq1_mmv_id_noalloc",
                     "tq1_dequantize_rows", "tq1_get_rows", "tq1_sync_status", "tq2_quantize_rows",
                     "tq2_mmv", "tq2_mmv_partials", "tq2_dequantize_rows", "tq2_get_rows", "tq2_mmv_id",
                     "tq2_mmv_id_slots", "tq2_mmv_f32", "tq2_mmv_add", "tq1_mmv_id_partials",
                     "tq2_mmv_id_partials", "tq1_mmv_ws", "tq2_mmv_ws", "tq1_rope_freqs", "tq1_rope_append",
                     "tq1_paged_attn", "tq1_pages_copy", "tq1_pages_resize", "tq1_pages_fork", "tq1_pages_compact"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def _addr(x) -> int | None:
    """Device address of a CUDA tensor (or an int address, or None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("libtq1 takes CUDA tensors only")
    if not x.is_contiguous():
        raise ValueError("libtq1 takes contiguous tensors only")
    return x.data_ptr()


def _current_stream():
    """A function that returns the address of the current device's current stream."""
    import torch
    try:  # the address alone: building a Stream object takes 3 us, as long as a small call's kernels
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    except AttributeError:
        return lambda: torch.cuda.current_stream().cuda_stream

    torch.cuda.init()
    return lambda: raw(device())


_current = None


def _stream(stream) -> int | None:
    if stream is None:
        global _current
        if _current is None:
            _current = _current_stream()
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != TQ1_OK:
        raise Tq1Error(rc, where)


def tq1_blocks_bytes(n: int, k: int) -> int:
    return int(library().tq1_blocks_bytes(n, k))


def tq1_q8_1_bytes(t: int, k: int) -> int:
    return int(library().tq1_q8_1_bytes(t, k))


def tq1_quantize_rows(w, blocks, n: int, k: int, stream=None) -> None:
    _check(library().tq1_quantize_rows(_addr(w), _addr(blocks), n, k, _stream(stream)), "tq1_quantize_rows")


def q8_1_quantize_acts(x, q8, t: int, k: int, stream=None) -> None:
    _check(library().q8_1_quantize_acts(_addr(x), _addr(q8), t, k, _stream(stream)), "q8_1_quantize_acts")


def tq1_mmv(blocks, q8, y, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq1_mmv(_addr(blocks), _addr(q8), _addr(y), n, k, t, _stream(stream)), "tq1_mmv")


def tq1_mmv_f32(blocks, x, y, n: int, k: int, t: int, stream=None) -> None:
    """Decode mat-vec from fp32 activations, quantised to Q8_1 inside the kernel (t <= 4)."""
    _check(library().tq1_mmv_f32(_addr(blocks), _addr(x), _addr(y), n, k, t, _stream(stream)), "tq1_mmv_f32")


def tq1_mmv_add(blocks, q8, res, y, n: int, k: int, t: int, stream=None) -> None:
    """y = res + W x (res may be y itself)."""
    _check(library().tq1_mmv_add(_addr(blocks), _addr(q8), _addr(res), _addr(y), n, k, t, _stream(stream)),
           "tq1_mmv_add")


def tq1_mmv_workspace_size(n: int, k: int, t: int) -> int:
    """Bytes tq1_mmv_ws / tq2_mmv_ws need (0: the call takes the allocation-free kernels)."""
    return int(library().tq1_mmv_workspace_size(n, k, t))


def tq1_mmv_ws(blocks, q8, y, n: int, k: int, t: int, ws, ws_bytes: int | None = None, res=None,
               stream=None) -> None:
    """tq1_mmv (res None) or tq1_mmv_add with a caller workspace: the tcgen05 tile path at prefill-sized t."""
    wsb = ws_bytes if ws_bytes is not None else (0 if ws is None else ws.numel() * ws.element_size())
    _check(library().tq1_mmv_ws(_addr(blocks), _addr(q8), _addr(res), _addr(y), n, k, t, _addr(ws), wsb,
                                _stream(stream)), "tq1_mmv_ws")


def tq2_mmv_ws(blocks, q8, y, n: int, k: int, t: int, ws, ws_bytes: int | None = None, res=None,
               stream=None) -> None:
    wsb = ws_bytes if ws_bytes is not None else (0 if ws is None else ws.numel() * ws.element_size())
    _check(library().tq2_mmv_ws(_addr(blocks), _addr(q8), _addr(res), _addr(y), n, k, t, _addr(ws), wsb,
                                _stream(stream)), "tq2_mmv_ws")


def tq1_mmv_partials(blocks, q8, part, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq1_mmv_partials(_addr(blocks), _addr(q8), _addr(part), n, k, t, _stream(stream)),
           "tq1_mmv_partials")


def tq1_mmv_id_workspace_size(n_experts: int, t: int, top_k: int) -> int:
    return int(library().tq1_mmv_id_workspace_size(n_experts, t, top_k))


def tq1_mmv_id(expert_blocks, n_experts: int, q8, ids, y, n: int, k: int, t: int, top_k: int, ws,
               ws_bytes: int | None = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(library().tq1_mmv_id(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(y), n, k, t, top_k,
                                _addr(ws), ws_bytes, _stream(stream)), "tq1_mmv_id")


def tq1_mmv_id_slots(expert_blocks, n_experts: int, q8, ids, y, n: int, k: int, t: int, top_k: int, ws,
                     ws_bytes: int | None = None, stream=None) -> None:
    """tq1_mmv_id with one Q8_1 activation row per (token, slot): q8 [t][top_k][k/32]."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(library().tq1_mmv_id_slots(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(y), n, k, t,
                                      top_k, _addr(ws), ws_bytes, _stream(stream)), "tq1_mmv_id_slots")


def tq1_mmv_id_partials(expert_blocks, n_experts: int, q8, ids, part, n: int, k: int, t: int, top_k: int, ws,
                        ws_bytes: int | None = None, stream=None) -> None:
    """Debug: the exact int32 partials part[t][top_k][n][k/32] of tq1_mmv_id."""
    wsb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check(library().tq1_mmv_id_partials(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(part), n, k,
                                         t, top_k, _addr(ws), wsb, _stream(stream)), "tq1_mmv_id_partials")


def tq2_mmv_id_partials(expert_blocks, n_experts: int, q8, ids, part, n: int, k: int, t: int, top_k: int, ws,
                        ws_bytes: int | None = None, stream=None) -> None:
    """Debug: the exact int32 partials part[t][top_k][n][k/32] of tq2_mmv_id."""
    wsb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check(library().tq2_mmv_id_partials(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(part), n, k,
                                         t, top_k, _addr(ws), wsb, _stream(stream)), "tq2_mmv_id_partials")


def tq1_mmv_id_noalloc(expert_blocks, n_experts: int, q8, ids, y, n: int, k: int, t: int, top_k: int,
                       stream=None) -> None:
    """tq1_mmv_id for callers that cannot allocate a workspace: the routing
    table lives in a fixed array inside the library (limits: 1024 experts,
    16384 routed token/slot pairs).  Make the first call on a device before
    any stream capture; calls that may overlap on the GPU race on the array."""
    _check(library().tq1_mmv_id_noalloc(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(y), n, k, t,
                                        top_k, _stream(stream)), "tq1_mmv_id_noalloc")


def tq1_dequantize_rows(blocks, out, n: int, k: int, out_f16: bool = False, stream=None) -> None:
    """out[n][k] (fp32, or fp16 when out_f16) = the values the TQ1_0 blocks encode."""
    _check(library().tq1_dequantize_rows(_addr(blocks), _addr(out), n, k, int(bool(out_f16)), _stream(stream)),
           "tq1_dequantize_rows")


def tq1_get_rows(blocks, row_ids, n_ids: int, out, n: int, k: int, out_f16: bool = False, stream=None) -> None:
    """out[i] = dequantised row row_ids[i] of the n x k TQ1_0 matrix."""
    _check(library().tq1_get_rows(_addr(blocks), _addr(row_ids), n_ids, _addr(out), n, k, int(bool(out_f16)),
                                  _stream(stream)), "tq1_get_rows")


def tq2_blocks_bytes(n: int, k: int) -> int:
    return int(library().tq2_blocks_bytes(n, k))


def tq2_quantize_rows(w, blocks, n: int, k: int, stream=None) -> None:
    _check(library().tq2_quantize_rows(_addr(w), _addr(blocks), n, k, _stream(stream)), "tq2_quantize_rows")


def tq2_mmv(blocks, q8, y, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq2_mmv(_addr(blocks), _addr(q8), _addr(y), n, k, t, _stream(stream)), "tq2_mmv")


def tq2_mmv_f32(blocks, x, y, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq2_mmv_f32(_addr(blocks), _addr(x), _addr(y), n, k, t, _stream(stream)), "tq2_mmv_f32")


def tq2_mmv_add(blocks, q8, res, y, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq2_mmv_add(_addr(blocks), _addr(q8), _addr(res), _addr(y), n, k, t, _stream(stream)),
           "tq2_mmv_add")


def tq2_mmv_partials(blocks, q8, part, n: int, k: int, t: int, stream=None) -> None:
    _check(library().tq2_mmv_partials(_addr(blocks), _addr(q8), _addr(part), n, k, t, _stream(stream)),
           "tq2_mmv_partials")


def tq2_mmv_id(expert_blocks, n_experts: int, q8, ids, y, n: int, k: int, t: int, top_k: int, ws,
               ws_bytes: int | None = None, stream=None) -> None:
    wsb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check(library().tq2_mmv_id(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(y), n, k, t, top_k,
                                _addr(ws), wsb, _stream(stream)), "tq2_mmv_id")


def tq2_mmv_id_slots(expert_blocks, n_experts: int, q8, ids, y, n: int, k: int, t: int, top_k: int, ws,
                     ws_bytes: int | None = None, stream=None) -> None:
    wsb = ws_bytes if ws_bytes is not None else ws.numel() * ws.element_size()
    _check(library().tq2_mmv_id_slots(_addr(expert_blocks), n_experts, _addr(q8), _addr(ids), _addr(y), n, k, t,
                                      top_k, _addr(ws), wsb, _stream(stream)), "tq2_mmv_id_slots")


def tq2_dequantize_rows(blocks, out, n: int, k: int, out_f16: bool = False, stream=None) -> None:
    _check(library().tq2_dequantize_rows(_addr(blocks), _addr(out), n, k, int(out_f16), _stream(stream)),
           "tq2_dequantize_rows")


def tq2_get_rows(blocks, row_ids, n_ids: int, out, n: int, k: int, out_f16: bool = False, stream=None) -> None:
    _check(library().tq2_get_rows(_addr(blocks), _addr(row_ids), n_ids, _addr(out), n, k, int(out_f16),
                                  _stream(stream)), "tq2_get_rows")


def tq1_sync_status(stream=None) -> int:
    """Synchronise the stream; return (and clear) the device status code."""
    return int(library().tq1_sync_status(_stream(stream)))


# ------------------------------------------------ paged key/value cache --
_dtypes = None


def _dtype(x) -> int:
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {torch.float32: TQ1_F32, torch.float16: TQ1_F16, torch.bfloat16: TQ1_BF16}
    code = _dtypes.get(x.dtype)
    if code is None:
        raise ValueError(f"libtq1 takes fp32, fp16 and bf16 here, not {x.dtype}")
    return code


_int32 = None


def _ints(x, n: int | None = None) -> int:
    """Device address of a contiguous int32 tensor (of n elements)."""
    global _int32
    if _int32 is None:
        import torch
        _int32 = torch.int32
    if x.dtype is not _int32:
        raise ValueError(f"libtq1 takes int32 indexes, not {x.dtype}")
    if n is not None and x.numel() != n:
        raise ValueError(f"expected {n} values, got {x.numel()}")
    return _addr(x)


def _rows(x, heads: int | None, d: int, what: str) -> tuple[int, int, int, int]:
    """Address, token stride (elements), tokens and heads of [t][heads][d] rows, e.g. a column range of a fused
    projection."""
    shape = x.shape
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads):
        raise ValueError(f"{what}: expected [t][{heads or 'heads'}][{d}], got {tuple(shape)}")
    if not x.is_cuda:
        raise ValueError("libtq1 takes CUDA tensors only")
    t, n, _ = shape
    st, sh, se = x.stride()
    if se != 1 or (n > 1 and sh != d):
        raise ValueError(f"{what}: a token's heads must be contiguous")
    return x.data_ptr(), st if t > 1 else n * d, t, n


def tq1_kv_cache(k, v) -> KvCache:
    """The cache of pages k, v [n_pages][n_kv][page_size][head_dim] (fp16 or bf16): any strides, the same for
    both, with unit stride along head_dim.  A pool kept as [n_pages][page_size][n_kv][head_dim] is passed
    as k.transpose(1, 2), v.transpose(1, 2)."""
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
        raise ValueError("k and v pages: two tensors of one shape [n_pages][n_kv][page_size][head_dim], type and strides")
    if not (k.is_cuda and v.is_cuda):
        raise ValueError("libtq1 takes CUDA tensors only")
    if k.stride(3) != 1:
        raise ValueError("k and v pages: unit stride along head_dim")
    c = KvCache(k.data_ptr(), v.data_ptr(), k.shape[0], k.shape[1], k.shape[2], k.shape[3], k.stride(0), k.stride(1),
                k.stride(2), _dtype(k))
    c.keep = (k, v)
    return c


def tq1_kv_batch(page_table, q_start, kv_len) -> KvBatch:
    """Sequences of a call: page_table [n_seqs][max_pages], q_start [n_seqs + 1], kv_len [n_seqs], int32."""
    n, width = page_table.shape
    b = KvBatch(_ints(page_table), _ints(q_start, n + 1), _ints(kv_len, n), n, width)
    b.keep = (page_table, q_start, kv_len)
    return b


def tq1_rope_freqs(inv_freq, rot_dim: int, base: float = 10000.0, factor: float = 1.0, orig_len: float = 0.0,
                   low: float = 1.0, high: float = 32.0, stream=None) -> None:
    """Fill inv_freq [rot_dim/2] (fp32): plain, or stretched for contexts `factor` times longer than orig_len."""
    if inv_freq.numel() != rot_dim // 2 or _dtype(inv_freq) != TQ1_F32:
        raise ValueError(f"inv_freq: expected {rot_dim // 2} fp32 values")
    _check(library().tq1_rope_freqs(_addr(inv_freq), rot_dim, base, factor, orig_len, low, high, _stream(stream)),
           "tq1_rope_freqs")


def tq1_rope_append(cache, batch, q, k, v, q_out, inv_freq, rot_dim: int, interleaved: bool = False,
                    mscale: float = 1.0, positions=None, stream=None) -> None:
    """Rotate q [t][n_q][d] into q_out and append the rotated k and the v [t][n_kv][d] to the cache's pages."""
    d, n_kv = cache.head_dim, cache.n_kv
    pq, ldq, t, n_q = _rows(q, None, d, "q")
    pk, ldk, tk, _ = _rows(k, n_kv, d, "k")
    pv, ldv, tv, _ = _rows(v, n_kv, d, "v")
    dtype = q.dtype
    if tk != t or tv != t or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k and v: one type and one number of tokens")
    if q_out.shape != (t, n_q, d) or _dtype(q_out) != cache.dtype:
        raise ValueError("q_out: q's shape and the cache's type")
    if inv_freq is not None and (inv_freq.numel() != rot_dim // 2 or _dtype(inv_freq) != TQ1_F32):
        raise ValueError(f"inv_freq: expected {rot_dim // 2} fp32 values")
    pos = None if positions is None else _ints(positions, t)
    _check(library().tq1_rope_append(cache, batch, pq, ldq, pk, ldk, pv, ldv, _dtype(q), _addr(q_out), t, n_q,
                                     _addr(inv_freq), rot_dim, 1 if interleaved else 0, mscale, pos, _stream(stream)),
           "tq1_rope_append")


def tq1_paged_attn_workspace_size(cache, t: int, n_q: int, n_seqs: int) -> int:
    return int(library().tq1_paged_attn_workspace_size(cache, t, n_q, n_seqs))


def tq1_paged_attn(cache, batch, q, out, scale: float, causal: bool = True, window: int = 0, ws=None,
                   ws_bytes: int | None = None, stream=None) -> None:
    """out [t][n_q][d] (the cache's type, or fp32) = attention of q [t][n_q][d] over the batch's pages."""
    d, dtype, out_dtype = cache.head_dim, cache.dtype, _dtype(out)
    pq, ldq, t, n_q = _rows(q, None, d, "q")
    po, ldo, to, _ = _rows(out, n_q, d, "out")
    if to != t or _dtype(q) != dtype or (out_dtype != dtype and out_dtype != TQ1_F32):
        raise ValueError("q: the cache's type; out: q's shape, the cache's type or fp32")
    wsb = ws_bytes if ws_bytes is not None else (0 if ws is None else ws.numel() * ws.element_size())
    _check(library().tq1_paged_attn(cache, batch, pq, ldq, t, n_q, scale, 1 if causal else 0, window, po, ldo,
                                    1 if out_dtype == TQ1_F32 else 0, _addr(ws), wsb, _stream(stream)), "tq1_paged_attn")


def tq1_page_pool(pools, page_table, kv_len, refs, page_size: int) -> PagePool:
    """The pools [n_pools][n_pages][...] (any type; each page contiguous) that share page_table [n_seqs][max_pages],
    kv_len [n_seqs] and refs [n_pages] (int32)."""
    if not pools.is_cuda or pools.dim() < 3 or not pools[0].is_contiguous():
        raise ValueError("pools: a CUDA tensor [n_pools][n_pages][...] with contiguous pools")
    n, width = page_table.shape
    n_pages, size = pools.shape[1], pools.element_size()
    page_bytes = pools[0, 0].numel() * size
    p = PagePool(pools.data_ptr(), pools.shape[0], pools.stride(0) * size if pools.shape[0] > 1 else n_pages * page_bytes,
                 page_bytes, n_pages, _ints(refs, n_pages), _ints(page_table), _ints(kv_len, n), n, width, page_size)
    p.keep = (pools, page_table, kv_len, refs)
    return p


def tq1_pages_workspace_size(pool) -> int:
    return int(library().tq1_pages_workspace_size(pool))


def tq1_pages_copy(pool, src, dst, stream=None) -> None:
    """Copy pages src[i] -> dst[i] in every pool."""
    _check(library().tq1_pages_copy(pool, _ints(src), _ints(dst, src.numel()), src.numel(), _stream(stream)),
           "tq1_pages_copy")


def tq1_pages_resize(pool, seqs, new_len, ws, stream=None) -> None:
    """Set the length of sequences seqs[i] to new_len[i]: pages are freed, given, and copied where shared."""
    n = seqs.numel()
    _check(library().tq1_pages_resize(pool, _ints(seqs), _ints(new_len, n), n, _addr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)), "tq1_pages_resize")


def tq1_pages_fork(pool, parents, children, ws, stream=None) -> None:
    """The empty sequences children[i] become copies of parents[i], sharing their full pages."""
    n = parents.numel()
    _check(library().tq1_pages_fork(pool, _ints(parents), _ints(children, n), n, _addr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)), "tq1_pages_fork")


def tq1_pages_compact(pool, ws, stream=None) -> None:
    """Move the pages in use to the lowest ids; tables and counts follow."""
    _check(library().tq1_pages_compact(pool, _addr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "tq1_pages_compact")
