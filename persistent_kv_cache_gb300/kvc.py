"""Python binding of the C ABI in include/kvc.h (argument marshalling only).

Every function has the C entry point's name and forwards torch tensors as raw
pointers plus the current CUDA stream; all the work happens in libkvc.so's
kernels.  There is no CPU path: a missing library raises ``KvcLibraryMissing``.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvc.so")

KVC_F32, KVC_BF16, KVC_F16 = 0, 1, 2
KVC_LINEAR, KVC_CIRCULAR = 0, 1
KVC_APPEND, KVC_COPY_BACK = 0, 1
KVC_INT8, KVC_E4M3 = 0, 1

KVC_OK = 0
STATUS_NAMES = {
    0: "KVC_OK", 1: "KVC_ERR_NULL", 2: "KVC_ERR_SHAPE", 3: "KVC_ERR_DTYPE", 4: "KVC_ERR_ALIGN",
    5: "KVC_ERR_UNSUPPORTED", 6: "KVC_ERR_CAPACITY", 7: "KVC_ERR_WINDOW",
    8: "KVC_ERR_WORKSPACE", 9: "KVC_ERR_CUDA",
}
# cache policies (the `windowed` argument)
KVC_CONTIGUOUS, KVC_WINDOWED, KVC_DRIFTING, KVC_RING = 0, 1, 2, 3
KVC_DEV_INDEX_OOB = 1
KVC_DEV_SEQLEN_RANGE = 2
KVC_DEV_CAPACITY = 4
KVC_DEV_ROPE_RANGE = 8
KVC_DEV_TIMEOUT = 16

EXPORTS = ("kvc_tensor_scatter", "kvc_seq_lengths", "kvc_window_append", "kvc_gqa_decode",
           "kvc_gqa_decode_workspace_size", "kvc_gqa_decode_noalloc", "kvc_gqa_decode_ring",
           "kvc_decode_step", "kvc_decode_step_workspace_size", "kvc_window_decode_step",
           "kvc_window_decode_step_workspace_size",
           "kvc_paged_append", "kvc_gqa_decode_paged", "kvc_window_append_inplace",
           "kvc_quantize_pages", "kvc_gqa_decode_paged_q",
           "kvc_gqa_prefill_chunk", "kvc_gqa_prefill_workspace_size", "kvc_window_prefill_step",
           "kvc_quant_append", "kvc_dequant_rows", "kvc_gqa_decode_quant",
           "kvc_gqa_decode_quant_workspace_size", "kvc_page_bounds", "kvc_gqa_decode_sparse",
           "kvc_gqa_decode_sparse_workspace_size", "kvc_tree_mask", "kvc_tree_append",
           "kvc_gqa_tree", "kvc_gqa_tree_workspace_size", "kvc_tree_commit",
           "kvc_status_string", "kvc_abi_version")
KVC_DECODE_STATIC_SCRATCH_BYTES = 16 << 20
KVC_PAGE_QUANT = 0x40000000  # block-table flag: the entry names an int8 page


class KvcLibraryMissing(RuntimeError):
    pass


class KvcError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")


class KvcLengths(ctypes.Structure):
    _fields_ = [("past_abs", ctypes.c_void_p), ("total_abs", ctypes.c_void_p),
                ("cache_past", ctypes.c_void_p), ("cache_total", ctypes.c_void_p),
                ("evict", ctypes.c_void_p)]


class Lengths:
    """Five int32 device tensors of [batch] (past_abs, total_abs, cache_past,
    cache_total, evict) written by kvc_seq_lengths."""

    FIELDS = ("past_abs", "total_abs", "cache_past", "cache_total", "evict")

    def __init__(self, batch: int, device):
        self.batch = batch
        self.buf = torch.empty((5, batch), dtype=torch.int32, device=device)
        self.at = self.buf.get_device()
        self._c = KvcLengths(*[self.buf[i].data_ptr() for i in range(5)])

    def __getattr__(self, name):
        if name in Lengths.FIELDS:
            return self.buf[Lengths.FIELDS.index(name)]
        raise AttributeError(name)

    def c(self) -> KvcLengths:
        return self._c


_lib = None


def library() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise KvcLibraryMissing(
                f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, I64, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
        L = KvcLengths
        sig = {
            "kvc_tensor_scatter": [P, P, P, P, I, P, I64, I, I, I, P, P],
            "kvc_seq_lengths": [P, I, I, I64, I, I, L, P, P],
            "kvc_window_append": [P, P, P, P, P, P, L, I, I, I, I64, I, I, I, I, P, P, I64, P, P],
            "kvc_window_append_inplace": [P, P, P, P, L, I, I, I, I64, I64, I, I, I, I, P, P, I64,
                                          P, P],
            "kvc_gqa_decode": [P, P, P, P, L, I, I, I, I64, I, I, I, F, P, P, I64, P, SZ, P, P],
            "kvc_gqa_decode_ring": [P, P, P, P, L, I, I, I, I64, I, I, I, F, P, P, I64, P, SZ, P,
                                    P],
            "kvc_gqa_decode_workspace_size": [I, I, I, I64, I, I],
            "kvc_paged_append": [P, P, P, P, P, I, I64, I, L, I, I, I, I, I, P, P, I64, P, P],
            "kvc_gqa_decode_paged": [P, P, P, P, P, I, I64, I, L, I, I, I, I, I, I, F, P, P, I64,
                                     P, SZ, P, P],
            "kvc_quantize_pages": [P, P, P, P, P, P, I, I64, I64, I, I, I, I, F, I, I, F, I, I, P,
                                   P, P],
            "kvc_gqa_decode_paged_q": [P, P, P, P, P, P, P, I64, P, I, I64, I, L, I, I, I, I, I, I,
                                       F, P, P, I64, P, SZ, P, P],
            "kvc_decode_step": [P, P, P, P, P, P, P, L, I, I, I, I64, I, I, I, I, F, P, P, I64, P,
                                SZ, P, P],
            "kvc_decode_step_workspace_size": [I, I, I, I64, I, I],
            "kvc_gqa_decode_noalloc": [P, P, P, P, L, I, I, I, I64, I, I, I, F, P, P, I64, P, P],
            "kvc_window_decode_step": [P, P, P, P, P, P, P, L, I, I, I, I64, I, I, I, I, F, P, P,
                                       I64, P, SZ, P, P],
            "kvc_window_decode_step_workspace_size": [I, I, I, I64, I, I],
            "kvc_gqa_prefill_chunk": [P, P, P, P, I64, L, I, I, I, I, I, I, I, F, P, P, I64, P, SZ,
                                      P, P],
            "kvc_gqa_prefill_workspace_size": [I, I, I, I, I64, I, I, I],
            "kvc_window_prefill_step": [P, P, P, P, P, P, P, P, L, I, I, I, I, I64, I, I, I, I,
                                        F, P, P, I64, P, SZ, P, P],
            "kvc_quant_append": [P, P, P, P, P, P, L, I, I, I, I64, I, I, I, I, P, P, I64, P, P],
            "kvc_dequant_rows": [P, P, P, P, P, P, L, I, I, I64, I64, I, I, I, I, P, P],
            "kvc_gqa_decode_quant": [P, P, P, P, P, P, L, I, I, I, I64, I, I, I, I, I, F, P, P, I64,
                                     P, SZ, P, P],
            "kvc_gqa_decode_quant_workspace_size": [I, I, I, I64, I],
            "kvc_page_bounds": [P, P, P, P, I, I64, I, L, I, I, I, I, I, P, P],
            "kvc_gqa_decode_sparse": [P, P, P, P, P, P, P, I, I64, I, L, I, I, I, I, I, I, I, I, P, F,
                                      P, P, I64, P, SZ, P, P],
            "kvc_gqa_decode_sparse_workspace_size": [I, I, I, I, I, I, I],
            "kvc_tree_mask": [P, I, I, P, P, P, P],
            "kvc_tree_append": [P, P, P, P, P, P, I, I64, I, L, I, I, I, I64, I, I, P, P, I64, P, P],
            "kvc_gqa_tree": [P, P, P, P, P, P, P, I, I64, I, L, I, I, I, I, I64, I, I, I, F, P, P, I64,
                             P, SZ, P, P],
            "kvc_gqa_tree_workspace_size": [I, I, I, I, I],
            "kvc_tree_commit": [P, P, P, P, I, P, I, I64, I, L, P, I, I, I, I64, I, I, P, P],
            "kvc_status_string": [I],
            "kvc_abi_version": [],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = I
        lib.kvc_gqa_decode_workspace_size.restype = SZ
        lib.kvc_decode_step_workspace_size.restype = SZ
        lib.kvc_window_decode_step_workspace_size.restype = SZ
        lib.kvc_gqa_prefill_workspace_size.restype = SZ
        lib.kvc_gqa_decode_quant_workspace_size.restype = SZ
        lib.kvc_gqa_decode_sparse_workspace_size.restype = SZ
        lib.kvc_gqa_tree_workspace_size.restype = SZ
        lib.kvc_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _ptr(t):
    """Device address of a tensor the library reads or writes as a dense
    array: it must live on a CUDA device and be contiguous (a strided view
    would be read in the wrong order, or past its storage)."""
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    raise ValueError(f"expected a contiguous tensor, got shape {tuple(t.shape)} "
                     f"with strides {t.stride()}")


# the current stream's handle without a Stream object around it (a twentieth of the time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_get_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _addresses(*tensors):
    """Device addresses (None for None) of tensors that the library reads or writes as dense
    arrays on the current device; the first one is there."""
    if not tensors[0].is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {tensors[0].device}")
    at = _get_device()
    found = []
    for t in tensors:
        if t is None:
            found.append(None)
        elif t.get_device() == at and t.is_contiguous():
            found.append(t.data_ptr())
        elif t.get_device() != at:
            raise ValueError(f"expected a CUDA tensor on the current device, cuda:{at}, "
                             f"got one on {t.device}")
        else:
            _ptr(t)  # (raises)
    return found


def _lengths_of(lengths, batch):
    if lengths.batch != batch:
        raise ValueError(f"lengths: made for {lengths.batch} batch rows, the tensors have {batch}")
    if lengths.at != _get_device():
        raise ValueError(f"lengths: expected on the current device, cuda:{_get_device()}, got {lengths.buf.device}")
    return lengths.c()


def _made_on(stream, make, *args):
    """make(*args), its tensors from the memory of the stream that the call runs on.  Memory of the
    current stream is not that stream's to write yet: a kernel queued on the current one may still
    read what the block held before, and given back it would go to the current one's next kernel
    while the call still runs."""
    if stream is None:
        return make(*args)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream))
    with torch.cuda.stream(s):
        return make(*args)


_DTYPE_CODES = {torch.float32: KVC_F32, torch.bfloat16: KVC_BF16, torch.float16: KVC_F16}


def _dtype_code(t: torch.Tensor) -> int:
    return _DTYPE_CODES[t.dtype]


def _check(fn: str, status: int):
    if status != KVC_OK:
        raise KvcError(fn, status)


def _rope(rope):
    if rope is None:
        return None, None, 0
    cos, sin = rope
    if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape:
        raise ValueError("rope: cos and sin are float32 tables of the same shape [max_pos, D/2]")
    return _ptr(cos), _ptr(sin), cos.shape[0]


def _tables(rope, D):
    """cos, sin and their length of a rope argument for head_dim D (the library gets the length
    alone, and would read tables of another width at the wrong places)"""
    if rope is None:
        return None, None, 0
    cos, sin = rope
    shape = cos.shape
    if (sin.shape != shape or len(shape) != 2 or 2 * shape[1] != D or cos.dtype is not torch.float32
            or sin.dtype is not torch.float32):
        raise ValueError(f"rope: cos and sin are float32 tables of the same shape [max_pos, {D // 2}], got "
                         f"{tuple(shape)} {cos.dtype} and {tuple(sin.shape)} {sin.dtype}")
    return cos, sin, shape[0]


def kvc_tensor_scatter(present, past, update, write_indices=None, axis=-2, mode=KVC_LINEAR,
                       status=None, stream=None):
    shape = (ctypes.c_int64 * past.dim())(*past.shape)
    seq_axis = axis if axis >= 0 else axis + past.dim()
    _check("kvc_tensor_scatter", library().kvc_tensor_scatter(
        _ptr(present), _ptr(past), _ptr(update), _ptr(write_indices), past.dim(), shape,
        update.shape[seq_axis], axis, mode, past.element_size(), _ptr(status), _stream(stream)))
    return present


def kvc_seq_lengths(seqlens_k, new_tokens, capacity, windowed, local_window_size=0, out=None,
                    status=None, stream=None):
    out = Lengths(seqlens_k.shape[0], seqlens_k.device) if out is None else out
    _check("kvc_seq_lengths", library().kvc_seq_lengths(
        _ptr(seqlens_k), seqlens_k.shape[0], new_tokens, capacity, int(windowed),
        local_window_size, out.c(), _ptr(status), _stream(stream)))
    return out


def kvc_window_append(k_cache, v_cache, new_k, new_v, lengths, windowed, phase=KVC_APPEND,
                      k_stage=None, v_stage=None, rope=None, status=None, stream=None):
    B, Hkv, C, D = k_cache.shape
    S = new_k.shape[2] if new_k is not None else (k_stage.shape[2] - C)
    cs, sn, rmax = _rope(rope)
    _check("kvc_window_append", library().kvc_window_append(
        _ptr(k_cache), _ptr(v_cache), _ptr(new_k), _ptr(new_v), _ptr(k_stage), _ptr(v_stage),
        lengths.c(), B, Hkv, S, C, D, _dtype_code(k_cache), int(windowed), phase, cs, sn, rmax,
        _ptr(status), _stream(stream)))


def kvc_window_append_inplace(k_rows, v_rows, new_k, new_v, lengths, capacity, windowed,
                              phase=KVC_APPEND, new_tokens=None, rope=None, status=None,
                              stream=None):
    """k_rows/v_rows: [B, Hkv, rows_per_head, D] with rows_per_head >= capacity + S; the
    cache lives in rows [0, Lp).  new_tokens is needed when new_k is None (KVC_COPY_BACK)."""
    B, Hkv, R, D = k_rows.shape
    S = new_k.shape[2] if new_k is not None else int(new_tokens)
    cs, sn, rmax = _rope(rope)
    _check("kvc_window_append_inplace", library().kvc_window_append_inplace(
        _ptr(k_rows), _ptr(v_rows), _ptr(new_k), _ptr(new_v), lengths.c(), B, Hkv, S, capacity, R,
        D, _dtype_code(k_rows), int(windowed), phase, cs, sn, rmax, _ptr(status),
        _stream(stream)))


def kvc_gqa_decode_workspace_size(batch, q_heads, kv_heads, capacity, head_dim, dtype):
    return library().kvc_gqa_decode_workspace_size(batch, q_heads, kv_heads, capacity, head_dim,
                                                   dtype)


def decode_workspace(q, k_cache):
    B, Hq, _, D = q.shape
    n = kvc_gqa_decode_workspace_size(B, Hq, k_cache.shape[1], k_cache.shape[2], D,
                                      _dtype_code(q))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def kvc_gqa_decode(out, q, k_cache, v_cache, lengths, local_window_size=0, scale=0.0, rope=None,
                   workspace=None, status=None, stream=None):
    B, Hq, _, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    ws = decode_workspace(q, k_cache) if workspace is None else workspace
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_decode", library().kvc_gqa_decode(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), lengths.c(), B, Hq, Hkv, C, D,
        _dtype_code(q), local_window_size, scale, cs, sn, rmax, _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))
    return out


def kvc_gqa_decode_ring(out, q, k_cache, v_cache, lengths, local_window_size=0, scale=0.0,
                        rope=None, workspace=None, status=None, stream=None):
    """kvc_gqa_decode over a ring of C slots (include/kvc.h)."""
    B, Hq, _, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    ws = decode_workspace(q, k_cache) if workspace is None else workspace
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_decode_ring", library().kvc_gqa_decode_ring(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), lengths.c(), B, Hq, Hkv, C, D,
        _dtype_code(q), local_window_size, scale, cs, sn, rmax, _ptr(ws), ws.numel(),
        _ptr(status), _stream(stream)))
    return out


def kvc_paged_append(k_pool, v_pool, new_k, new_v, block_table, lengths, rope=None, status=None,
                     stream=None):
    """Append on a paged cache: pools [pages, Hkv, page_size, D], block_table
    int32 [B, max_pages] (include/kvc.h)."""
    n_pages, Hkv, ps, D = k_pool.shape
    B, _, S, _ = new_k.shape
    cs, sn, rmax = _rope(rope)
    _check("kvc_paged_append", library().kvc_paged_append(
        _ptr(k_pool), _ptr(v_pool), _ptr(new_k), _ptr(new_v), _ptr(block_table),
        block_table.shape[1], n_pages, ps, lengths.c(), B, Hkv, S, D, _dtype_code(k_pool), cs,
        sn, rmax, _ptr(status), _stream(stream)))


def kvc_quantize_pages(k_pool, v_pool, qk_pool, qv_pool, src_pages, dst_pages, qparams, k_scale,
                       k_zero_point=0, k_unsigned=False, v_scale=None, v_zero_point=None,
                       v_unsigned=None, status=None, stream=None):
    """Int8 pages dst_pages[i] <- 16-bit pages src_pages[i] (include/kvc.h); V takes K's
    format unless given its own."""
    n_pool, Hkv, ps, D = k_pool.shape
    v_scale = k_scale if v_scale is None else v_scale
    v_zero_point = k_zero_point if v_zero_point is None else v_zero_point
    v_unsigned = k_unsigned if v_unsigned is None else v_unsigned
    _check("kvc_quantize_pages", library().kvc_quantize_pages(
        _ptr(k_pool), _ptr(v_pool), _ptr(qk_pool), _ptr(qv_pool), _ptr(src_pages),
        _ptr(dst_pages), src_pages.numel(), n_pool, qk_pool.shape[0], ps, Hkv, D,
        _dtype_code(k_pool), float(k_scale), int(k_zero_point), int(bool(k_unsigned)),
        float(v_scale), int(v_zero_point), int(bool(v_unsigned)), _ptr(qparams), _ptr(status),
        _stream(stream)))


def kvc_gqa_decode_paged_q(out, q, k_pool, v_pool, qk_pool, qv_pool, qparams, block_table,
                           lengths, local_window_size=0, scale=0.0, rope=None, workspace=None,
                           status=None, stream=None):
    """kvc_gqa_decode_paged over 16-bit and int8 pages (include/kvc.h)."""
    B, Hq, _, D = q.shape
    n_pages, Hkv, ps, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if workspace is None:
        n = kvc_gqa_decode_workspace_size(B, Hq, Hkv, max_pages * ps, D, _dtype_code(q))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_decode_paged_q", library().kvc_gqa_decode_paged_q(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(qk_pool), _ptr(qv_pool),
        _ptr(qparams), qk_pool.shape[0], _ptr(block_table), max_pages, n_pages, ps, lengths.c(),
        B, Hq, Hkv, D, _dtype_code(q), local_window_size, scale, cs, sn, rmax, _ptr(workspace),
        workspace.numel(), _ptr(status), _stream(stream)))
    return out


def kvc_gqa_decode_paged(out, q, k_pool, v_pool, block_table, lengths, local_window_size=0,
                         scale=0.0, rope=None, workspace=None, status=None, stream=None):
    """kvc_gqa_decode over a paged cache (include/kvc.h)."""
    B, Hq, _, D = q.shape
    n_pages, Hkv, ps, _ = k_pool.shape
    max_pages = block_table.shape[1]
    if workspace is None:
        n = kvc_gqa_decode_workspace_size(B, Hq, Hkv, max_pages * ps, D, _dtype_code(q))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_decode_paged", library().kvc_gqa_decode_paged(
        _ptr(out), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table), max_pages, n_pages,
        ps, lengths.c(), B, Hq, Hkv, D, _dtype_code(q), local_window_size, scale, cs, sn, rmax,
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream)))
    return out


def kvc_gqa_decode_noalloc(out, q, k_cache, v_cache, lengths, local_window_size=0, scale=0.0,
                           rope=None, status=None, stream=None):
    """kvc_gqa_decode with the library's own scratch (see include/kvc.h)."""
    B, Hq, _, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_decode_noalloc", library().kvc_gqa_decode_noalloc(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), lengths.c(), B, Hq, Hkv, C, D,
        _dtype_code(q), local_window_size, scale, cs, sn, rmax, _ptr(status), _stream(stream)))
    return out


def decode_step_workspace(q, k_cache):
    """Workspace for kvc_decode_step (the split partials)."""
    B, Hq, _, D = q.shape
    n = library().kvc_decode_step_workspace_size(B, Hq, k_cache.shape[1], k_cache.shape[2], D,
                                                 _dtype_code(q))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def kvc_decode_step(out, q, k_cache, v_cache, new_k, new_v, seqlens_k, local_window_size=0,
                    lengths=None, scale=0.0, rope=None, workspace=None, status=None, stream=None,
                    windowed=None):
    """Fused lengths + one-token append + split decode on a contiguous cache
    (default) or a ring (windowed=KVC_RING); include/kvc.h."""
    windowed = KVC_CONTIGUOUS if windowed is None else int(windowed)
    B, Hq, _, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    ws = decode_step_workspace(q, k_cache) if workspace is None else workspace
    cs, sn, rmax = _rope(rope)
    lc = lengths.c() if lengths is not None else KvcLengths(None, None, None, None, None)
    _check("kvc_decode_step", library().kvc_decode_step(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(new_k), _ptr(new_v),
        _ptr(seqlens_k), lc, B, Hq, Hkv, C, D, _dtype_code(q), windowed, local_window_size,
        scale, cs, sn, rmax, _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return out


def window_step_workspace(q, k_cache):
    """Workspace for kvc_window_decode_step (None for a window held on chip)."""
    B, Hq, _, D = q.shape
    n = library().kvc_window_decode_step_workspace_size(B, Hq, k_cache.shape[1],
                                                        k_cache.shape[2], D, _dtype_code(q))
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def kvc_window_decode_step(out, q, k_cache, v_cache, new_k, new_v, seqlens_k, local_window_size,
                           lengths=None, scale=0.0, rope=None, status=None, stream=None,
                           windowed=None, workspace="auto"):
    """Lengths + windowed one-token append + GQA decode (include/kvc.h).
    ``windowed``: KVC_WINDOWED (default), KVC_DRIFTING or KVC_RING;
    ``workspace``: "auto" allocates what the call needs (large windows only)."""
    windowed = KVC_WINDOWED if windowed is None else int(windowed)
    B, Hq, _, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    if isinstance(workspace, str):
        workspace = window_step_workspace(q, k_cache)
    cs, sn, rmax = _rope(rope)
    lc = lengths.c() if lengths is not None else KvcLengths(None, None, None, None, None)
    _check("kvc_window_decode_step", library().kvc_window_decode_step(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(new_k), _ptr(new_v),
        _ptr(seqlens_k), lc, B, Hq, Hkv, C, D, _dtype_code(q), windowed, local_window_size,
        scale, cs, sn, rmax, _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _ptr(status), _stream(stream)))
    return out


def prefill_workspace(q, k_rows, local_window_size=0):
    """Workspace for kvc_gqa_prefill_chunk's KV split (None when it would
    not split)."""
    B, Hq, S, D = q.shape
    _, Hkv, R, _ = k_rows.shape
    n = library().kvc_gqa_prefill_workspace_size(B, Hq, Hkv, S, R, D, _dtype_code(q),
                                                 local_window_size)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def kvc_gqa_prefill_chunk(out, q, k_rows, v_rows, lengths, local_window_size=0, scale=0.0,
                          rope=None, status=None, stream=None, workspace="auto"):
    """workspace: "auto" allocates what the call can use, None runs unsplit."""
    B, Hq, S, D = q.shape
    _, Hkv, R, _ = k_rows.shape
    if isinstance(workspace, str):
        workspace = prefill_workspace(q, k_rows, local_window_size)
    cs, sn, rmax = _rope(rope)
    _check("kvc_gqa_prefill_chunk", library().kvc_gqa_prefill_chunk(
        _ptr(out), _ptr(q), _ptr(k_rows), _ptr(v_rows), R, lengths.c(), B, Hq, Hkv, S, D,
        _dtype_code(q), local_window_size, scale, cs, sn, rmax, _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(status), _stream(stream)))
    return out


def kvc_status_string(code: int) -> str:
    return library().kvc_status_string(code).decode()


def kvc_abi_version() -> int:
    return library().kvc_abi_version()


def kvc_window_prefill_step(out, q, k_cache, v_cache, new_k, new_v, lengths, windowed,
                            local_window_size, k_stage=None, v_stage=None, scale=0.0, rope=None,
                            status=None, stream=None, workspace="auto"):
    """One windowed S-token step that stages only the rows whose eviction its
    chunk would see (include/kvc.h).  k_stage/v_stage: [B, Hkv, C + S, D]
    (needed for S > 1).  workspace: "auto" allocates what the attention can
    use, None runs it unsplit."""
    B, Hq, S, D = q.shape
    _, Hkv, C, _ = k_cache.shape
    if isinstance(workspace, str):
        n = library().kvc_gqa_prefill_workspace_size(B, Hq, Hkv, S, C, D, _dtype_code(q),
                                                     local_window_size)
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    cs, sn, rmax = _rope(rope)
    _check("kvc_window_prefill_step", library().kvc_window_prefill_step(
        _ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(new_k), _ptr(new_v),
        _ptr(k_stage), _ptr(v_stage), lengths.c(), B, Hq, Hkv, S, C, D, _dtype_code(q),
        int(windowed), local_window_size, scale, cs, sn, rmax, _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(status), _stream(stream)))
    return out


def _same(name, t, shape, dtype=None):
    """t has the shape (and type) that the other arguments fix: the library
    gets sizes once, from one of them, and cannot see the others'."""
    if t.shape != shape or (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{name}: expected {tuple(shape)}{'' if dtype is None else f' {dtype}'}, "
                         f"got {tuple(t.shape)} {t.dtype}")


_CODE_FORMATS = {torch.int8: KVC_INT8, torch.float8_e4m3fn: KVC_E4M3}


def _code_format(kq):
    fmt = _CODE_FORMATS.get(kq.dtype)
    if fmt is None:
        raise ValueError(f"a quantised cache is torch.int8 or torch.float8_e4m3fn, got {kq.dtype}")
    return fmt


def _quant_cache(kq, vq, k_scale, v_scale):
    """The sizes and format of a quantised cache: kq, vq [B, Hkv, C, D] codes and k_scale,
    v_scale [B, Hkv, C] float32."""
    fmt, shape = _code_format(kq), kq.shape
    B, Hkv, C, _ = shape
    _same("vq", vq, shape, kq.dtype)
    _same("k_scale", k_scale, (B, Hkv, C), torch.float32)
    _same("v_scale", v_scale, (B, Hkv, C), torch.float32)
    return shape, fmt


def kvc_quant_append(kq, vq, k_scale, v_scale, new_k, new_v, lengths, windowed, rope=None,
                     status=None, stream=None):
    """Write new rows [B, Hkv, S, D] into a quantised cache (include/kvc.h): kq, vq
    [B, Hkv, C, D] int8 or float8_e4m3fn, k_scale, v_scale [B, Hkv, C] float32."""
    (B, Hkv, C, D), fmt = _quant_cache(kq, vq, k_scale, v_scale)
    shape = new_k.shape
    S = shape[2]
    _same("new_v", new_v, shape, new_k.dtype)
    if shape != (B, Hkv, S, D):
        _same("new_k", new_k, (B, Hkv, S, D))
    cos, sin, rmax = _tables(rope, D)
    a, b, c, d, e, f, cs, sn, st = _addresses(kq, vq, k_scale, v_scale, new_k, new_v, cos, sin,
                                              status)
    _check("kvc_quant_append", library().kvc_quant_append(
        a, b, c, d, e, f, _lengths_of(lengths, B), B, Hkv, S, C, D, _dtype_code(new_k), fmt,
        int(windowed), cs, sn, rmax, st, _stream(stream)))


def kvc_dequant_rows(k_out, v_out, kq, vq, k_scale, v_scale, lengths, windowed, status=None,
                     stream=None):
    """The resident rows of a quantised cache, oldest first, into k_out, v_out
    [B, Hkv, rows, D] (include/kvc.h)."""
    (B, Hkv, C, D), fmt = _quant_cache(kq, vq, k_scale, v_scale)
    shape = k_out.shape
    R = shape[2]
    _same("v_out", v_out, shape, k_out.dtype)
    if shape != (B, Hkv, R, D):
        _same("k_out", k_out, (B, Hkv, R, D))
    a, b, c, d, e, f, st = _addresses(k_out, v_out, kq, vq, k_scale, v_scale, status)
    _check("kvc_dequant_rows", library().kvc_dequant_rows(
        a, b, c, d, e, f, _lengths_of(lengths, B), B, Hkv, C, R, D, _dtype_code(k_out), fmt,
        int(windowed), st, _stream(stream)))


def quant_decode_workspace(q, kq):
    """Workspace for kvc_gqa_decode_quant (None when it needs none)."""
    B, Hq, _, D = q.shape
    n = library().kvc_gqa_decode_quant_workspace_size(B, Hq, kq.shape[1], kq.shape[2], D)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def kvc_gqa_decode_quant(out, q, kq, vq, k_scale, v_scale, lengths, windowed, local_window_size=0,
                         scale=0.0, rope=None, workspace="auto", status=None, stream=None):
    """One-token attention over a quantised cache (include/kvc.h).  workspace: "auto" allocates
    what the call needs."""
    (B, Hkv, C, D), fmt = _quant_cache(kq, vq, k_scale, v_scale)
    shape = q.shape
    Hq = shape[1]
    if shape != (B, Hq, 1, D):
        _same("q", q, (B, Hq, 1, D))
    _same("out", out, shape, q.dtype)
    if isinstance(workspace, str):
        workspace = _made_on(stream, quant_decode_workspace, q, kq)
    cos, sin, rmax = _tables(rope, D)
    a, b, c, d, e, f, cs, sn, ws, st = _addresses(out, q, kq, vq, k_scale, v_scale, cos, sin,
                                                  workspace, status)
    _check("kvc_gqa_decode_quant", library().kvc_gqa_decode_quant(
        a, b, c, d, e, f, _lengths_of(lengths, B), B, Hq, Hkv, C, D, _dtype_code(q), fmt,
        int(windowed), local_window_size, scale, cs, sn, rmax, ws,
        0 if workspace is None else workspace.nbytes, st, _stream(stream)))
    return out


def kvc_page_bounds(bounds, bound_scale, k_pool, block_table, lengths, new_tokens, status=None,
                    stream=None):
    """Bounds of the pages that a step of new_tokens filled (include/kvc.h): bounds int8
    [pages, Hkv, 2, D], bound_scale float32 [pages, Hkv], k_pool [pages, Hkv, page_size, D]."""
    n_pages, Hkv, ps, D = k_pool.shape
    B, max_pages = block_table.shape
    _same("bounds", bounds, (n_pages, Hkv, 2, D), torch.int8)
    _same("bound_scale", bound_scale, (n_pages, Hkv), torch.float32)
    if block_table.dtype is not torch.int32:
        _same("block_table", block_table, (B, max_pages), torch.int32)
    a, b, c, d, st = _addresses(bounds, bound_scale, k_pool, block_table, status)
    _check("kvc_page_bounds", library().kvc_page_bounds(
        a, b, c, d, max_pages, n_pages, ps, _lengths_of(lengths, B), B, Hkv, new_tokens, D,
        _dtype_code(k_pool), st, _stream(stream)))


def sparse_workspace(q, k_pool, selected):
    """Workspace for kvc_gqa_decode_sparse."""
    B, Hq, _, D = q.shape
    n = library().kvc_gqa_decode_sparse_workspace_size(B, Hq, k_pool.shape[1], k_pool.shape[2],
                                                       selected.shape[2], D, _dtype_code(q))
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def kvc_gqa_decode_sparse(out, q, k_pool, v_pool, bounds, bound_scale, block_table, lengths,
                          selected, sink_pages=1, recent_pages=1, scale=0.0, rope=None,
                          workspace="auto", status=None, stream=None):
    """One-token attention over the pages that their bounds select (include/kvc.h); the pages
    taken go to selected, int32 [B, Hkv, n]."""
    pool = k_pool.shape
    n_pages, Hkv, ps, D = pool
    B, Hq, one, _ = shape = q.shape
    n, max_pages = selected.shape[-1], block_table.shape[-1]
    if one != 1 or shape[3] != D or q.dtype is not k_pool.dtype:
        _same("q", q, (B, Hq, 1, D), k_pool.dtype)
    _same("out", out, shape, q.dtype)
    _same("v_pool", v_pool, pool, q.dtype)
    _same("bounds", bounds, (n_pages, Hkv, 2, D), torch.int8)
    _same("bound_scale", bound_scale, (n_pages, Hkv), torch.float32)
    _same("block_table", block_table, (B, max_pages), torch.int32)
    _same("selected", selected, (B, Hkv, n), torch.int32)
    if isinstance(workspace, str):
        workspace = _made_on(stream, sparse_workspace, q, k_pool, selected)
    cos, sin, rmax = _tables(rope, D)
    a, b, c, d, e, f, g, h, cs, sn, ws, st = _addresses(
        out, q, k_pool, v_pool, bounds, bound_scale, block_table, selected, cos, sin, workspace,
        status)
    _check("kvc_gqa_decode_sparse", library().kvc_gqa_decode_sparse(
        a, b, c, d, e, f, g, max_pages, n_pages, ps, _lengths_of(lengths, B), B, Hq, Hkv, D,
        _dtype_code(q), n, sink_pages, recent_pages, h, scale, cs, sn, rmax, ws,
        0 if workspace is None else workspace.nbytes, st, _stream(stream)))
    return out


def tree_buffers(parents):
    """(mask, depth) for kvc_tree_mask: int32 [B, N, ceil(N / 32)] (the bit words) and [B, N]."""
    B, N = parents.shape
    return (torch.empty((B, N, (N + 31) // 32), dtype=torch.int32, device=parents.device),
            torch.empty((B, N), dtype=torch.int32, device=parents.device))


def kvc_tree_mask(parents, mask=None, depth=None, status=None, stream=None):
    """Ancestor bits and depths of the drafted trees parents, int32 [B, N] (include/kvc.h), in mask
    and depth where they are given."""
    B, N = parents.shape
    if mask is None or depth is None:
        made = _made_on(stream, tree_buffers, parents)
        if stream is not None:  # (the caller reads them on the current stream too)
            for t in made:
                t.record_stream(torch.cuda.current_stream())
        mask, depth = made[0] if mask is None else mask, made[1] if depth is None else depth
    if parents.dtype is not torch.int32:
        _same("parents", parents, (B, N), torch.int32)
    _same("mask", mask, (B, N, (N + 31) // 32), torch.int32)
    _same("depth", depth, (B, N), torch.int32)
    a, b, c, st = _addresses(parents, mask, depth, status)
    _check("kvc_tree_mask", library().kvc_tree_mask(a, B, N, b, c, st, _stream(stream)))
    return mask, depth


def _cache_rows(k_cache, v_cache, block_table, B):
    """(max_pages, pool pages, page_size, kv heads, capacity, D) of a contiguous cache
    [B, Hkv, C, D] (no block table) or of page pools [pages, Hkv, page_size, D]."""
    n, Hkv, rows, D = shape = k_cache.shape
    _same("v_cache", v_cache, shape, k_cache.dtype)
    if block_table is None:
        if n != B:
            _same("k_cache", k_cache, (B, Hkv, rows, D))
        return 0, 0, 0, Hkv, rows, D
    max_pages = block_table.shape[-1]
    _same("block_table", block_table, (B, max_pages), torch.int32)
    return max_pages, n, rows, Hkv, 0, D


def kvc_tree_append(k_cache, v_cache, new_k, new_v, depth, lengths, block_table=None, rope=None,
                    status=None, stream=None):
    """The drafted nodes' rows [B, Hkv, N, D] behind the cache, K rotated at P + depth
    (include/kvc.h)."""
    B, _, N, _ = shape = new_k.shape
    m, n, ps, Hkv, C, D = _cache_rows(k_cache, v_cache, block_table, B)
    _same("new_k", new_k, (B, Hkv, N, D), k_cache.dtype)
    _same("new_v", new_v, shape, k_cache.dtype)
    _same("depth", depth, (B, N), torch.int32)
    cos, sin, rmax = _tables(rope, D)
    a, b, c, d, e, table, cs, sn, st = _addresses(k_cache, v_cache, new_k, new_v, depth,
                                                  block_table, cos, sin, status)
    _check("kvc_tree_append", library().kvc_tree_append(
        a, b, c, d, e, table, m, n, ps, _lengths_of(lengths, B), B, Hkv, N, C, D,
        _dtype_code(k_cache), cs, sn, rmax, st, _stream(stream)))


def tree_workspace(q, k_cache):
    """Workspace for kvc_gqa_tree."""
    B, Hq, N, D = q.shape
    n = library().kvc_gqa_tree_workspace_size(B, Hq, k_cache.shape[1], N, D)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def kvc_gqa_tree(out, q, k_cache, v_cache, mask, depth, lengths, block_table=None,
                 local_window_size=0, scale=0.0, rope=None, workspace="auto", status=None,
                 stream=None):
    """Attention of the drafted nodes' queries [B, Hq, N, D] (include/kvc.h)."""
    B, Hq, N, _ = shape = q.shape
    m, n, ps, Hkv, C, D = _cache_rows(k_cache, v_cache, block_table, B)
    if shape[3] != D or q.dtype is not k_cache.dtype:
        _same("q", q, (B, Hq, N, D), k_cache.dtype)
    _same("out", out, shape, q.dtype)
    _same("mask", mask, (B, N, (N + 31) // 32), torch.int32)
    _same("depth", depth, (B, N), torch.int32)
    if isinstance(workspace, str):
        workspace = _made_on(stream, tree_workspace, q, k_cache)
    cos, sin, rmax = _tables(rope, D)
    a, b, c, d, e, f, table, cs, sn, ws, st = _addresses(
        out, q, k_cache, v_cache, mask, depth, block_table, cos, sin, workspace, status)
    _check("kvc_gqa_tree", library().kvc_gqa_tree(
        a, b, c, d, e, f, table, m, n, ps, _lengths_of(lengths, B), B, Hq, Hkv, N, C, D,
        _dtype_code(q), local_window_size, scale, cs, sn, rmax, ws,
        0 if workspace is None else workspace.nbytes, st, _stream(stream)))
    return out


def kvc_tree_commit(k_cache, v_cache, path, accepted, lengths, seqlens_k, nodes, block_table=None,
                    status=None, stream=None):
    """Keep the nodes path[b, :accepted[b]] of each tree (include/kvc.h): their rows follow the
    cache, seqlens_k holds the total so far minus one."""
    B, path_len = path.shape
    m, n, ps, Hkv, C, D = _cache_rows(k_cache, v_cache, block_table, B)
    if path.dtype is not torch.int32:
        _same("path", path, (B, path_len), torch.int32)
    _same("accepted", accepted, (B,), torch.int32)
    _same("seqlens_k", seqlens_k, (B,), torch.int32)
    a, b, c, d, e, table, st = _addresses(k_cache, v_cache, path, accepted, seqlens_k, block_table,
                                          status)
    _check("kvc_tree_commit", library().kvc_tree_commit(
        a, b, c, d, path_len, table, m, n, ps, _lengths_of(lengths, B), e, B, Hkv, nodes, C, D,
        _dtype_code(k_cache), st, _stream(stream)))
