"""tiled_attention_forward_gb300 -- Python binding of libfattn.

Exact scaled-dot-product attention forward on one GB300 (sm_103a), computed
FlashAttention-2 style by hand-written CUDA kernels behind a C ABI
(``include/fattn.h``).  This module only marshals arguments: it turns torch
tensors into device pointers and the current CUDA stream into a
``cudaStream_t`` and calls the library.  Every step of the computation runs in
the library's kernels; there is no fallback of any kind.  If ``libfattn.so``
has not been built (``python -m tiled_attention_forward_gb300.build``), every
call raises ``FattnLibraryMissing``.

    import torch, tiled_attention_forward_gb300 as fattn
    o, lse = fattn.fwd(q, k, v, causal=True)     # q,k,v: [B,H,N,D] cuda tensors
"""
import ctypes
import importlib.util
import math
import os

import torch

__all__ = ["fwd", "fwd_host", "bwd", "bwd_host", "bwd_workspace_bytes", "fwd_unfused", "fwd_unfused_static", "unfused_workspace_bytes",
           "UNFUSED_STATIC_BYTES", "plan", "get_device_status", "selftest_wait_timeout",
           "status_string", "library_path", "load", "FattnError", "FattnLibraryMissing",
           "DTYPE_CODES", "STATUS", "cache_append", "cache_append_kv4", "decode", "decode_kv4",
           "decode_workspace_bytes", "KV4_GROUP", "fwd_packed", "packed_workspace_bytes"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libfattn.so")

DTYPE_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
STATUS = {0: "FATTN_OK", 1: "FATTN_ERR_INVALID_ARG", 2: "FATTN_ERR_UNSUPPORTED",
          3: "FATTN_ERR_MISALIGNED", 4: "FATTN_ERR_CUDA", 5: "FATTN_ERR_TIMEOUT",
          6: "FATTN_ERR_NO_DEVICE", 7: "FATTN_ERR_INTERNAL"}
UNFUSED_STATIC_BYTES = 64 << 20  # FATTN_UNFUSED_STATIC_BYTES
KV4_GROUP = 32  # elements of a 4-bit cache row that share one (scale, zero)
PLAN_FIELDS = ("path", "grid_x", "grid_y", "threads", "smem_bytes", "tasks", "kv_tiles",
               "rows_per_task", "keys_per_kv_tile")


class FattnError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s returned %s (%d)" % (where, STATUS.get(code, "?"), code))


class FattnLibraryMissing(RuntimeError):
    pass


_lib = None


def library_path():
    return _LIB_PATH


def load():
    """Load libfattn.so (once).  Raises FattnLibraryMissing if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise FattnLibraryMissing(
            "libfattn.so is not built at %s; run `python -m tiled_attention_forward_gb300.build`"
            % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, f32, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
    lib.fattn_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, f32, ci, ci, vp]
    lib.fattn_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, ci, ci, vp]
    lib.fattn_fwd_f32_rowwise.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, f32, ci, vp]
    lib.fattn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   i64, i64, i64, i64, f32, ci, ci, vp]
    lib.fattn_fwd_unfused.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, f32, ci,
                                      ci, vp]
    lib.fattn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, f32,
                              ci, ci, vp]
    lib.fattn_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                  i64, f32, ci, ci, vp]
    lib.fattn_bwd_host.argtypes = [vp] * 19 + [i64, i64, i64, i64, i64, f32, ci, ci, vp]
    lib.fattn_bwd_workspace_bytes.argtypes = [i64, i64, i64]
    lib.fattn_bwd_workspace_bytes.restype = i64
    lib.fattn_fwd_unfused_static.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, f32, ci, ci, vp]
    lib.fattn_unfused_workspace_bytes.argtypes = [i64, i64, i64]
    lib.fattn_unfused_workspace_bytes.restype = i64
    lib.fattn_plan.argtypes = [i64, i64, i64, i64, ci, ci, ci, ctypes.POINTER(i64)]
    lib.fattn_plan_head_group.argtypes = [i64, i64, i64, i64, i64, ctypes.POINTER(i64)]
    lib.fattn_packed_workspace_bytes.argtypes = [i64, i64]
    lib.fattn_packed_workspace_bytes.restype = i64
    lib.fattn_fwd_packed.argtypes = [vp] * 8 + [i64] * 6 + [f32, ci, ci, vp]
    lib.fattn_cache_append.argtypes = [vp] * 8 + [i64] * 3 + [vp] * 4 + [i64] * 2 + [ci] + [i64] * 4 + [ci, vp]
    lib.fattn_cache_append_kv4.argtypes = ([vp] * 11 + [i64] * 2 + [vp] * 4 + [i64] * 2 + [ci] * 2 + [i64] * 4 +
                                           [ci, vp])
    lib.fattn_decode_workspace_bytes.argtypes = [i64] * 5
    lib.fattn_decode_workspace_bytes.restype = i64
    lib.fattn_decode.argtypes = ([vp] * 6 + [i64] * 3 + [vp, i64, vp, vp] + [i64] * 6 + [f32, ci, vp])
    lib.fattn_decode_kv4.argtypes = ([vp] * 8 + [i64] * 2 + [vp, i64, vp, vp] + [i64] * 6 + [f32, ci, vp])
    lib.fattn_get_device_status.argtypes = [vp]
    lib.fattn_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.fattn_status_string.argtypes = [ci]
    lib.fattn_status_string.restype = ctypes.c_char_p
    lib.fattn_version.argtypes = []
    for f in ("fattn_fwd", "fattn_fwd_gqa", "fattn_fwd_host", "fattn_fwd_unfused", "fattn_bwd", "fattn_bwd_gqa", "fattn_bwd_host",
              "fattn_fwd_unfused_static", "fattn_plan", "fattn_plan_head_group",
              "fattn_fwd_packed", "fattn_cache_append", "fattn_cache_append_kv4", "fattn_decode", "fattn_decode_kv4",
              "fattn_get_device_status",
              "fattn_selftest_wait_timeout", "fattn_version"):
        getattr(lib, f).restype = ci
    _lib = lib
    return lib


def status_string(code):
    return load().fattn_status_string(int(code)).decode()


def _check(code, where):
    if code != 0:
        raise FattnError(code, where)


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _default_scale(D):
    # 1/sqrt(D) rounded once to fp32, the value the library multiplies by.
    return float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32).item())


def _check_qkv(q, k, v, allow_gqa=False):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, D]")
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape")
    if allow_gqa:
        B, H, N, D = q.shape
        if k.shape[0] != B or k.shape[2] != N or k.shape[3] != D:
            raise ValueError("k, v must be [B, Hkv, N, D] with q's B, N and D")
    elif k.shape != q.shape:
        raise ValueError("q, k, v must have the same shape")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same dtype")
    if q.dtype not in DTYPE_CODES:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous row-major [B, H, N, D]")


def fwd(q, k, v, causal=False, scale=None, out=None, lse=None, return_lse=True, stream=None):
    """Attention forward on CUDA tensors.

    q: [B, H, N, D]; k, v: [B, Hkv, N, D] with H a multiple of Hkv
    (grouped-query attention when Hkv < H); contiguous CUDA tensors of one
    dtype (float32, float16 or bfloat16), D in {64, 128}.  Returns (o, lse): o has q's dtype
    and shape; lse is float32 [B, H, N] (natural-log log-sum-exp of the
    scaled scores), or None when return_lse is False.  ``out`` / ``lse`` may
    be given to write into existing tensors.  Enqueued on ``stream`` (default:
    torch's current stream); no synchronisation.
    """
    _check_qkv(q, k, v, allow_gqa=True)
    if not q.is_cuda:
        raise ValueError("fwd needs CUDA tensors; see fwd_host for host buffers")
    B, H, N, D = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = _default_scale(D)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lse_ptr = lse.data_ptr() if (return_lse and lse is not None) else None
    lib = load()
    with torch.cuda.device(q.device):
        if Hkv == H:
            rc = lib.fattn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse_ptr,
                               B, H, N, D, float(scale), int(bool(causal)), DTYPE_CODES[q.dtype],
                               _stream_handle(stream))
        else:
            rc = lib.fattn_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                   lse_ptr, B, H, Hkv, N, D, float(scale), int(bool(causal)),
                                   DTYPE_CODES[q.dtype], _stream_handle(stream))
    _check(rc, "fattn_fwd" if Hkv == H else "fattn_fwd_gqa")
    return out, (lse if return_lse else None)


def fwd_f32_rowwise(q, k, v, causal=False, scale=None, out=None, lse=None, return_lse=True,
                    stream=None):
    """fp32 forward through the one-query-row-per-thread CUDA-core kernel
    (fattn_fwd_f32_rowwise).  q, k, v: contiguous float32 CUDA tensors of one
    shape [B, H, N, D]; otherwise as fwd."""
    _check_qkv(q, k, v)
    if not q.is_cuda or q.dtype != torch.float32:
        raise ValueError("fwd_f32_rowwise needs float32 CUDA tensors")
    B, H, N, D = q.shape
    if scale is None:
        scale = _default_scale(D)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lse_ptr = lse.data_ptr() if (return_lse and lse is not None) else None
    lib = load()
    with torch.cuda.device(q.device):
        rc = lib.fattn_fwd_f32_rowwise(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                       lse_ptr, B, H, N, D, float(scale), int(bool(causal)),
                                       _stream_handle(stream))
    _check(rc, "fattn_fwd_f32_rowwise")
    return out, (lse if return_lse else None)


def fwd_host(q_host, k_host, v_host, q_dev, k_dev, v_dev, o_dev, o_host, lse_dev=None,
             lse_host=None, causal=False, scale=None, stream=None):
    """End-to-end forward from host tensors: host->device copies, the kernels and
    the device->host copies of O (and LSE) are enqueued by the library, in up
    to four groups of heads so that copies overlap the kernels (two internal
    copy streams, joined to ``stream`` with events).  Host tensors should be
    pinned; the caller synchronises ``stream``."""
    _check_qkv(q_host, k_host, v_host)
    B, H, N, D = q_host.shape
    if scale is None:
        scale = _default_scale(D)
    lib = load()
    with torch.cuda.device(q_dev.device):
        rc = lib.fattn_fwd_host(q_host.data_ptr(), k_host.data_ptr(), v_host.data_ptr(),
                                o_host.data_ptr(),
                                lse_host.data_ptr() if lse_host is not None else None,
                                q_dev.data_ptr(), k_dev.data_ptr(), v_dev.data_ptr(),
                                o_dev.data_ptr(),
                                lse_dev.data_ptr() if lse_dev is not None else None,
                                B, H, N, D, float(scale), int(bool(causal)),
                                DTYPE_CODES[q_host.dtype], _stream_handle(stream))
    _check(rc, "fattn_fwd_host")


def bwd_workspace_bytes(B, H, N):
    """Bytes of workspace bwd needs (fp32 per-row statistics, rows padded to 128)."""
    return int(load().fattn_bwd_workspace_bytes(int(B), int(H), int(N)))


def bwd(q, k, v, o, lse, dout, causal=False, scale=None, dq=None, dk=None, dv=None,
        workspace=None, stream=None):
    """Attention backward on CUDA tensors: gradients of sum(dout * O) where
    (o, lse) is what ``fwd`` returned for (q, k, v).  bfloat16 / float16;
    q, o, dout [B, H, N, D]; k, v [B, Hkv, N, D] with H a multiple of Hkv
    (grouped-query attention when Hkv < H: dk, dv are summed over each
    group); lse float32 [B, H, N].  Returns (dq, dk, dv) in the input dtype
    with q's and k's shapes.  ``workspace`` (a CUDA uint8 tensor of at least
    ``bwd_workspace_bytes(B, H, N)`` bytes) is allocated here when None."""
    _check_qkv(q, k, v, allow_gqa=True)
    for t in (o, dout):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError("o and dout must be contiguous with q's shape and dtype")
    if lse.dtype != torch.float32 or tuple(lse.shape) != tuple(q.shape[:3]) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [B, H, N]")
    if not q.is_cuda:
        raise ValueError("bwd needs CUDA tensors")
    B, H, N, D = q.shape
    Hkv = k.shape[1]
    if scale is None:
        scale = _default_scale(D)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(max(bwd_workspace_bytes(B, H, N), 16), dtype=torch.uint8,
                                device=q.device)
    lib = load()
    with torch.cuda.device(q.device):
        rc = lib.fattn_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                               dv.data_ptr(), workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), B, H, Hkv, N, D,
                               float(scale), int(bool(causal)), DTYPE_CODES[q.dtype],
                               _stream_handle(stream))
    _check(rc, "fattn_bwd_gqa")
    return dq, dk, dv


def bwd_host(hosts, devs, grads_host, grads_dev, workspace, causal=False, scale=None, stream=None):
    """End-to-end backward from host tensors (multi-head, bfloat16 / float16).

    hosts = (q, k, v, o, dout, lse) pinned host tensors; devs = the matching
    device buffers; grads_host / grads_dev = (dq, dk, dv) host / device
    buffers; workspace as for ``bwd``.  Copies in, the backward and copies
    out are enqueued by the library in groups of heads that overlap; the
    caller synchronises ``stream``."""
    q = hosts[0]
    B, H, N, D = q.shape
    if scale is None:
        scale = _default_scale(D)
    ptrs = [t.data_ptr() for t in hosts] + [t.data_ptr() for t in grads_host] + \
        [t.data_ptr() for t in devs] + [t.data_ptr() for t in grads_dev] + [workspace.data_ptr()]
    lib = load()
    with torch.cuda.device(devs[0].device):
        rc = lib.fattn_bwd_host(*ptrs, workspace.numel() * workspace.element_size(), B, H, N, D,
                                float(scale), int(bool(causal)), DTYPE_CODES[q.dtype],
                                _stream_handle(stream))
    _check(rc, "fattn_bwd_host")


def unfused_workspace_bytes(B, H, N):
    """Bytes of workspace fwd_unfused needs (S fp32 then P 16-bit, rows padded to 8)."""
    return int(load().fattn_unfused_workspace_bytes(int(B), int(H), int(N)))


def fwd_unfused(q, k, v, causal=False, scale=None, out=None, lse=None, workspace=None,
                return_lse=True, stream=None):
    """The materialising comparator: S = scale Q K^T and P = softmax(S) are
    written to ``workspace`` (a CUDA uint8 tensor of at least
    ``unfused_workspace_bytes(B, H, N)`` bytes; allocated here when None) and
    O = P V is computed from P.  bfloat16 / float16 only, q, k, v of one shape.
    Returns (o, lse) like ``fwd``."""
    _check_qkv(q, k, v)
    if not q.is_cuda:
        raise ValueError("fwd_unfused needs CUDA tensors")
    B, H, N, D = q.shape
    if scale is None:
        scale = _default_scale(D)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    need = unfused_workspace_bytes(B, H, N)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    lse_ptr = lse.data_ptr() if (return_lse and lse is not None) else None
    lib = load()
    with torch.cuda.device(q.device):
        rc = lib.fattn_fwd_unfused(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                   lse_ptr, workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), B, H, N, D,
                                   float(scale), int(bool(causal)), DTYPE_CODES[q.dtype],
                                   _stream_handle(stream))
    _check(rc, "fattn_fwd_unfused")
    return out, (lse if return_lse else None)


def fwd_unfused_static(q, k, v, causal=False, scale=None, out=None, lse=None, return_lse=True,
                       stream=None):
    """``fwd_unfused`` with the library's fixed per-device workspace of
    UNFUSED_STATIC_BYTES (no workspace argument, nothing allocated by the
    library).  Calls on one device must not overlap in time (one stream)."""
    _check_qkv(q, k, v)
    if not q.is_cuda:
        raise ValueError("fwd_unfused_static needs CUDA tensors")
    B, H, N, D = q.shape
    if scale is None:
        scale = _default_scale(D)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lse_ptr = lse.data_ptr() if (return_lse and lse is not None) else None
    lib = load()
    with torch.cuda.device(q.device):
        rc = lib.fattn_fwd_unfused_static(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                          lse_ptr, B, H, N, D, float(scale), int(bool(causal)),
                                          DTYPE_CODES[q.dtype], _stream_handle(stream))
    _check(rc, "fattn_fwd_unfused_static")
    return out, (lse if return_lse else None)


# ---------------------------------------------------------------------------
# Serving: rows by strides, paged caches
# ---------------------------------------------------------------------------
# These calls are short (a decode step's kernels take a few microseconds), so
# their tensors are checked and turned into the library's arguments by
# _fattn_binding (csrc/binding.cpp); the functions below only fill in what the
# caller left out.
_BINDING_PATH = os.path.join(_HERE, "_fattn_binding.so")
_fast = None


def _binding():
    global _fast
    if _fast is None:
        load()
        if not os.path.exists(_BINDING_PATH):
            raise FattnLibraryMissing(
                "_fattn_binding.so is not built at %s; run `python -m tiled_attention_forward_gb300.build`"
                % _BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_fattn_binding", _BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _fast = module
    return _fast


def _handle(stream, t):
    """The stream's handle (-1: torch's current one on the tensors' device)."""
    if stream is None:
        return -1
    if stream.device_index != t.get_device():
        raise ValueError("the stream must be one of %s" % t.device)
    return stream.cuda_stream


def _new(shape, dtype, like, stream, make=torch.empty):
    """A tensor for a call on `stream`, beside `like`: allocated (and filled) in
    that stream's order, so that what held its memory before is done with it,
    and so that a workspace can be dropped when the call returns."""
    if not like.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _dims(name, t, n):
    if t.dim() != n:
        raise ValueError("%s must have %d dimensions" % (name, n))
    return t.shape


def packed_workspace_bytes(B, T):
    """Bytes of workspace ``fwd_packed`` needs for B sequences of T tokens in all."""
    return int(load().fattn_packed_workspace_bytes(int(B), int(T)))


def fwd_packed(q, k, v, cu_seqlens, causal=True, scale=None, out=None, lse=None, workspace=None, return_lse=True,
               stream=None):
    """Attention of sequences of different lengths packed one after the other.

    q: [T, H, D]; k, v: [T, Hkv, D] with H a multiple of Hkv; float16 or
    bfloat16 CUDA tensors, D in {64, 128}, any token and head strides (slices
    of one projection), last dimension contiguous.  cu_seqlens: int32 [B + 1]
    on the GPU; sequence b is tokens cu_seqlens[b] .. cu_seqlens[b+1] - 1 and
    attends to itself alone.  Returns (o, lse): o [T, H, D], lse float32
    [H, T] or None; rows of no sequence are left as they were in ``out`` and
    ``lse`` (zero where those are allocated here).  ``workspace``: a CUDA uint8
    tensor of at least ``packed_workspace_bytes(B, T)`` bytes (allocated here
    when None); calls running at the same time need one each."""
    if scale is None or out is None or workspace is None or (return_lse and lse is None):
        T, H, D = _dims("q", q, 3)
        scale = _default_scale(D) if scale is None else scale
        if out is None:
            out = _new((T, H, D), q.dtype, q, stream, torch.zeros)
        if return_lse and lse is None:
            lse = _new((H, T), torch.float32, q, stream, torch.zeros)
        if workspace is None:
            need = packed_workspace_bytes(_dims("cu_seqlens", cu_seqlens, 1)[0] - 1, T)
            workspace = _new(max(need, 16), torch.uint8, q, stream)
    if not return_lse:
        lse = None
    rc = _binding().fwd_packed(q, k, v, cu_seqlens, out, lse, workspace, scale, 1 if causal else 0, _handle(stream, q))
    if rc != 0:
        raise FattnError(rc, "fattn_fwd_packed")
    return out, lse


def cache_append(k, v, k_pages, v_pages, slots, pos=None, cos=None, sin=None, interleaved=False, q=None,
                 q_out=None, k_out=None, stream=None):
    """Appends T new tokens to a 16-bit paged cache, rotating k and q by position.

    k, v: [T, Hkv, D] CUDA tensors (float16 or bfloat16, D in {64, 128}), q
    (optional): [T, H, D]; any token and head strides (slices of one
    projection), last dimension contiguous.  k_pages, v_pages: [pages, Hkv,
    page_size, D], page_size a multiple of 16, one stride between pages.
    slots: int64 [T] = page * page_size + place, all different; a negative
    slot skips its token.  pos: int32 [T], rows of cos and sin, float32
    [max_pos, rot/2] (rot a multiple of 16, the first rot elements of a row
    turn: element i with i + rot/2, or 2i with 2i+1 when ``interleaved``);
    without cos and sin nothing turns.  Returns (q_out, k_out): q rotated (None
    without q; allocated here when None) and, where ``k_out`` is given, k as
    the cache holds it.  ``q_out`` may be q itself.  An index out of range is
    skipped and reported by ``get_device_status``."""
    if q is not None and q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    rc = _binding().cache_append(k, v, k_pages, v_pages, slots, pos, cos, sin, 1 if interleaved else 0, q, q_out, k_out,
                                 _handle(stream, k))
    if rc != 0:
        raise FattnError(rc, "fattn_cache_append")
    return q_out, k_out


def cache_append_kv4(k, v, k_codes, k_scales, v_codes, v_scales, slots, pos=None, cos=None, sin=None,
                     interleaved=False, q=None, q_out=None, k_out=None, v_out=None, held=False, stream=None):
    """``cache_append`` into a 4-bit cache: k_codes, v_codes uint8 [pages, Hkv,
    page_size, D/2]; k_scales, v_scales float16 [pages, Hkv, page_size, D/32,
    2] = (scale, zero) of each group of 32 elements (the nibble order is in
    include/fattn.h).  Returns (q_out, k_out, v_out); where given, k_out and
    v_out receive the rotated k and v, or with ``held`` the values that the
    cache now stands for."""
    if q is not None and q_out is None:
        q_out = _new(q.shape, q.dtype, q, stream)
    rc = _binding().cache_append_kv4(k, v, k_codes, k_scales, v_codes, v_scales, slots, pos, cos, sin,
                                     1 if interleaved else 0, q, q_out, k_out, v_out, 1 if held else 0,
                                     _handle(stream, k))
    if rc != 0:
        raise FattnError(rc, "fattn_cache_append_kv4")
    return q_out, k_out, v_out


def decode_workspace_bytes(B, H, Nq, D, Hkv=None):
    """Bytes of workspace ``decode`` and ``decode_kv4`` need (whatever the
    sequences' lengths); without ``Hkv`` what is enough for any number of K/V
    heads (the most query rows a K/V head take the most)."""
    return int(load().fattn_decode_workspace_bytes(int(B), int(H), int(1 if Hkv is None else Hkv), int(Nq), int(D)))


def _decode_defaults(q, Hkv, scale, out, lse, workspace, return_lse, stream):
    B, H, Nq, D = _dims("q", q, 4)
    if scale is None:
        scale = _default_scale(D)
    if out is None:
        out = _new((B, H, Nq, D), q.dtype, q, stream)
    if return_lse and lse is None:
        lse = _new((B, H, Nq), torch.float32, q, stream)
    if workspace is None:
        workspace = _new(max(decode_workspace_bytes(B, H, Nq, D, Hkv), 16), torch.uint8, q, stream)
    return scale, out, lse, workspace


def decode(q, k_pages, v_pages, block_table, seq_lens, scale=None, out=None, lse=None, workspace=None,
           return_lse=True, stream=None):
    """Attention of the last Nq tokens of each sequence over a 16-bit paged
    cache that already holds them (``cache_append``).

    q: [B, H, Nq, D] (any strides, last dimension contiguous); k_pages,
    v_pages: [pages, Hkv, page_size, D] with H a multiple of Hkv; block_table:
    int32 [B, pages per sequence]; seq_lens: int32 [B], cached tokens of each
    sequence.  Token i of the Nq sees keys 0 .. seq_lens[b] - Nq + i.  Returns
    (o, lse) like ``fwd``: o [B, H, Nq, D], lse float32 [B, H, Nq]; a row
    without keys gives o = 0, lse = -inf.  ``workspace``: a CUDA uint8 tensor
    of at least ``decode_workspace_bytes`` bytes (allocated here when None);
    calls running at the same time need one each."""
    if scale is None or out is None or workspace is None or (return_lse and lse is None):
        scale, out, lse, workspace = _decode_defaults(q, _dims("k_pages", k_pages, 4)[1], scale, out, lse, workspace,
                                                      return_lse, stream)
    if not return_lse:
        lse = None
    rc = _binding().decode(q, k_pages, v_pages, block_table, seq_lens, scale, out, lse, workspace, _handle(stream, q))
    if rc != 0:
        raise FattnError(rc, "fattn_decode")
    return out, lse


def decode_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, scale=None, out=None, lse=None,
               workspace=None, return_lse=True, stream=None):
    """``decode`` over a 4-bit cache (``cache_append_kv4``)."""
    if scale is None or out is None or workspace is None or (return_lse and lse is None):
        scale, out, lse, workspace = _decode_defaults(q, _dims("k_codes", k_codes, 4)[1], scale, out, lse, workspace,
                                                      return_lse, stream)
    if not return_lse:
        lse = None
    rc = _binding().decode_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, scale, out, lse, workspace,
                               _handle(stream, q))
    if rc != 0:
        raise FattnError(rc, "fattn_decode_kv4")
    return out, lse


def plan(B, H, N, D, causal=False, dtype=torch.bfloat16, num_sms=0):
    """Launch plan (host only when num_sms > 0) as a dict; see fattn_plan."""
    out = (ctypes.c_int64 * 9)()
    code = DTYPE_CODES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    rc = load().fattn_plan(B, H, N, D, int(bool(causal)), code, int(num_sms), out)
    _check(rc, "fattn_plan")
    return dict(zip(PLAN_FIELDS, list(out)))


def plan_head_group(B, H, N, D, Hkv=None):
    """Query heads per group of the causal task order (host only); see
    fattn_plan_head_group."""
    out = ctypes.c_int64(0)
    rc = load().fattn_plan_head_group(B, H, H if Hkv is None else Hkv, N, D, ctypes.byref(out))
    _check(rc, "fattn_plan_head_group")
    return out.value


def get_device_status(stream=None):
    """Synchronise the stream and return (and clear) the device error word."""
    return load().fattn_get_device_status(_stream_handle(stream))


def selftest_wait_timeout(timeout_ns, stream=None):
    rc = load().fattn_selftest_wait_timeout(int(timeout_ns), _stream_handle(stream))
    _check(rc, "fattn_selftest_wait_timeout")
