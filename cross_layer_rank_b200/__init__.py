"""B200 (sm_100a) xKV hot path: thin Python binding of libxkv.so.

Every call below marshals torch tensors into the C ABI declared in
include/xkv.h and returns; all arithmetic runs in the library's CUDA kernels.
There is no CPU or PyTorch fallback: importing this package fails loudly when
libxkv.so has not been built (``python cross_layer_rank_b200/build.py``).

Functions keep the C names (xkv_compress_group, xkv_build_landmarks,
xkv_sr_attention_decode, xkv_full_reconstruct, xkv_ner, xkv_kv8_append, ...).  Tensors must be
CUDA tensors, contiguous, of the dtype named by the call; errors raise
XKVError carrying the library's status code.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libxkv.so")

XKV_OK = 0
XKV_ERR_INVALID_ARG = 1
XKV_ERR_UNSUPPORTED = 2
XKV_ERR_WORKSPACE = 3
XKV_ERR_CUDA = 4
XKV_ERR_NUMERICAL = 5
XKV_ERR_DEVICE_TIMEOUT = 6
XKV_F32 = 0
XKV_BF16 = 1

EXPORTS = (
    "xkv_status_string", "xkv_version", "xkv_get_device_status",
    "xkv_gram_workspace_size", "xkv_gram_accumulate",
    "xkv_compress_workspace_size", "xkv_compress_group",
    "xkv_factor_workspace_size", "xkv_factor_gram", "xkv_project_workspace_size", "xkv_project",
    "xkv_build_landmarks",
    "xkv_sr_workspace_size", "xkv_sr_attention_decode",
    "xkv_sr_attention_decode_noalloc",
    "xkv_xk_sr_workspace_size", "xkv_xk_sr_attention_decode",
    "xkv_xk_sr_host_workspace_size", "xkv_xk_sr_attention_decode_host_values",
    "xkv_sr_profile_enable", "xkv_sr_profile_read",
    "xkv_sr_append_workspace_size", "xkv_sr_append",
    "xkv_sr_scores", "xkv_sr_topk", "xkv_sr_partial_workspace_size", "xkv_sr_attention_partial",
    "xkv_merge_partials",
    "xkv_selftest_expired_wait",
    "xkv_full_reconstruct",
    "xkv_dense_workspace_size", "xkv_dense_attention_decode",
    "xkv_kv8_append", "xkv_kv8_workspace_size", "xkv_kv8_attention_decode", "xkv_kv8_evict",
    "xkv_ner_workspace_size", "xkv_ner", "xkv_energy_rank",
)


class XKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class SRParams(C.Structure):
    """Mirror of xkv_sr_params."""
    _fields_ = [("batch", C.c_int), ("n_q_heads", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("T", C.c_int64), ("rank_k", C.c_int), ("rank_v", C.c_int), ("chunk", C.c_int),
                ("topk", C.c_int), ("sink", C.c_int), ("recent", C.c_int), ("rope_theta", C.c_float),
                ("dtype", C.c_int), ("a_k_batch_stride", C.c_int64), ("a_v_batch_stride", C.c_int64),
                ("bt_k_batch_stride", C.c_int64), ("bt_v_batch_stride", C.c_int64),
                ("window_batch_stride", C.c_int64), ("landmark_capacity", C.c_int64)]


class AppendParams(C.Structure):
    """Mirror of xkv_append_params."""
    _fields_ = [("batch", C.c_int), ("group", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("chunk", C.c_int), ("sink", C.c_int), ("recent", C.c_int), ("rope_theta", C.c_float),
                ("dtype", C.c_int), ("T", C.c_int64), ("rank_k", C.c_int), ("rank_v", C.c_int),
                ("a_k_batch_stride", C.c_int64), ("a_v_batch_stride", C.c_int64),
                ("bt_k_batch_stride", C.c_int64), ("bt_v_batch_stride", C.c_int64),
                ("window_batch_stride", C.c_int64), ("landmark_capacity", C.c_int64)]


class ShardParams(C.Structure):
    """Mirror of xkv_sr_shard."""
    _fields_ = [("position_offset", C.c_int64), ("chunk_begin", C.c_int64)]


class DenseParams(C.Structure):
    """Mirror of xkv_dense_params."""
    _fields_ = [("batch", C.c_int), ("n_q_heads", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int),
                ("T", C.c_int64), ("dtype", C.c_int)]


class KV8Params(C.Structure):
    """Mirror of xkv_kv8_params."""
    _fields_ = [("batch", C.c_int), ("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("block", C.c_int),
                ("capacity", C.c_int64)]


class KV8Pointers(C.Structure):
    """Mirror of xkv_kv8_cache."""
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("weight", C.c_void_p), ("ids", C.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libxkv.so not built ({LIB_PATH}); run `python cross_layer_rank_b200/build.py`")
    lib = C.CDLL(LIB_PATH)
    vp, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
    sig = {
        "xkv_status_string": (C.c_char_p, [C.c_int]),
        "xkv_version": (C.c_int, []),
        "xkv_get_device_status": (C.c_int, [vp]),
        "xkv_gram_workspace_size": (C.c_int, [C.c_int, i64, C.c_int, C.c_int, C.POINTER(sz)]),
        "xkv_gram_accumulate": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, C.c_int, vp, vp, sz, vp]),
        "xkv_compress_workspace_size": (C.c_int, [C.c_int, i64, C.c_int, C.c_int, C.c_int, i64, C.c_int,
                                                  C.POINTER(sz)]),
        "xkv_compress_group": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, C.c_int, C.c_int, C.c_int, C.c_int, i64,
                                         C.c_uint64, vp, vp, vp, vp, vp, sz, vp]),
        "xkv_factor_workspace_size": (C.c_int, [C.c_int, C.c_int, i64, C.c_int, C.c_int, C.c_int, C.POINTER(sz)]),
        "xkv_factor_gram": (C.c_int, [vp, C.c_int, C.c_int, i64, C.c_int, C.c_int, C.c_int, C.c_int, C.c_uint64,
                                      vp, vp, vp, vp, sz, vp]),
        "xkv_project_workspace_size": (C.c_int, [C.c_int, C.c_int, C.c_int, C.POINTER(sz)]),
        "xkv_project": (C.c_int, [vp, C.c_int, i64, C.c_int, i64, C.c_int, vp, C.c_int, C.c_int, vp, i64, vp, sz,
                                  vp]),
        "xkv_build_landmarks": (C.c_int, [vp, i64, i64, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                                          C.c_float, vp, vp]),
        "xkv_sr_workspace_size": (C.c_int, [C.POINTER(SRParams), C.POINTER(sz)]),
        "xkv_sr_attention_decode": (C.c_int, [C.POINTER(SRParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                              vp]),
        "xkv_sr_attention_decode_noalloc": (C.c_int, [C.POINTER(SRParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                      vp]),
        "xkv_xk_sr_workspace_size": (C.c_int, [C.POINTER(SRParams), C.POINTER(sz)]),
        "xkv_xk_sr_attention_decode": (C.c_int, [C.POINTER(SRParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                                 vp]),
        "xkv_xk_sr_host_workspace_size": (C.c_int, [C.POINTER(SRParams), C.POINTER(sz)]),
        "xkv_xk_sr_attention_decode_host_values": (C.c_int, [C.POINTER(SRParams), vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                             vp, sz, vp]),
        "xkv_sr_scores": (C.c_int, [C.POINTER(SRParams), vp, vp, vp, i64, vp]),
        "xkv_sr_topk": (C.c_int, [vp, i64, C.c_int, i64, C.c_int, vp, vp]),
        "xkv_sr_partial_workspace_size": (C.c_int, [C.POINTER(SRParams), C.POINTER(sz)]),
        "xkv_sr_attention_partial": (C.c_int, [C.POINTER(SRParams), C.POINTER(ShardParams), vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp, vp, sz, vp]),
        "xkv_merge_partials": (C.c_int, [vp, vp, C.c_int, C.c_int, C.c_int, vp, vp]),
        "xkv_selftest_expired_wait": (C.c_int, [vp]),
        "xkv_sr_append_workspace_size": (C.c_int, [C.POINTER(AppendParams), C.POINTER(sz)]),
        "xkv_sr_append": (C.c_int, [C.POINTER(AppendParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, C.POINTER(C.c_int),
                                    vp, sz, vp]),
        "xkv_sr_profile_enable": (C.c_int, [C.c_int]),
        "xkv_sr_profile_read": (C.c_int, [C.POINTER(C.c_float)]),
        "xkv_full_reconstruct": (C.c_int, [vp, vp, i64, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_float,
                                           C.c_int, vp, vp]),
        "xkv_dense_workspace_size": (C.c_int, [C.POINTER(DenseParams), C.POINTER(sz)]),
        "xkv_dense_attention_decode": (C.c_int, [C.POINTER(DenseParams), vp, vp, vp, vp, vp, sz, vp]),
        "xkv_kv8_append": (C.c_int, [C.POINTER(KV8Params), C.POINTER(KV8Pointers), vp, vp, i64, C.c_int, vp, vp, i64,
                                     i64, vp]),
        "xkv_kv8_workspace_size": (C.c_int, [C.POINTER(KV8Params), C.c_int, C.POINTER(sz)]),
        "xkv_kv8_attention_decode": (C.c_int, [C.POINTER(KV8Params), C.POINTER(KV8Pointers), vp, C.c_int, C.c_int, vp,
                                               vp, C.c_int, vp, sz, vp]),
        "xkv_kv8_evict": (C.c_int, [C.POINTER(KV8Params), C.POINTER(KV8Pointers), vp, C.c_int, C.c_int, C.c_int, vp,
                                    vp]),
        "xkv_ner_workspace_size": (C.c_int, [C.c_int, C.c_int, C.POINTER(sz)]),
        "xkv_ner": (C.c_int, [vp, C.c_int, C.c_int, C.c_double, vp, vp, vp, vp, sz, vp]),
        "xkv_energy_rank": (C.c_int, [vp, C.c_int, C.c_int, C.c_double, vp, vp, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.xkv_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != XKV_OK:
        raise XKVError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return XKV_BF16
    if t == torch.float32:
        return XKV_F32
    raise ValueError(f"unsupported dtype {t}")


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Caller-owned scratch (256-byte aligned, as torch's allocator guarantees)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def _pool_of(stream, device):
    """Context in which torch allocates from the pool of the stream that a call runs on.  What a call allocates itself
    has to come from there: memory of the current stream's pool may still be used by earlier work on that stream, and
    goes to later work on it while the call runs."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        # 0 and 1 both name the default stream
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace for one call, which others may have once the call has returned."""
    with _pool_of(stream, device):
        return workspace(nbytes, device)


def _wsize(fn, *args) -> int:
    n = C.c_size_t(0)
    _check(fn(*args, C.byref(n)), fn.__name__)
    return int(n.value)


def get_device_status(stream=None) -> int:
    """Deferred device-side status (synchronises the stream), cleared on read."""
    return int(lib.xkv_get_device_status(_stream(stream)))


# ------------------------------------------------------------------- Gram
def xkv_gram_workspace_size(G: int, rows: int, d: int, dtype: torch.dtype) -> int:
    return _wsize(lib.xkv_gram_workspace_size, G, rows, d, dtype_code(dtype))


def xkv_gram_accumulate(layers: Sequence[torch.Tensor], C_out: torch.Tensor, ws: Optional[torch.Tensor] = None,
                        stream=None):
    """C_out += X^T X over X = [layers...] (each rows x d)."""
    G = len(layers)
    rows, d = layers[0].shape
    ldx = layers[0].stride(0)
    ptrs = (C.c_void_p * G)(*[t.data_ptr() for t in layers])
    nbytes = xkv_gram_workspace_size(G, rows, d, layers[0].dtype)
    if ws is None:
        ws = _scratch(nbytes, layers[0].device, stream)
    _check(lib.xkv_gram_accumulate(ptrs, G, rows, d, ldx, dtype_code(layers[0].dtype), _ptr(C_out), _ptr(ws),
                                   ws.numel(), _stream(stream)), "xkv_gram_accumulate")


# ------------------------------------------------------------ compression
def xkv_compress_workspace_size(G, T, d, rank, oversample, shard_rows, dtype: torch.dtype) -> int:
    return _wsize(lib.xkv_compress_workspace_size, G, T, d, rank, oversample, shard_rows, dtype_code(dtype))


def xkv_compress_group(layers: Sequence[torch.Tensor], rank: int, A: torch.Tensor, Bt: torch.Tensor,
                       iters: int = 8, oversample: int = 64, shard_rows: int = 8192, seed: int = 0x784B56,
                       eigvals: Optional[torch.Tensor] = None, gram_out: Optional[torch.Tensor] = None,
                       ws: Optional[torch.Tensor] = None, stream=None):
    """Cross-layer factorisation of one group into A (T x rank) and Bt (G d x rank)."""
    G = len(layers)
    T, d = layers[0].shape
    ldx = layers[0].stride(0)
    for t in layers:
        if t.shape != layers[0].shape or t.stride(0) != ldx or t.stride(1) != 1:
            raise ValueError("layers must share shape and row stride")
    dt = dtype_code(layers[0].dtype)
    nbytes = xkv_compress_workspace_size(G, T, d, rank, oversample, shard_rows, layers[0].dtype)
    if ws is None:
        ws = _scratch(nbytes, layers[0].device, stream)
    ptrs = (C.c_void_p * G)(*[t.data_ptr() for t in layers])
    _check(lib.xkv_compress_group(ptrs, G, T, d, ldx, dt, rank, iters, oversample, shard_rows, seed, _ptr(A),
                                  _ptr(Bt), _ptr(eigvals), _ptr(gram_out), _ptr(ws), ws.numel(), _stream(stream)),
           "xkv_compress_group")


def xkv_factor_workspace_size(G, d, rows, rank, oversample, dtype: torch.dtype) -> int:
    return _wsize(lib.xkv_factor_workspace_size, G, d, rows, rank, oversample, dtype_code(dtype))


def xkv_factor_gram(gram: torch.Tensor, G: int, d: int, rows: int, rank: int, Bt: torch.Tensor,
                    iters: int = 8, oversample: int = 64, seed: int = 0x784B56, Vr_out: Optional[torch.Tensor] = None,
                    eigvals: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None):
    """Top-r basis of a given (G d)^2 f32 Gram: Bt (G d x rank, Bt's dtype), optional f32 V_r and Ritz values."""
    nbytes = xkv_factor_workspace_size(G, d, rows, rank, oversample, Bt.dtype)
    if ws is None:
        ws = _scratch(nbytes, gram.device, stream)
    _check(lib.xkv_factor_gram(_ptr(gram), G, d, rows, dtype_code(Bt.dtype), rank, iters, oversample, seed, _ptr(Bt),
                               _ptr(Vr_out), _ptr(eigvals), _ptr(ws), ws.numel(), _stream(stream)), "xkv_factor_gram")


def xkv_project_workspace_size(G, d, rank) -> int:
    return _wsize(lib.xkv_project_workspace_size, G, d, rank)


def xkv_project(layers: Sequence[torch.Tensor], V: torch.Tensor, A: torch.Tensor, ws: Optional[torch.Tensor] = None,
                stream=None):
    """A = [layers...] V; A may be a row-strided view (rows of rank elements)."""
    G = len(layers)
    T, d = layers[0].shape
    ldx = layers[0].stride(0)
    for t in layers:
        if t.shape != layers[0].shape or t.stride(0) != ldx or t.stride(1) != 1:
            raise ValueError("layers must share shape and row stride")
    rank = V.shape[1]
    if A.shape[-1] != rank or A.stride(-1) != 1 or not A.is_cuda:
        raise ValueError("A must be T x rank with contiguous rows")
    if ws is None:
        ws = _scratch(xkv_project_workspace_size(G, d, rank), layers[0].device, stream)
    ptrs = (C.c_void_p * G)(*[t.data_ptr() for t in layers])
    _check(lib.xkv_project(ptrs, G, T, d, ldx, dtype_code(layers[0].dtype), _ptr(V), dtype_code(V.dtype), rank,
                           C.c_void_p(A.data_ptr()), A.stride(0), _ptr(ws), ws.numel(), _stream(stream)),
           "xkv_project")


# -------------------------------------------------------------- landmarks
def xkv_build_landmarks(K: torch.Tensor, n_kv_heads: int, head_dim: int, chunk: int, sink: int, recent: int,
                        rope_theta: float, out: torch.Tensor, stream=None):
    T = K.shape[0]
    if K.stride(1) != 1:
        raise ValueError("K rows must be contiguous")
    _check(lib.xkv_build_landmarks(C.c_void_p(K.data_ptr()), T, K.stride(0), n_kv_heads, head_dim,
                                   dtype_code(K.dtype), chunk, sink, recent, rope_theta, _ptr(out), _stream(stream)),
           "xkv_build_landmarks")


# -------------------------------------------------------------- SR decode
def sr_params(batch, n_q_heads, n_kv_heads, head_dim, T, rank_k, rank_v, chunk, topk, sink, recent, rope_theta,
              dtype: torch.dtype, a_k_batch_stride=None, a_v_batch_stride=None, bt_k_batch_stride=None,
              bt_v_batch_stride=None, window_batch_stride=0, landmark_capacity=0) -> SRParams:
    """Batch strides default to dense [B][T][r] A and per-batch dense [B][d][r] Bt;
    window and landmark strides default to the exact sizes (0)."""
    d = n_kv_heads * head_dim
    return SRParams(batch, n_q_heads, n_kv_heads, head_dim, T, rank_k, rank_v, chunk, topk, sink, recent,
                    float(rope_theta), dtype_code(dtype),
                    T * rank_k if a_k_batch_stride is None else a_k_batch_stride,
                    T * rank_v if a_v_batch_stride is None else a_v_batch_stride,
                    d * rank_k if bt_k_batch_stride is None else bt_k_batch_stride,
                    d * rank_v if bt_v_batch_stride is None else bt_v_batch_stride,
                    window_batch_stride, landmark_capacity)


def xkv_sr_workspace_size(p: SRParams) -> int:
    return _wsize(lib.xkv_sr_workspace_size, C.byref(p))


def _addr(t: Optional[torch.Tensor]):
    """Device address of a tensor whose layout the call's strides describe (a
    view such as one layer's rows of a group basis is accepted)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("expected contiguous rows")
    return C.c_void_p(t.data_ptr())


def xkv_sr_attention_decode(p: SRParams, q, A_K, Bt_K, A_V, Bt_V, landmarks, sr_K, sr_V, out,
                            sel_out=None, ws=None, stream=None):
    """One SR decode step of one layer; writes out [B][Hq][hd] f32 (and sel_out).
    A, Bt, landmarks and windows may be views: their strides come from p."""
    if ws is None:
        ws = _scratch(xkv_sr_workspace_size(p), q.device, stream)
    _check(lib.xkv_sr_attention_decode(C.byref(p), _ptr(q), _addr(A_K), _addr(Bt_K), _addr(A_V), _addr(Bt_V),
                                       _addr(landmarks), _addr(sr_K), _addr(sr_V), _ptr(out), _ptr(sel_out),
                                       _ptr(ws), ws.numel(), _stream(stream)), "xkv_sr_attention_decode")


SR_STATIC_SCRATCH_BYTES = 8 << 20


def xkv_sr_attention_decode_noalloc(p: SRParams, q, A_K, Bt_K, A_V, Bt_V, landmarks, sr_K, sr_V, out,
                                    sel_out=None, stream=None):
    """One SR decode step with the library's fixed scratch array (no workspace,
    no allocation); calls that overlap in time race on that array."""
    _check(lib.xkv_sr_attention_decode_noalloc(C.byref(p), _ptr(q), _ptr(A_K), _ptr(Bt_K), _ptr(A_V), _ptr(Bt_V),
                                               _ptr(landmarks), _ptr(sr_K), _ptr(sr_V), _ptr(out), _ptr(sel_out),
                                               _stream(stream)), "xkv_sr_attention_decode_noalloc")


def xk_sr_params(batch, n_q_heads, n_kv_heads, head_dim, T, rank_k, chunk, topk, sink, recent, rope_theta,
                 dtype: torch.dtype, a_k_batch_stride=None, v_batch_stride=None, bt_k_batch_stride=None) -> SRParams:
    """Parameters of the xK-SR mode: keys as in sr_params, values an uncompressed
    [B][T][d] cache (batch stride defaults to T d)."""
    d = n_kv_heads * head_dim
    return SRParams(batch, n_q_heads, n_kv_heads, head_dim, T, rank_k, head_dim, chunk, topk, sink, recent,
                    float(rope_theta), dtype_code(dtype),
                    T * rank_k if a_k_batch_stride is None else a_k_batch_stride,
                    T * d if v_batch_stride is None else v_batch_stride,
                    d * rank_k if bt_k_batch_stride is None else bt_k_batch_stride, 0, 0, 0)


def xkv_xk_sr_host_workspace_size(p: SRParams) -> int:
    return _wsize(lib.xkv_xk_sr_host_workspace_size, C.byref(p))


def xkv_xk_sr_attention_decode_host_values(p: SRParams, q, A_K, Bt_K, V_host: torch.Tensor, landmarks, sr_K, sr_V,
                                           out, sel_out=None, ws=None, stream=None):
    """xK-SR step with V [B][T][d] in pinned host memory (V_host.is_pinned());
    only the kept chunks' rows are read over the host link."""
    if V_host.is_cuda or not V_host.is_pinned():
        raise ValueError("V_host must be a pinned host tensor")
    if ws is None:
        ws = _scratch(xkv_xk_sr_host_workspace_size(p), q.device, stream)
    _check(lib.xkv_xk_sr_attention_decode_host_values(C.byref(p), _ptr(q), _addr(A_K), _addr(Bt_K),
                                                      C.c_void_p(V_host.data_ptr()), _addr(landmarks), _addr(sr_K),
                                                      _addr(sr_V), _ptr(out), _ptr(sel_out), _ptr(ws), ws.numel(),
                                                      _stream(stream)), "xkv_xk_sr_attention_decode_host_values")


def xkv_xk_sr_workspace_size(p: SRParams) -> int:
    return _wsize(lib.xkv_xk_sr_workspace_size, C.byref(p))


def xkv_xk_sr_attention_decode(p: SRParams, q, A_K, Bt_K, V, landmarks, sr_K, sr_V, out, sel_out=None, ws=None,
                               stream=None):
    """One xK-SR decode step of one layer (values read from the uncompressed V
    [B][T][d]); writes out [B][Hq][hd] f32 (and sel_out)."""
    if ws is None:
        ws = _scratch(xkv_xk_sr_workspace_size(p), q.device, stream)
    _check(lib.xkv_xk_sr_attention_decode(C.byref(p), _ptr(q), _ptr(A_K), _ptr(Bt_K), _ptr(V), _ptr(landmarks),
                                          _ptr(sr_K), _ptr(sr_V), _ptr(out), _ptr(sel_out), _ptr(ws), ws.numel(),
                                          _stream(stream)), "xkv_xk_sr_attention_decode")


def xkv_selftest_expired_wait(stream=None) -> None:
    """Launch the bounded-wait self-test (a wait that runs out after about one
    second); read the outcome with get_device_status()."""
    _check(lib.xkv_selftest_expired_wait(_stream(stream)), "xkv_selftest_expired_wait")


def xkv_sr_profile_enable(enable: bool = True) -> None:
    """Record CUDA events around the four launches of each later SR decode call."""
    _check(lib.xkv_sr_profile_enable(int(bool(enable))), "xkv_sr_profile_enable")


def xkv_sr_profile_read() -> list:
    """Durations (ms) of the last timed call: scores, top-k + window, attend, combine."""
    buf = (C.c_float * 4)()
    _check(lib.xkv_sr_profile_read(buf), "xkv_sr_profile_read")
    return [float(x) for x in buf]


# --------------------------------------------------- full reconstruction
def xkv_full_reconstruct(A, Bt, n_kv_heads: int, head_dim: int, apply_rope: bool, rope_theta: float, out,
                         stream=None):
    T, r = A.shape
    d = Bt.shape[0]
    _check(lib.xkv_full_reconstruct(_ptr(A), _ptr(Bt), T, r, d, n_kv_heads, head_dim, int(bool(apply_rope)),
                                    float(rope_theta), dtype_code(A.dtype), _ptr(out), _stream(stream)),
           "xkv_full_reconstruct")


def dense_params(batch, n_q_heads, n_kv_heads, head_dim, T, dtype: torch.dtype) -> DenseParams:
    return DenseParams(batch, n_q_heads, n_kv_heads, head_dim, T, dtype_code(dtype))


def xkv_dense_workspace_size(p: DenseParams) -> int:
    return _wsize(lib.xkv_dense_workspace_size, C.byref(p))


def xkv_dense_attention_decode(p: DenseParams, q, K, V, out, ws=None, stream=None):
    if ws is None:
        ws = _scratch(xkv_dense_workspace_size(p), q.device, stream)
    _check(lib.xkv_dense_attention_decode(C.byref(p), _ptr(q), _ptr(K), _ptr(V), _ptr(out), _ptr(ws), ws.numel(),
                                          _stream(stream)), "xkv_dense_attention_decode")


# ------------------------------------------------------- 8-bit KV cache
def kv8_params(batch, n_kv_heads, head_dim, block, capacity) -> KV8Params:
    return KV8Params(batch, n_kv_heads, head_dim, block, capacity)


class KV8Cache:
    """One layer's 8-bit KV cache: k, v [B][Hkv][capacity][hd] float8_e4m3fn, k_scale, v_scale
    [B][Hkv][capacity / block] f32 and, for eviction, weight (f32) and ids (int32) of the same
    shape as the scales.  The tensors stay the caller's; the object keeps them alive.  One may be replaced
    by another of its size (cache.k = cache.k[order]), and the next call takes that one; sizes stay, and so
    does each tensor's memory while it is part of the cache (no resize_, set_ or assignment to .data)."""

    TENSORS = ("k", "v", "k_scale", "v_scale", "weight", "ids")

    def __init__(self, k, v, k_scale, v_scale, weight=None, ids=None):
        self._take(k, v, k_scale, v_scale, weight, ids)

    def __setattr__(self, name, value):
        if name not in self.TENSORS:
            return object.__setattr__(self, name, value)
        held = {x: getattr(self, x) for x in self.TENSORS}
        if name in ("k", "v") and value.shape != held[name].shape:
            raise ValueError("a cache keeps its sizes: make a new KV8Cache")
        self._take(**{**held, name: value})

    def _take(self, k, v, k_scale, v_scale, weight, ids):
        for t, dt in ((k, torch.float8_e4m3fn), (v, torch.float8_e4m3fn), (k_scale, torch.float32),
                      (v_scale, torch.float32), (weight, torch.float32), (ids, torch.int32)):
            if t is None:
                continue
            if t.dtype != dt or t.dim() != (4 if dt == torch.float8_e4m3fn else 3):
                raise ValueError("k, v are 4-d float8_e4m3fn; scales and weight 3-d float32, ids 3-d int32")
            if t.device != k.device:
                raise ValueError("the tensors of a cache must be on one device")
        if v.shape != k.shape or k_scale.shape[:2] != k.shape[:2] or k_scale.shape[2] == 0 or \
                k.shape[2] % k_scale.shape[2] != 0:
            raise ValueError("k and v need one shape, and scales [B][Hkv][capacity / block]")
        for t in (v_scale, weight, ids):
            if t is not None and t.shape != k_scale.shape:
                raise ValueError("scales, weight and ids need one shape")
        tensors = (k, v, k_scale, v_scale, weight, ids)
        # a new object each time: a copy of this cache may share the old one
        pointers = KV8Pointers(*(_ptr(t) for t in tensors))
        self.__dict__.update(zip(self.TENSORS, tensors))
        self.index = k.get_device()
        self.sizes = (*k.shape, k.shape[2] // k_scale.shape[2])
        self.pointers = pointers

    @classmethod
    def empty(cls, p: KV8Params, device=None):
        """Room for p.capacity rows of every (sequence, KV head), with weight and ids."""
        device = device or "cuda"
        nblk = (p.batch, p.n_kv_heads, p.capacity // p.block)
        rows = (p.batch, p.n_kv_heads, p.capacity, p.head_dim)
        return cls(torch.empty(rows, dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(rows, dtype=torch.float8_e4m3fn, device=device),
                   *(torch.empty(nblk, dtype=torch.float32, device=device) for _ in range(3)),
                   torch.empty(nblk, dtype=torch.int32, device=device))


def _kv8_check(p: KV8Params, cache: KV8Cache, stream, *tensors):
    """What the C call cannot see: the cache is p's and everything lies on the current device.
    Returns the stream, the device's current one where none is given."""
    if cache.sizes != (p.batch, p.n_kv_heads, p.capacity, p.head_dim, p.block):
        raise ValueError("the cache's tensors do not have p's sizes")
    device = cache.index
    if device != torch.cuda.current_device():
        raise ValueError("the cache is not on the current CUDA device")
    for t in tensors:
        if t.get_device() != device:
            raise ValueError("all tensors must be on the cache's device")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _lens_ptr(p: KV8Params, t):
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != p.batch or not t.is_contiguous():
        raise ValueError("lengths and counts are contiguous int32 tensors of one entry per sequence")
    return t.data_ptr()


def xkv_kv8_append(p: KV8Params, cache: KV8Cache, lens, k_new, v_new, counts=None, stream=None):
    """Round new rows k_new, v_new [B][n][Hkv hd] (views with contiguous rows are accepted) into the
    cache at positions lens[b] ...; counts[b] <= n rows where given.  lens is not advanced."""
    stream = _kv8_check(p, cache, stream, lens, k_new, v_new, lens if counts is None else counts)
    shape, strides, dtype = k_new.shape, k_new.stride(), k_new.dtype
    if len(shape) != 3 or v_new.shape != shape or v_new.dtype != dtype or shape[0] != p.batch or \
            shape[2] != p.n_kv_heads * p.head_dim:
        raise ValueError("k_new and v_new are [B][n][Hkv hd] of one dtype")
    # a stride over one row or one sequence is not used, and torch leaves it open
    other = v_new.stride()
    if strides[2] != 1 or other[2] != 1 or (strides[1] != other[1] and shape[1] > 1) or \
            (strides[0] != other[0] and shape[0] > 1):
        raise ValueError("k_new and v_new need contiguous rows and the same strides")
    _check(lib.xkv_kv8_append(p, cache.pointers, _lens_ptr(p, lens), _lens_ptr(p, counts), shape[1],
                              dtype_code(dtype), k_new.data_ptr(), v_new.data_ptr(),
                              strides[1] if shape[1] > 1 else shape[2], strides[0] if shape[0] > 1 else 0,
                              stream), "xkv_kv8_append")


def xkv_kv8_workspace_size(p: KV8Params, n_q_heads: int) -> int:
    return _wsize(lib.xkv_kv8_workspace_size, C.byref(p), n_q_heads)


def xkv_kv8_attention_decode(p: KV8Params, cache: KV8Cache, lens, q, out, accumulate: bool = False, ws=None,
                             stream=None):
    """One decode step over the 8-bit cache; writes out [B][Hq][hd] f32 and, with accumulate, adds
    every block's attention weight to cache.weight."""
    raw = _kv8_check(p, cache, stream, lens, q, out, lens if ws is None else ws)
    if ws is None:
        ws = _scratch(xkv_kv8_workspace_size(p, q.shape[1] if q.dim() == 3 else 0), q.device, stream)
    shape = q.shape
    if len(shape) != 3 or shape[0] != p.batch or shape[2] != p.head_dim or out.shape != shape or \
            out.dtype != torch.float32:
        raise ValueError("q is [B][Hq][hd] and out the same shape in float32")
    if not (q.is_contiguous() and out.is_contiguous() and ws.is_contiguous()):
        raise ValueError("expected contiguous tensors")
    _check(lib.xkv_kv8_attention_decode(p, cache.pointers, _lens_ptr(p, lens), shape[1], dtype_code(q.dtype),
                                        q.data_ptr(), out.data_ptr(), 1 if accumulate else 0, ws.data_ptr(),
                                        ws.numel() * ws.element_size(), raw), "xkv_kv8_attention_decode")


def xkv_kv8_evict(p: KV8Params, cache: KV8Cache, lens, budget: int, sink: int, recent: int, lens_out, stream=None):
    """Keep `budget` blocks of every longer sequence and KV head: the first `sink`, the newest
    `recent` and those with the most weight.  lens_out receives the lengths after it."""
    stream = _kv8_check(p, cache, stream, lens, lens_out)
    _check(lib.xkv_kv8_evict(p, cache.pointers, _lens_ptr(p, lens), budget, sink, recent, _lens_ptr(p, lens_out),
                             stream), "xkv_kv8_evict")


# -------------------------------------------------------------------- NER
def xkv_ner_workspace_size(n: int, block: int) -> int:
    return _wsize(lib.xkv_ner_workspace_size, n, block)


def xkv_ner(gram: torch.Tensor, block: int, ner_out, erank_out=None, rank_out=None, rank_rel_tol: float = 1e-9,
            ws=None, stream=None):
    n = gram.shape[0]
    if ws is None:
        ws = _scratch(xkv_ner_workspace_size(n, block), gram.device, stream)
    _check(lib.xkv_ner(_ptr(gram), n, block, rank_rel_tol, _ptr(ner_out), _ptr(erank_out), _ptr(rank_out), _ptr(ws),
                       ws.numel(), _stream(stream)), "xkv_ner")


def xkv_energy_rank(gram, block: int, energy: float = 0.95, rank_out=None, lambda_out=None, ws=None, stream=None):
    """Per diagonal block: the rank keeping `energy` of the block's eigenvalue
    total, and optionally its eigenvalues in descending order."""
    n = gram.shape[0]
    count = n // block
    if rank_out is None:
        with _pool_of(stream, gram.device):
            rank_out = torch.empty(count, dtype=torch.int32, device=gram.device)
    if ws is None:
        ws = _scratch(xkv_ner_workspace_size(n, block), gram.device, stream)
    _check(lib.xkv_energy_rank(_ptr(gram), n, block, float(energy), _ptr(rank_out), _ptr(lambda_out), _ptr(ws),
                               ws.numel(), _stream(stream)), "xkv_energy_rank")
    return rank_out


# ------------------------------------------------------- multi-step decode
def decode_layout(T: int, sink: int, recent: int, chunk: int):
    """(n_mid, window rows) of a cache of T tokens built by prefill plus appends:
    n0 = T - sink - recent; n_mid = n0 // chunk; the window holds recent + n0 % chunk rows."""
    n0 = T - sink - recent
    return n0 // chunk, recent + n0 % chunk


def append_params(batch, group, n_kv_heads, head_dim, chunk, sink, recent, rope_theta, dtype: torch.dtype, T,
                  rank_k, rank_v, a_k_batch_stride, a_v_batch_stride, bt_k_batch_stride, bt_v_batch_stride,
                  window_batch_stride, landmark_capacity) -> AppendParams:
    return AppendParams(batch, group, n_kv_heads, head_dim, chunk, sink, recent, float(rope_theta), dtype_code(dtype),
                        T, rank_k, rank_v, a_k_batch_stride, a_v_batch_stride, bt_k_batch_stride, bt_v_batch_stride,
                        window_batch_stride, landmark_capacity)


def xkv_sr_append(p: AppendParams, k_new, v_new, win_K, win_V, Bt_K, Bt_V, A_K, A_V, landmarks, ws=None,
                  stream=None) -> bool:
    """Append one token per layer (lists of G tensors); returns True when a chunk was rolled."""
    G = p.group
    arr = lambda ts: (C.c_void_p * G)(*[t.data_ptr() for t in ts])
    n = C.c_size_t(0)
    _check(lib.xkv_sr_append_workspace_size(C.byref(p), C.byref(n)), "xkv_sr_append_workspace_size")
    if ws is None:
        ws = _scratch(n.value, A_K.device, stream)
    rolled = C.c_int(0)
    _check(lib.xkv_sr_append(C.byref(p), arr(k_new), arr(v_new), arr(win_K), arr(win_V), _ptr(Bt_K), _ptr(Bt_V),
                             _ptr(A_K), _ptr(A_V), arr(landmarks), C.byref(rolled), _ptr(ws), ws.numel(),
                             _stream(stream)), "xkv_sr_append")
    return bool(rolled.value)


# ------------------------------------------------------- token sharding
def xkv_sr_scores(p: SRParams, q, landmarks, scores, stream=None):
    """scores [B][Hkv][ld] f32 (ld >= n_mid, a multiple of 4): the local chunk scores."""
    _check(lib.xkv_sr_scores(C.byref(p), _ptr(q), _addr(landmarks), _addr(scores), scores.stride(-2),
                             _stream(stream)), "xkv_sr_scores")


def xkv_sr_topk(scores, n: int, k: int, sel_out, stream=None):
    """Exact top-k of each row of scores [..., ld] over its first n entries."""
    rows = scores.numel() // scores.shape[-1]
    _check(lib.xkv_sr_topk(_addr(scores), scores.stride(-2), rows, n, k, _ptr(sel_out), _stream(stream)),
           "xkv_sr_topk")


def xkv_sr_attention_partial(p: SRParams, shard: ShardParams, sel, q, A_K, Bt_K, A_V, Bt_V, sr_K, sr_V, out, ml_out,
                             ws=None, stream=None):
    """Attention of this device's token slice for the global selection sel; out
    normalised by its own sum, ml_out = (M, L) per (sequence, query head)."""
    if ws is None:
        n = C.c_size_t(0)
        _check(lib.xkv_sr_partial_workspace_size(C.byref(p), C.byref(n)), "xkv_sr_partial_workspace_size")
        ws = _scratch(n.value, q.device, stream)
    _check(lib.xkv_sr_attention_partial(C.byref(p), C.byref(shard), _ptr(sel), _ptr(q), _addr(A_K), _addr(Bt_K),
                                        _addr(A_V), _addr(Bt_V), _addr(sr_K), _addr(sr_V), _ptr(out), _ptr(ml_out),
                                        _ptr(ws), ws.numel(), _stream(stream)), "xkv_sr_attention_partial")


def xkv_merge_partials(o, ml, out, stream=None):
    """o [R][rows][hd], ml [R][rows][2] -> out [rows][hd] (the exact softmax combination)."""
    R, rows, hd = o.shape[0], o.numel() // (o.shape[0] * o.shape[-1]), o.shape[-1]
    _check(lib.xkv_merge_partials(_ptr(o), _ptr(ml), R, rows, hd, _ptr(out), _stream(stream)), "xkv_merge_partials")

