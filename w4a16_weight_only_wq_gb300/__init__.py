"""Thin Python binding of libwq (include/wq.h): argument marshalling only.

Every step of the path (packing, dequant, GEMM) runs in the library's CUDA
kernels; this module converts torch tensors to device pointers and the
current torch stream to a ``cudaStream_t``.  There is no fallback: if the
library is missing, importing the binding raises.

Two layers:
  * ``wq_*`` functions with the C names and C arguments (integer device
    pointers, sizes, stream handle) -- the ABI as-is;
  * tensor helpers (``pack_symmetric``, ``pack_codes``, ``unpack``,
    ``gemm_w4a16``, ``gemm_w8a16``, ``kv4_append``, ``kv4_attention``,
    ``token_logprobs``, ...) that allocate outputs with torch and call the
    ABI on the current stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libwq.so")

WQ_OK = 0
WQ_ERR_NULL = 1
WQ_ERR_SHAPE = 2
WQ_ERR_UNSUPPORTED = 3
WQ_ERR_ALIGN = 4
WQ_ERR_CUDA = 5
WQ_ERR_DEVICE_TIMEOUT = 6
WQ_ERR_DEVICE_BOUNDS = 7
WQ_F32 = 0
WQ_BF16 = 1
WQ_ACT_NONE = 0
WQ_ACT_SILU = 1
GROUP = 128

EXPORTED = (
    "wq_packed_words", "wq_packed_bytes", "wq_pack_symmetric", "wq_pack_codes", "wq_unpack", "wq_dequantize",
    "wq_import_packed_nk",
    "wq_gemm_w4a16", "wq_gemm_w8a16", "wq_mlp_w4a16", "wq_mlp_w8a16", "wq_swa_attention",
    "wq_last_device_error",
    "wq_clear_device_error", "wq_status_string", "wq_debug_set_wait_limit_ns",
    "wq_debug_force_timeout", "wq_gemm_regime", "wq_debug_set_split",
    "wq_set_programmatic_launch", "wq_last_cuda_error", "wq_debug_force_regime",
    "wq_kv4_pool_bytes", "wq_kv4_locate", "wq_debug_kv4_sequence", "wq_debug_kv4_seventh",
    "wq_kv4_append", "wq_kv4_read",
    "wq_kv4_workspace_bytes", "wq_kv4_attention", "wq_logprobs_workspace_bytes", "wq_token_logprobs",
)


class _CacheStruct(ctypes.Structure):  # wq_kv4_cache
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("group", ctypes.c_int)]


class _BatchStruct(ctypes.Structure):  # wq_kv4_batch
    _fields_ = [("page_table", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("num_seqs", ctypes.c_int64), ("num_tokens", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("max_q", ctypes.c_int64)]


class _RowsStruct(ctypes.Structure):  # wq_rows
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class WQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {status_string(status)}"
        if status == WQ_ERR_CUDA:
            msg += f" ({wq_last_cuda_error()})"
        super().__init__(msg)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libwq.so not found at {LIB_PATH}; build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    C, B, R = (ctypes.POINTER(t) for t in (_CacheStruct, _BatchStruct, _RowsStruct))  # a struct passes its address
    sig = {
        "wq_packed_words": ([I, I64, I64], ctypes.c_size_t),
        "wq_packed_bytes": ([I, I64, I64], ctypes.c_size_t),
        "wq_pack_symmetric": ([P, I, I64, I64, I, I, P, P, P, P], I),
        "wq_pack_codes": ([P, I64, I64, I, P, P], I),
        "wq_unpack": ([P, I, I64, I64, P, P], I),
        "wq_dequantize": ([P, P, I, I64, I64, I, P, P], I),
        "wq_import_packed_nk": ([P, P, I, I64, I64, I, P, P, P], I),
        "wq_gemm_w4a16": ([P, P, P, P, I64, I64, I64, I, P], I),
        "wq_gemm_w8a16": ([P, P, P, P, I64, I64, I64, I, P], I),
        "wq_mlp_w4a16": ([P, P, P, P, P, P, P, I64, I64, I64, I64, I, I, P], I),
        "wq_mlp_w8a16": ([P, P, P, P, P, P, P, I64, I64, I64, I64, I, I, P], I),
        "wq_swa_attention": ([P, P, P, P, I64, I64, I64, I64, I64, I64, P], I),
        "wq_last_device_error": ([], I),
        "wq_clear_device_error": ([], I),
        "wq_status_string": ([I], ctypes.c_char_p),
        "wq_debug_set_wait_limit_ns": ([ctypes.c_uint64], None),
        "wq_debug_force_timeout": ([I], None),
        "wq_gemm_regime": ([I, I64, I64, I64], I),
        "wq_debug_set_split": ([I], None),
        "wq_set_programmatic_launch": ([I], None),
        "wq_last_cuda_error": ([], ctypes.c_char_p),
        "wq_debug_force_regime": ([I], None),
        "wq_kv4_pool_bytes": ([I64, I, I, I, I], ctypes.c_size_t),
        "wq_kv4_locate": ([C, I64, I, I, I, I, P, P], I64),
        "wq_debug_kv4_sequence": ([I64, I64, I64, I64, I64, P], I),
        "wq_debug_kv4_seventh": ([P, P, I64], None),
        "wq_kv4_append": ([C, B, R, R, I64, R, R, P, I64, I, I, P, P], I),
        "wq_kv4_read": ([C, B, R, R, P], I),
        "wq_kv4_workspace_bytes": ([I64, I, I], ctypes.c_size_t),
        "wq_kv4_attention": ([C, B, R, R, I64, ctypes.c_float, I64, P, ctypes.c_size_t, P], I),
        "wq_logprobs_workspace_bytes": ([I64, I64, I], ctypes.c_size_t),
        "wq_token_logprobs": ([P, I, I64, I64, I64, P, P, I, P, P, P, P, P, P, ctypes.c_size_t, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


# ------------------------------------------------------------ raw C ABI ---
def wq_packed_words(bits: int, K: int, N: int) -> int:
    return int(_lib.wq_packed_words(bits, K, N))


def wq_packed_bytes(bits: int, K: int, N: int) -> int:
    return int(_lib.wq_packed_bytes(bits, K, N))


def wq_pack_symmetric(W, wdt, K, N, bits, group, scales_in, scales_out, packed,
                      stream) -> int:
    return _lib.wq_pack_symmetric(W, wdt, K, N, bits, group, scales_in,
                                  scales_out, packed, stream)


def wq_pack_codes(codes, K, N, bits, packed, stream) -> int:
    return _lib.wq_pack_codes(codes, K, N, bits, packed, stream)


def wq_unpack(packed, bits, K, N, codes, stream) -> int:
    return _lib.wq_unpack(packed, bits, K, N, codes, stream)


def wq_import_packed_nk(qweight, scales_nk, bits, K, N, group, packed, scales_out,
                        stream) -> int:
    return _lib.wq_import_packed_nk(qweight, scales_nk, bits, K, N, group, packed,
                                    scales_out, stream)


def wq_dequantize(packed, scales, bits, K, N, group, W, stream) -> int:
    return _lib.wq_dequantize(packed, scales, bits, K, N, group, W, stream)


def wq_gemm_w4a16(X, Wp, scales, Y, M, N, K, group, stream) -> int:
    return _lib.wq_gemm_w4a16(X, Wp, scales, Y, M, N, K, group, stream)


def wq_gemm_w8a16(X, Wp, scales, Y, M, N, K, group, stream) -> int:
    return _lib.wq_gemm_w8a16(X, Wp, scales, Y, M, N, K, group, stream)


def wq_last_device_error() -> int:
    return int(_lib.wq_last_device_error())


def wq_clear_device_error() -> int:
    return int(_lib.wq_clear_device_error())


def wq_last_cuda_error() -> str:
    return _lib.wq_last_cuda_error().decode()


def status_string(status: int) -> str:
    return _lib.wq_status_string(int(status)).decode()


def wq_debug_set_wait_limit_ns(ns: int) -> None:
    _lib.wq_debug_set_wait_limit_ns(int(ns))


def wq_debug_force_timeout(mode) -> None:
    """0 off, 1 a wait on a barrier nothing completes, 2 data waits that
    give up (see include/wq.h)."""
    _lib.wq_debug_force_timeout(int(mode))


def wq_gemm_regime(bits: int, M: int, N: int, K: int) -> int:
    return int(_lib.wq_gemm_regime(bits, M, N, K))


def wq_debug_set_split(cs: int) -> None:
    _lib.wq_debug_set_split(int(cs))


def wq_debug_force_regime(regime: int) -> None:
    """0 small-M kernel, 1 tensor-core kernel, -1 automatic."""
    _lib.wq_debug_force_regime(int(regime))


def wq_set_programmatic_launch(on: bool) -> None:
    _lib.wq_set_programmatic_launch(1 if on else 0)


# ---------------------------------------------------------- tensor layer ---
def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _check(status: int, what: str) -> None:
    if status != WQ_OK:
        raise WQError(status, what)


def pack_symmetric(W: torch.Tensor, bits: int, scales: torch.Tensor | None = None,
                   stream=None):
    """Round W [K,N] (fp32/bf16) onto the group-128 grid and pack it.
    Returns (packed int32 words, bf16 scales [K/128, N])."""
    K, N = W.shape
    wdt = {torch.float32: WQ_F32, torch.bfloat16: WQ_BF16}.get(W.dtype)
    if wdt is None:
        raise ValueError("W must be float32 or bfloat16")
    words = wq_packed_words(bits, K, N)
    if words == 0:
        raise WQError(WQ_ERR_SHAPE, "pack_symmetric")
    packed = torch.empty(words, dtype=torch.int32, device=W.device)
    s_out = torch.empty((K // GROUP, N), dtype=torch.bfloat16, device=W.device)
    _check(wq_pack_symmetric(_ptr(W), wdt, K, N, bits, GROUP, _ptr(scales),
                             _ptr(s_out), _ptr(packed), _stream(stream)),
           "wq_pack_symmetric")
    return packed, s_out


def pack_codes(codes: torch.Tensor, bits: int, stream=None) -> torch.Tensor:
    """Interleave int8 codes [K,N] into packed words."""
    K, N = codes.shape
    words = wq_packed_words(bits, K, N)
    if words == 0:
        raise WQError(WQ_ERR_SHAPE, "pack_codes")
    packed = torch.empty(words, dtype=torch.int32, device=codes.device)
    _check(wq_pack_codes(_ptr(codes), K, N, bits, _ptr(packed), _stream(stream)),
           "wq_pack_codes")
    return packed


def unpack(packed: torch.Tensor, K: int, N: int, bits: int,
           stream=None) -> torch.Tensor:
    codes = torch.empty((K, N), dtype=torch.int8, device=packed.device)
    _check(wq_unpack(_ptr(packed), bits, K, N, _ptr(codes), _stream(stream)),
           "wq_unpack")
    return codes


def import_packed_nk(qweight: torch.Tensor, scales_nk: torch.Tensor, bits: int,
                     stream=None):
    """Repack an output-channel-major checkpoint layer (qweight int32
    [N, K*bits/32], scales [N, K/128] bf16) into this library's layout:
    returns (packed words, scales [K/128, N])."""
    if scales_nk.dtype != torch.bfloat16:
        raise ValueError("scales must be bfloat16")
    N, G = scales_nk.shape
    K = G * GROUP
    packed = torch.empty((wq_packed_words(bits, K, N),), dtype=torch.int32,
                         device=qweight.device)
    scales = torch.empty((G, N), dtype=torch.bfloat16, device=qweight.device)
    _check(wq_import_packed_nk(_ptr(qweight), _ptr(scales_nk), bits, K, N, GROUP,
                               _ptr(packed), _ptr(scales), _stream(stream)),
           "wq_import_packed_nk")
    return packed, scales


def dequantize(packed: torch.Tensor, scales: torch.Tensor, bits: int,
               stream=None) -> torch.Tensor:
    """The effective bf16 weight [K, N] = bf16(s * q) of a packed layer."""
    if scales.dtype != torch.bfloat16:
        raise ValueError("scales must be bfloat16")
    K, N = scales.shape[0] * GROUP, scales.shape[1]
    W = torch.empty((K, N), dtype=torch.bfloat16, device=packed.device)
    _check(wq_dequantize(_ptr(packed), _ptr(scales), bits, K, N, GROUP, _ptr(W),
                         _stream(stream)), "wq_dequantize")
    return W


def _gemm(fn, name, X, Wp, scales, N, Y=None, stream=None):
    M, K = X.shape
    if X.dtype != torch.bfloat16 or scales.dtype != torch.bfloat16:
        raise ValueError("X and scales must be bfloat16")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _check(fn(_ptr(X), _ptr(Wp), _ptr(scales), _ptr(Y), M, N, K, GROUP,
              _stream(stream)), name)
    return Y


def gemm_w4a16(X: torch.Tensor, Wp: torch.Tensor, scales: torch.Tensor,
               N: int | None = None, Y: torch.Tensor | None = None, stream=None):
    """Y[M,N] = X[M,K] . dequant(Wp INT4, scales)."""
    N = scales.shape[1] if N is None else N
    return _gemm(wq_gemm_w4a16, "wq_gemm_w4a16", X, Wp, scales, N, Y, stream)


def gemm_w8a16(X: torch.Tensor, Wp: torch.Tensor, scales: torch.Tensor,
               N: int | None = None, Y: torch.Tensor | None = None, stream=None):
    """Y[M,N] = X[M,K] . dequant(Wp INT8, scales)."""
    N = scales.shape[1] if N is None else N
    return _gemm(wq_gemm_w8a16, "wq_gemm_w8a16", X, Wp, scales, N, Y, stream)


def wq_mlp_w4a16(X, Wu, Su, Wd, Sd, H, Y, M, K, N1, N2, group, act, stream) -> int:
    return _lib.wq_mlp_w4a16(X, Wu, Su, Wd, Sd, H, Y, M, K, N1, N2, group, act, stream)


def wq_mlp_w8a16(X, Wu, Su, Wd, Sd, H, Y, M, K, N1, N2, group, act, stream) -> int:
    return _lib.wq_mlp_w8a16(X, Wu, Su, Wd, Sd, H, Y, M, K, N1, N2, group, act, stream)


_ACTS = {"none": WQ_ACT_NONE, "silu": WQ_ACT_SILU}


def mlp(X: torch.Tensor, Wu: torch.Tensor, Su: torch.Tensor, Wd: torch.Tensor,
        Sd: torch.Tensor, bits: int, act: str = "none", H: torch.Tensor | None = None,
        Y: torch.Tensor | None = None, stream=None):
    """The two projections of an MLP block: H = act(bf16(X . Wu)),
    Y = bf16(H . Wd).  Returns (H, Y)."""
    M, K = X.shape
    N1, N2 = Su.shape[1], Sd.shape[1]
    if X.dtype != torch.bfloat16 or Su.dtype != torch.bfloat16 or Sd.dtype != torch.bfloat16:
        raise ValueError("X and scales must be bfloat16")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    if H is None:
        H = torch.empty((M, N1), dtype=torch.bfloat16, device=X.device)
    if Y is None:
        Y = torch.empty((M, N2), dtype=torch.bfloat16, device=X.device)
    fn, name = (wq_mlp_w4a16, "wq_mlp_w4a16") if bits == 4 else (wq_mlp_w8a16, "wq_mlp_w8a16")
    _check(fn(_ptr(X), _ptr(Wu), _ptr(Su), _ptr(Wd), _ptr(Sd), _ptr(H), _ptr(Y), M, K, N1, N2,
              GROUP, _ACTS[act], _stream(stream)), name)
    return H, Y


def wq_swa_attention(Q, K, V, O, B, Hq, Hkv, D, T, window, stream) -> int:
    return _lib.wq_swa_attention(Q, K, V, O, B, Hq, Hkv, D, T, window, stream)


def swa_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, window: int,
                  O: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The drafter's symmetric sliding-window attention.  Q [B, Hq, 128],
    K and V [Hkv, T, 128] (bf16); query b sits at position T - B + b and
    sees keys within window // 2 of it (window 0: all keys).  Returns
    O [B, Hq, 128]."""
    if Q.dtype != torch.bfloat16 or K.dtype != torch.bfloat16 or V.dtype != torch.bfloat16:
        raise ValueError("Q, K and V must be bfloat16")
    B, Hq, D = Q.shape
    Hkv, T, _ = K.shape
    if O is None:
        O = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=Q.device)
    _check(wq_swa_attention(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), B, Hq, Hkv, D, T, window,
                            _stream(stream)), "wq_swa_attention")
    return O


# ------------------------------------- the 4-bit key/value cache, raw ABI ---
# Structs are passed as ctypes objects (or None); see include/wq.h.
def wq_kv4_pool_bytes(num_pages, page_size, Hkv, D, group) -> int:
    return int(_lib.wq_kv4_pool_bytes(num_pages, page_size, Hkv, D, group))


def wq_kv4_locate(cache, page, head, slot, dim, value):
    """(byte offset or -1, nibble, scale offset) of one cached number."""
    nibble, scale = ctypes.c_int(-1), ctypes.c_int64(-1)
    off = _lib.wq_kv4_locate(cache, page, head, slot, dim, value, ctypes.byref(nibble),
                             ctypes.byref(scale))
    return int(off), nibble.value, scale.value


def wq_debug_kv4_sequence(cu0, cu1, kv_len, num_tokens, capacity):
    """(clamped?, first token, new tokens, cached tokens)."""
    out = (ctypes.c_int64 * 3)()
    bad = _lib.wq_debug_kv4_sequence(cu0, cu1, kv_len, num_tokens, capacity, out)
    return (int(bad), *out)


def wq_debug_kv4_seventh(values, out, n) -> None:
    """Host addresses of n floats each."""
    _lib.wq_debug_kv4_seventh(values, out, n)


def wq_kv4_append(cache, batch, Q, Q_out, Hq, K, V, rope, max_pos, rot_dim, interleaved, positions,
                  stream) -> int:
    return _lib.wq_kv4_append(cache, batch, Q, Q_out, Hq, K, V, rope, max_pos, rot_dim, interleaved, positions,
                              stream)


def wq_kv4_read(cache, batch, K, V, stream) -> int:
    return _lib.wq_kv4_read(cache, batch, K, V, stream)


def wq_kv4_workspace_bytes(Hq, Hkv, D) -> int:
    return int(_lib.wq_kv4_workspace_bytes(Hq, Hkv, D))


def wq_kv4_attention(cache, batch, Q, O, Hq, scale, window, workspace, workspace_bytes, stream) -> int:
    return _lib.wq_kv4_attention(cache, batch, Q, O, Hq, scale, window, workspace, workspace_bytes, stream)


def wq_logprobs_workspace_bytes(T, V, k) -> int:
    return int(_lib.wq_logprobs_workspace_bytes(T, V, k))


def wq_token_logprobs(logits, dt, T, V, row_stride, tokens, inv_temperature, k, logprob, entropy, rank,
                      top_ids, top_logprobs, workspace, workspace_bytes, stream) -> int:
    return _lib.wq_token_logprobs(logits, dt, T, V, row_stride, tokens, inv_temperature, k, logprob, entropy,
                                  rank, top_ids, top_logprobs, workspace, workspace_bytes, stream)


# --------------------------------- the 4-bit key/value cache, tensor layer ---
# These helpers run before every launch of a decoding step, so they ask torch
# for little: the device's number, and the current stream's handle directly.
def _on(stream):
    """Outputs and workspaces that a call allocates belong to the stream it runs on."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch_stream(stream, device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else int(stream.cuda_stream)


def _same_device(what: str, device: int, *tensors) -> None:
    """All tensors of a call on the current GPU: the library launches there."""
    if device != torch._C._cuda_getDevice():
        raise ValueError(f"{what}: tensors must live on the current GPU")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{what}: tensors must live on the current GPU")


def _rows(t: torch.Tensor, what: str, T: int, heads: int, D: int) -> _RowsStruct:
    """A [T, heads, D] bf16 tensor, its last dimension contiguous, as rows."""
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{what} must be bfloat16")
    if t.shape != (T, heads, D):
        raise ValueError(f"{what} must be [{T}, {heads}, {D}], got {list(t.shape)}")
    by_token, by_head, by_dim = t.stride()
    if by_dim != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    # the stride of a dimension of size one says nothing
    return _RowsStruct(t.data_ptr(), by_token if T > 1 else 0, by_head if heads > 1 else 0)


def _new_rows(T: int, heads: int, D: int, device, stream):
    """A new [T, heads, D] bf16 tensor, and it as rows."""
    t = _empty((T, heads, D), torch.bfloat16, device, stream)
    return t, _RowsStruct(t.data_ptr(), heads * D, D)


def _heads(t: torch.Tensor, what: str) -> int:
    if t.dim() != 3:
        raise ValueError(f"{what} must be [tokens, heads, dimensions], got {list(t.shape)}")
    return t.shape[1]


class Kv4Cache:
    """A pool of pages of 4-bit keys and values (layout: include/wq.h).  ``pool`` is the uint8 tensor
    [num_pages, Hkv, block]; the cache keeps no other state, so pages are handed out by the caller's tables."""

    def __init__(self, num_pages: int, Hkv: int, D: int, page_size: int, group: int, pool: torch.Tensor):
        self.num_pages, self.Hkv, self.D, self.page_size, self.group = num_pages, Hkv, D, page_size, group
        self.pool, self.device, self._index = pool, pool.device, pool.get_device()
        self._struct = _CacheStruct(pool.data_ptr(), num_pages, page_size, Hkv, D, group)


def kv4_cache(num_pages: int, Hkv: int, D: int, page_size: int = 64, group: int = 128,
              pool: torch.Tensor | None = None, device="cuda") -> Kv4Cache:
    """A cache of ``num_pages`` pages of ``page_size`` tokens; ``pool``: an existing pool of its size."""
    n = wq_kv4_pool_bytes(num_pages, page_size, Hkv, D, group)
    if n == 0:
        raise WQError(WQ_ERR_SHAPE, "kv4_cache")
    if pool is None:
        pool = torch.zeros((num_pages, Hkv, n // num_pages // Hkv), dtype=torch.uint8, device=device)
    elif pool.dtype != torch.uint8 or pool.numel() != n or not pool.is_contiguous() or not pool.is_cuda:
        raise ValueError(f"pool must be a contiguous uint8 GPU tensor of {n} bytes")
    return Kv4Cache(num_pages, Hkv, D, page_size, group, pool)


class Kv4Batch:
    """One step's sequences: which pages they have, where their new tokens lie and how long they are.  Holds the
    tensors; the kernels read what they contain when they run."""

    def __init__(self, page_table, cu_q, kv_len, tokens: int, max_q: int):
        self.page_table, self.cu_q, self.kv_len, self.tokens, self.max_q = page_table, cu_q, kv_len, tokens, max_q
        self._struct = _BatchStruct(page_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), page_table.shape[0],
                                    tokens, page_table.shape[1], max_q)


def kv4_batch(page_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, tokens: int,
              max_q: int = 0) -> Kv4Batch:
    """page_table int32 [B, pages], cu_q int32 [B + 1] (prefix sums of the new tokens), kv_len int32 [B] (cached
    tokens, the new ones included), ``tokens`` new tokens in all, at most ``max_q`` of one sequence.  ``max_q`` picks the
    attention's kernel; 0 (not known) is guessed from the number of tokens and sequences, rightly for single tokens, but
    blocks of several sequences run up to a fifth slower than with it.  Every layer of a step uses the same batch."""
    for name, t, shape in (("page_table", page_table, None), ("cu_q", cu_q, (page_table.shape[0] + 1,)),
                           ("kv_len", kv_len, (page_table.shape[0],))):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
        if (shape is None and t.dim() != 2) or (shape is not None and tuple(t.shape) != shape):
            raise ValueError(f"{name} has shape {list(t.shape)}")
    _same_device("kv4_batch", page_table.get_device(), cu_q, kv_len)
    return Kv4Batch(page_table, cu_q, kv_len, int(tokens), int(max_q))


def rope_table(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_pos, rot_dim / 2, 2]: cos and sin of position * base^(-2i / rot_dim), computed in 64 bits."""
    freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq[None, :]
    return torch.stack([angle.cos(), angle.sin()], dim=-1).float()


def kv4_append(cache: Kv4Cache, batch: Kv4Batch, K: torch.Tensor, V: torch.Tensor, Q: torch.Tensor | None = None,
               rope: torch.Tensor | None = None, interleaved: bool = False, positions: torch.Tensor | None = None,
               Q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rotate Q and K by position, write K and V into the cache in 4 bits, return the rotated queries.  Q [T, Hq, D],
    K and V [T, Hkv, D] bf16 (views of a fused projection's output are fine); rope [max_pos, rot_dim / 2, 2] fp32
    (None: no rotation); positions int32 [T] (None: the tokens' places in their sequences).  Q_out may be Q."""
    T, D = batch.tokens, cache.D
    if rope is not None and (rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[2] != 2):
        raise ValueError("rope must be float32 [max_pos, rot_dim / 2, 2]")
    if positions is not None and (positions.dtype != torch.int32 or positions.shape != (T,)):
        raise ValueError(f"positions must be int32 [{T}]")
    if Q is None and Q_out is not None:
        raise ValueError("Q_out without Q")
    device = cache._index
    _same_device("kv4_append", device, batch.cu_q, K, V, Q, rope, positions, Q_out)
    k, v = _rows(K, "K", T, cache.Hkv, D), _rows(V, "V", T, cache.Hkv, D)
    q = qo = None
    Hq = 0
    if Q is not None:
        Hq = _heads(Q, "Q")
        q = _rows(Q, "Q", T, Hq, D)
        if Q_out is None:
            Q_out, qo = _new_rows(T, Hq, D, cache.device, stream)
        else:
            qo = _rows(Q_out, "Q_out", T, Hq, D)
    _check(wq_kv4_append(cache._struct, batch._struct, q, qo, Hq, k, v, _ptr(rope),
                         0 if rope is None else rope.shape[0], 0 if rope is None else 2 * rope.shape[1],
                         1 if interleaved else 0, _ptr(positions), _launch_stream(stream, device)), "wq_kv4_append")
    return Q_out


def kv4_read(cache: Kv4Cache, batch: Kv4Batch, K: torch.Tensor | None = None, V: torch.Tensor | None = None,
             stream=None):
    """The batch's tokens as they are cached: bf16 K and V [T, Hkv, D], rounded once from scale times code.  Given
    tensors (any strides with a contiguous last dimension) are filled and returned."""
    T, Hkv, D, device = batch.tokens, cache.Hkv, cache.D, cache._index
    _same_device("kv4_read", device, batch.cu_q, K, V)
    K, k = _new_rows(T, Hkv, D, cache.device, stream) if K is None else (K, _rows(K, "K", T, Hkv, D))
    V, v = _new_rows(T, Hkv, D, cache.device, stream) if V is None else (V, _rows(V, "V", T, Hkv, D))
    _check(wq_kv4_read(cache._struct, batch._struct, k, v, _launch_stream(stream, device)), "wq_kv4_read")
    return K, V


def kv4_workspace(Hq: int, cache: Kv4Cache) -> torch.Tensor:
    """The attention's workspace for ``Hq`` query heads over this cache: one per stream, for any batch."""
    n = wq_kv4_workspace_bytes(Hq, cache.Hkv, cache.D)
    if n == 0:
        raise WQError(WQ_ERR_SHAPE, "kv4_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=cache.pool.device)


def kv4_attention(Q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, scale: float | None = None, window: int = 0,
                  O: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the batch's new tokens over their whole cached sequences (themselves included).  Q [T, Hq,
    D] bf16; query head h reads key/value head h // (Hq // Hkv); scale: 1 / sqrt(D) by default; window > 0: only the
    newest ``window`` keys up to the query.  Returns O [T, Hq, D].  ``workspace``: a ``kv4_workspace`` that the caller
    keeps for this stream (a fresh one otherwise)."""
    T, D, device = batch.tokens, cache.D, cache._index
    Hq = _heads(Q, "Q")
    q = _rows(Q, "Q", T, Hq, D)
    _same_device("kv4_attention", device, batch.cu_q, Q, O, workspace)
    O, o = _new_rows(T, Hq, D, cache.device, stream) if O is None else (O, _rows(O, "O", T, Hq, D))
    if workspace is None:
        with _on(stream):
            workspace = kv4_workspace(Hq, cache)
    _check(wq_kv4_attention(cache._struct, batch._struct, q, o, Hq,
                            D ** -0.5 if scale is None else scale, window, _ptr(workspace), workspace.nbytes,
                            _launch_stream(stream, device)), "wq_kv4_attention")
    return O


# ------------------------------------------- log probabilities of tokens ---
def logprobs_workspace(T: int, V: int, k: int = 0, device="cuda") -> torch.Tensor:
    """``token_logprobs``' workspace for up to T rows of up to V logits and up to k alternatives: one per stream, for
    calls of any such sizes."""
    n = wq_logprobs_workspace_bytes(T, V, k)
    if n == 0:
        raise WQError(WQ_ERR_SHAPE, "logprobs_workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, k: int = 0,
                   inv_temperature: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Per row of logits [T, V] (fp32 or bf16, rows any distance apart) and its token (int64 [T]): returns (log
    probability [T], entropy [T], rank [T] int32, top ids [T, k] int32, top log probabilities [T, k]) of the softmax
    of inv_temperature * logits.  The rank is the number of larger logits, so tokens that tie share it; the top ids put
    the lowest id of equal logits first."""
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be [T, V], float32 or bfloat16")
    T, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits: the last dimension must be contiguous")
    if tokens.dtype != torch.int64 or tokens.shape != (T,):
        raise ValueError(f"tokens must be int64 [{T}]")
    if inv_temperature is not None and (inv_temperature.dtype != torch.float32 or
                                        inv_temperature.shape != (T,)):
        raise ValueError(f"inv_temperature must be float32 [{T}]")
    at, device = logits.device, logits.get_device()
    logprob = _empty((T,), torch.float32, at, stream)  # (views of one tensor cost more than tensors of their own)
    entropy = _empty((T,), torch.float32, at, stream)
    rank = _empty((T,), torch.int32, at, stream)
    ids = _empty((T, max(k, 0)), torch.int32, at, stream)
    top = _empty((T, max(k, 0)), torch.float32, at, stream)
    if workspace is None:
        with _on(stream):
            workspace = logprobs_workspace(T, V, k, at)
    _same_device("token_logprobs", device, tokens, inv_temperature, workspace)
    _check(wq_token_logprobs(logits.data_ptr(), WQ_F32 if logits.dtype is torch.float32 else WQ_BF16, T, V,
                             logits.stride(0) if T > 1 else 0, _ptr(tokens), _ptr(inv_temperature), k,
                             logprob.data_ptr(), entropy.data_ptr(), rank.data_ptr(), ids.data_ptr(), top.data_ptr(),
                             _ptr(workspace), workspace.nbytes, _launch_stream(stream, device)), "wq_token_logprobs")
    return logprob, entropy, rank, ids, top
