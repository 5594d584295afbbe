"""Python binding of the C ABI in include/hqq_b200.h (argument marshalling only).

Every step of quantize and dequantize runs in the CUDA kernels of libhqq_b200.so; this module
allocates output buffers with torch when the caller does not pass them, hands raw device
pointers and the current CUDA stream to the library, and raises on a non-zero return code.
There is no CPU fallback: loading fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhqq_b200.so")

HQQ_OK = 0
HQQ_MAX_GROUP_SIZE = 256
HQQ_MAX_ITERS = 64


class HqqOpt(ctypes.Structure):
    _fields_ = [("iters", ctypes.c_int32), ("lp_norm", ctypes.c_double),
                ("beta", ctypes.c_double), ("kappa", ctypes.c_double),
                ("eps_tiny", ctypes.c_float), ("scale_max", ctypes.c_float)]


class HqqKvCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_meta", ctypes.c_void_p), ("v_meta", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("nbits", ctypes.c_int32), ("group_size", ctypes.c_int32)]


class HqqError(RuntimeError):
    pass


_lib = None

# (name, restype, argtypes) of every symbol the header declares
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "hqq_default_opt": (None, [ctypes.POINTER(HqqOpt)]),
    "hqq_packed_bytes": (_I64, [_I64, _I32]),
    "hqq_quantize_workspace_bytes": (_SZ, [_I64, _I64, _I32, _I64, _I32, _I32]),
    "hqq_quantize": (_I32, [_P, _I64, _I64, _I32, _I64, _I32, ctypes.POINTER(HqqOpt), _P, _P, _P,
                            _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "hqq_dequantize": (_I32, [_P, _P, _P, _I64, _I64, _I32, _I64, _I32, _P, _P]),
    "hqq_quantize_noalloc": (_I32, [_P, _I64, _I64, _I32, _I64, _I32, ctypes.POINTER(HqqOpt), _P,
                                    _P, _P, _P, _P, _P, _P, _P, _P]),
    "hqq_gemv": (_I32, [_P, _P, _P, _I64, _I64, _I32, _I64, _I32, _P, _P, _P]),
    "hqq_gemm": (_I32, [_P, _P, _P, _I64, _I64, _I32, _I64, _I32, _P, _I64, _P, _P]),
    "hqq_shrink_lp": (_I32, [_P, _I64, ctypes.c_double, ctypes.c_double, _P, _P]),
    "hqq_kv_append": (_I32, [_P, _P, _P, _I32, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P]),
    "hqq_kv_read": (_I32, [_P, _P, _I64, _I32, _P, _P, _P]),
    "hqq_kv_attention_workspace_bytes": (_SZ, [_P, _I64, _I64, _I64, _I64, _I64, _I64]),
    "hqq_kv_attention": (_I32, [_P, _P, _I32, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64, _I64, _P,
                                _I64, _I64, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "hqq_kv_prefix_attention": (_I32, [_P, _P, _I32, _I64, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P,
                                       _I64, _I64, _P, _I64, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "hqq_strerror": (ctypes.c_char_p, [_I32]),
}


def lib():
    """The loaded CUDA library; raises if libhqq_b200.so has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise HqqError(f"{LIB_PATH} is missing: build it with "
                           "`python -m free_weight_quantization_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != HQQ_OK:
        raise HqqError(f"{what}: {lib().hqq_strerror(rc).decode()} (code {rc})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def default_opt() -> HqqOpt:
    o = HqqOpt()
    lib().hqq_default_opt(ctypes.byref(o))
    return o


def hqq_packed_bytes(n: int, nbits: int) -> int:
    return int(lib().hqq_packed_bytes(n, nbits))


def hqq_quantize_workspace_bytes(rows: int, cols: int, nbits: int, group_size: int, axis: int,
                                 iters: int) -> int:
    return int(lib().hqq_quantize_workspace_bytes(rows, cols, nbits, group_size, axis, iters))


@dataclass
class Quantized:
    """Packed codes + fp16 metadata (the page's W_q, scale = Delta = 1/s, zero) and the shape."""
    packed: torch.Tensor
    scale: torch.Tensor
    zero: torch.Tensor
    rows: int
    cols: int
    nbits: int
    group_size: int
    axis: int
    iters_run: torch.Tensor | None = None
    s: torch.Tensor | None = None
    z: torch.Tensor | None = None
    err_trace: torch.Tensor | None = None
    rounds: torch.Tensor | None = None


def hqq_quantize(W: torch.Tensor, nbits: int = 4, group_size: int = 64, axis: int = 1,
                 iters: int = 20, lp_norm: float = 0.7, beta: float = 10.0, kappa: float = 1.01,
                 eps_tiny: float = 1e-4, scale_max: float = 2e4, *, out: Quantized | None = None,
                 workspace: torch.Tensor | None = None, debug: bool = False,
                 stream: torch.cuda.Stream | None = None) -> Quantized:
    """HQQ quantize + pack of an fp16 CUDA matrix [rows, cols] (see hqq_quantize in the header).
    With debug=True also returns iters_run, binary32 s and z, the exact error trace and the
    rounds each group needed."""
    if W.dtype != torch.float16 or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
        raise HqqError("W must be a contiguous 2-D float16 CUDA tensor")
    rows, cols = W.shape
    N = rows * cols
    if group_size <= 0 or N % group_size:
        raise HqqError("rows*cols must be a positive multiple of group_size")
    G = N // group_size
    dev = W.device
    if out is None:
        pb = hqq_packed_bytes(N, nbits)
        if pb < 0:
            raise HqqError("nbits must be 2, 3 or 4")
        out = Quantized(torch.empty(max(pb, 1), dtype=torch.uint8, device=dev),
                        torch.empty(G, dtype=torch.float16, device=dev),
                        torch.empty(G, dtype=torch.float16, device=dev),
                        rows, cols, nbits, group_size, axis)
        if debug:
            out.iters_run = torch.zeros(1, dtype=torch.int32, device=dev)
            out.s = torch.empty(G, dtype=torch.float32, device=dev)
            out.z = torch.empty(G, dtype=torch.float32, device=dev)
            out.err_trace = torch.zeros(max(2 * iters, 2), dtype=torch.int64, device=dev)
            out.rounds = torch.empty(G, dtype=torch.uint8, device=dev)
    wsb = hqq_quantize_workspace_bytes(rows, cols, nbits, group_size, axis, iters)
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    opt = HqqOpt(iters, lp_norm, beta, kappa, eps_tiny, scale_max)
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):  # launches go to the current device: W's
        rc = lib().hqq_quantize(_ptr(W), rows, cols, nbits, group_size, axis, ctypes.byref(opt),
                                _ptr(out.packed), _ptr(out.scale), _ptr(out.zero), _ptr(out.iters_run),
                                _ptr(out.s), _ptr(out.z), _ptr(out.err_trace), _ptr(out.rounds),
                                _ptr(workspace),
                                workspace.numel() * workspace.element_size(),
                                ctypes.c_void_p(st.cuda_stream))
    _check(rc, "hqq_quantize")
    return out


HQQ_NOALLOC_SCRATCH_BYTES = 4 << 20


def hqq_quantize_noalloc(W: torch.Tensor, nbits: int = 4, group_size: int = 64, axis: int = 1,
                         iters: int = 20, lp_norm: float = 0.7, beta: float = 10.0,
                         kappa: float = 1.01, eps_tiny: float = 1e-4, scale_max: float = 2e4, *,
                         out: Quantized, stream: torch.cuda.Stream | None = None) -> Quantized:
    """hqq_quantize for callers that cannot allocate device memory: the caller passes every
    output buffer in `out` and the library uses its own fixed 4 MiB scratch buffer instead of a
    workspace (see hqq_quantize_noalloc in the header).  Nothing is allocated here either."""
    if W.dtype != torch.float16 or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
        raise HqqError("W must be a contiguous 2-D float16 CUDA tensor")
    rows, cols = W.shape
    bufs = [out.packed, out.scale, out.zero, out.iters_run, out.s, out.z, out.err_trace, out.rounds]
    if any(t is not None and t.device != W.device for t in bufs):
        raise HqqError("hqq_quantize_noalloc: every output must live on W's device")
    opt = HqqOpt(iters, lp_norm, beta, kappa, eps_tiny, scale_max)
    st = stream if stream is not None else torch.cuda.current_stream(W.device)
    if st.device != W.device:
        raise HqqError("hqq_quantize_noalloc: the stream must belong to W's device")
    # the library finds its scratch buffer on the calling thread's current device
    with torch.cuda.device(W.device):
        rc = lib().hqq_quantize_noalloc(_ptr(W), rows, cols, nbits, group_size, axis,
                                        ctypes.byref(opt), _ptr(out.packed), _ptr(out.scale),
                                        _ptr(out.zero), _ptr(out.iters_run), _ptr(out.s), _ptr(out.z),
                                        _ptr(out.err_trace), _ptr(out.rounds),
                                        ctypes.c_void_p(st.cuda_stream))
    if rc == 3:
        raise HqqError("hqq_quantize_noalloc: this problem needs "
                       f"{hqq_quantize_workspace_bytes(rows, cols, nbits, group_size, axis, iters)}"
                       f" bytes of scratch, more than the built-in {HQQ_NOALLOC_SCRATCH_BYTES}")
    _check(rc, "hqq_quantize_noalloc")
    return out


def hqq_dequantize(q: Quantized, out: torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Unpack + (q - zero) * scale -> fp16 [rows, cols] (see hqq_dequantize in the header)."""
    if out is None:
        out = torch.empty(q.rows, q.cols, dtype=torch.float16, device=q.packed.device)
    st = stream if stream is not None else torch.cuda.current_stream(q.packed.device)
    with torch.cuda.device(q.packed.device):
        rc = lib().hqq_dequantize(_ptr(q.packed), _ptr(q.scale), _ptr(q.zero), q.rows, q.cols, q.nbits,
                                  q.group_size, q.axis, _ptr(out), ctypes.c_void_p(st.cuda_stream))
    _check(rc, "hqq_dequantize")
    return out


def hqq_gemv(q: Quantized, x: torch.Tensor, out: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y = W_hat @ x with dequantization fused in (see hqq_gemv in the header): x is a
    contiguous fp16 CUDA vector of q.cols entries, y a binary32 vector of q.rows."""
    if x.dtype != torch.float16 or not x.is_cuda or x.dim() != 1 or x.numel() != q.cols or not x.is_contiguous():
        raise HqqError("x must be a contiguous fp16 CUDA vector with cols entries")
    if out is None:
        out = torch.empty(q.rows, dtype=torch.float32, device=q.packed.device)
    st = stream if stream is not None else torch.cuda.current_stream(q.packed.device)
    with torch.cuda.device(q.packed.device):
        rc = lib().hqq_gemv(_ptr(q.packed), _ptr(q.scale), _ptr(q.zero), q.rows, q.cols, q.nbits,
                            q.group_size, q.axis, _ptr(x), _ptr(out), ctypes.c_void_p(st.cuda_stream))
    _check(rc, "hqq_gemv")
    return out


def hqq_gemm(q: Quantized, X: torch.Tensor, out: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Y = X @ W_hat.T for a batch of inputs with dequantization fused in (see hqq_gemm in the
    header): X is a contiguous fp16 CUDA matrix [batch, cols], Y binary32 [batch, rows]."""
    if X.dtype != torch.float16 or not X.is_cuda or X.dim() != 2 or X.shape[1] != q.cols or not X.is_contiguous():
        raise HqqError("X must be a contiguous fp16 CUDA matrix [batch, cols]")
    batch = X.shape[0]
    if out is None:
        out = torch.empty(batch, q.rows, dtype=torch.float32, device=q.packed.device)
    st = stream if stream is not None else torch.cuda.current_stream(q.packed.device)
    with torch.cuda.device(q.packed.device):
        rc = lib().hqq_gemm(_ptr(q.packed), _ptr(q.scale), _ptr(q.zero), q.rows, q.cols, q.nbits,
                            q.group_size, q.axis, _ptr(X), batch, _ptr(out), ctypes.c_void_p(st.cuda_stream))
    _check(rc, "hqq_gemm")
    return out


def hqq_shrink_lp(r: torch.Tensor, beta: float, p: float = 0.7, out: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The proximal step's lp shrink of binary32 residuals, as the quantizer evaluates it (see
    hqq_shrink_lp in the header)."""
    if r.dtype != torch.float32 or not r.is_cuda or not r.is_contiguous():
        raise HqqError("r must be a contiguous float32 CUDA tensor")
    if out is None:
        out = torch.empty_like(r)
    st = stream if stream is not None else torch.cuda.current_stream(r.device)
    with torch.cuda.device(r.device):
        rc = lib().hqq_shrink_lp(_ptr(r), r.numel(), float(beta), float(p), _ptr(out),
                                 ctypes.c_void_p(st.cuda_stream))
    _check(rc, "hqq_shrink_lp")
    return out


def err_trace_ints(t: torch.Tensor, n: int) -> list[int]:
    """Exact per-round error sums (units of 2^-32) from the (low, high) uint64 pairs."""
    v = t.cpu().view(torch.int64).tolist()
    return [(v[2 * i] & (2 ** 64 - 1)) + ((v[2 * i + 1] & (2 ** 64 - 1)) << 64) for i in range(n)]


# ---- the key/value cache (hqq_kv_* in the header) ------------------------------------------
# These calls are for serving and have no backward pass: what they return requires no grad, whatever
# their inputs require.

_KV_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


class KVCache:
    """A paged, group-quantized key/value cache: the tensors that the header's hqq_kv_cache
    describes, and that description.

    k_codes, v_codes: uint8 [pages, kv_heads, page_size, head_dim * nbits / 8]; k_meta, v_meta:
    float16 [pages, kv_heads, page_size, head_dim / group_size, 2], (scale, zero).  Contiguous, on
    one CUDA device; hqq_kv_cache() allocates them."""

    __slots__ = ("k_codes", "v_codes", "k_meta", "v_meta", "num_pages", "kv_heads", "page_size",
                 "head_dim", "nbits", "group_size", "device", "_c", "_ref")

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_meta: torch.Tensor,
                 v_meta: torch.Tensor, nbits: int, group_size: int):
        if nbits not in (2, 4, 8):
            raise HqqError("KVCache: nbits must be 2, 4 or 8")
        if group_size not in (32, 64, 128):
            raise HqqError("KVCache: group_size must be 32, 64 or 128")
        if k_codes.dim() != 4:
            raise HqqError("KVCache: codes must be [pages, kv_heads, page_size, head_dim * nbits / 8]")
        pages, heads, page_size, row = k_codes.shape
        head_dim = row * 8 // nbits
        if head_dim not in (64, 128, 256) or row * 8 % nbits or head_dim % group_size:
            raise HqqError("KVCache: head_dim must be 64, 128 or 256 and a multiple of group_size")
        if heads < 1 or not 16 <= page_size <= 1024 or page_size & (page_size - 1):
            raise HqqError("KVCache: page_size must be a power of two from 16 to 1024, kv_heads at least 1")
        meta = (pages, heads, page_size, head_dim // group_size, 2)
        for name, t, shape, dtype in (("k_codes", k_codes, k_codes.shape, torch.uint8),
                                      ("v_codes", v_codes, k_codes.shape, torch.uint8),
                                      ("k_meta", k_meta, meta, torch.float16),
                                      ("v_meta", v_meta, meta, torch.float16)):
            if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
                raise HqqError(f"KVCache: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
        if any(not t.is_cuda or t.device != k_codes.device for t in (k_codes, v_codes, k_meta, v_meta)):
            raise HqqError("KVCache: the tensors must live on one CUDA device")
        self.k_codes, self.v_codes, self.k_meta, self.v_meta = k_codes, v_codes, k_meta, v_meta
        self.num_pages, self.kv_heads, self.page_size = pages, heads, page_size
        self.head_dim, self.nbits, self.group_size = head_dim, nbits, group_size
        self.device = k_codes.device
        self._c = HqqKvCache(k_codes.data_ptr(), v_codes.data_ptr(), k_meta.data_ptr(), v_meta.data_ptr(),
                             pages, page_size, heads, head_dim, nbits, group_size)
        self._ref = ctypes.addressof(self._c)


def hqq_kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, nbits: int = 4,
                 group_size: int = 64, device="cuda") -> KVCache:
    """An empty KVCache (every row reads as zeros)."""
    if num_pages < 0 or nbits not in (2, 4, 8) or group_size not in (32, 64, 128) or head_dim % group_size:
        raise HqqError("hqq_kv_cache: nbits must be 2, 4 or 8, group_size 32, 64 or 128 and divide head_dim")
    if kv_heads < 1 or head_dim not in (64, 128, 256) or not 16 <= page_size <= 1024 or page_size & (page_size - 1):
        raise HqqError("hqq_kv_cache: head_dim must be 64, 128 or 256, page_size a power of two from 16 to 1024, "
                       "kv_heads at least 1")
    codes = (num_pages, kv_heads, page_size, head_dim * nbits // 8)
    meta = (num_pages, kv_heads, page_size, head_dim // group_size, 2)
    return KVCache(torch.zeros(codes, dtype=torch.uint8, device=device),
                   torch.zeros(codes, dtype=torch.uint8, device=device),
                   torch.zeros(meta, dtype=torch.float16, device=device),
                   torch.zeros(meta, dtype=torch.float16, device=device), nbits, group_size)


def _kv_stream(device: torch.device, stream: torch.cuda.Stream | None) -> int:
    """The handle of the launching stream.  (The raw query of the current one takes 0.1 us where
    torch.cuda.current_stream takes 2, which is half of what a small call costs on the GPU.)"""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise HqqError("the stream must belong to the cache's device")
    return stream.cuda_stream


def _kv_rows(what: str, cache: KVCache, t: torch.Tensor, tokens: int):
    if t.dtype not in _KV_DTYPES or t.device != cache.device:
        raise HqqError(f"{what} must be a float16 or bfloat16 tensor on the cache's device")
    if t.shape != (tokens, cache.kv_heads, cache.head_dim):
        raise HqqError(f"{what} must be [tokens, kv_heads, head_dim]")
    if t.stride(2) != 1 and t.numel():
        raise HqqError(f"{what}: the values of a head must be contiguous")


def _kv_out(what: str, t: torch.Tensor, shape, dtype, device):
    if t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise HqqError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the cache's device")


def _kv_slots(cache: KVCache, slots: torch.Tensor):
    if slots.dtype != torch.int64 or slots.device != cache.device or slots.dim() != 1 or not slots.is_contiguous():
        raise HqqError("slots must be a contiguous 1-D int64 tensor on the cache's device")
    return slots.shape[0]


def _on_device(call):
    """Runs a call under the cache's device, and under the launching stream when one is given: what
    the call allocates then belongs to that stream, and its memory is reused in that stream's order."""
    @functools.wraps(call)
    def run(cache, *args, stream=None, **kwargs):
        if stream is None and cache.device.index == torch.cuda.current_device():
            return call(cache, *args, **kwargs)
        with torch.cuda.device(cache.device):
            if stream is None:
                return call(cache, *args, **kwargs)
            _kv_stream(cache.device, stream)
            with torch.cuda.stream(stream):
                return call(cache, *args, stream=stream, **kwargs)
    return run


@_on_device
def hqq_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *,
                  return_values: bool = False, out: tuple[torch.Tensor, torch.Tensor] | None = None,
                  stream: torch.cuda.Stream | None = None):
    """Quantizes keys and values [tokens, kv_heads, head_dim] (fp16 or bf16; tokens and heads may be
    strided, as slices of a fused projection are) into `slots` (int64 page * page_size + offset;
    negative: skipped) of the cache.  With return_values (or out=(k, v)) also returns the values that
    the cache now stands for.  Rounding has no gradient: k and v are taken without theirs.  See
    hqq_kv_append in the header."""
    tokens = _kv_slots(cache, slots)
    _kv_rows("k", cache, k, tokens)
    _kv_rows("v", cache, v, tokens)
    if k.dtype != v.dtype:
        raise HqqError("k and v must have the same type")
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if out is not None:
        for name, t in zip(("out[0]", "out[1]"), out, strict=True):
            _kv_out(name, t, shape, k.dtype, cache.device)
    elif return_values:
        out = (k.new_empty(shape), k.new_empty(shape))
    ks, vs = k.stride(), v.stride()
    rc = lib().hqq_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), _KV_DTYPES[k.dtype], tokens, ks[0], ks[1], vs[0],
                             vs[1], slots.data_ptr(), None if out is None else out[0].data_ptr(),
                             None if out is None else out[1].data_ptr(), _kv_stream(cache.device, stream))
    _check(rc, "hqq_kv_append")
    return out


@_on_device
def hqq_kv_read(cache: KVCache, slots: torch.Tensor, dtype: torch.dtype = torch.float16, *,
                out: tuple[torch.Tensor, torch.Tensor] | None = None,
                stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The keys and values [tokens, kv_heads, head_dim] that the cache's `slots` stand for (zeros for
    a negative slot).  See hqq_kv_read in the header."""
    tokens = _kv_slots(cache, slots)
    if dtype not in _KV_DTYPES:
        raise HqqError("dtype must be float16 or bfloat16")
    shape = (tokens, cache.kv_heads, cache.head_dim)
    if out is not None:
        for name, t in zip(("out[0]", "out[1]"), out, strict=True):
            _kv_out(name, t, shape, dtype, cache.device)
    else:
        out = (slots.new_empty(shape, dtype=dtype), slots.new_empty(shape, dtype=dtype))
    rc = lib().hqq_kv_read(cache._ref, slots.data_ptr(), tokens, _KV_DTYPES[dtype], out[0].data_ptr(),
                           out[1].data_ptr(), _kv_stream(cache.device, stream))
    _check(rc, "hqq_kv_read")
    return out


def _kv_attend(cache: KVCache, q, pages, lens, prefix, window, scale, max_len, out, return_lse,
               workspace, stream):
    dev = cache.device
    if q.dtype not in _KV_DTYPES or q.device != dev or q.dim() != 4 or q.shape[3] != cache.head_dim:
        raise HqqError("q must be a float16 or bfloat16 tensor [batch, nq, heads, head_dim] on the cache's device")
    batch, nq, heads, dim = q.shape
    if heads < 1 or heads % cache.kv_heads:
        raise HqqError("heads must be a positive multiple of the cache's kv_heads")
    if q.stride(3) != 1 and q.numel():
        raise HqqError("q: the values of a head must be contiguous")
    if pages.dtype != torch.int32 or pages.device != dev or pages.dim() != 2 or pages.shape[0] != batch \
            or (pages.shape[1] > 1 and pages.stride(1) != 1):
        raise HqqError("pages must be an int32 tensor [batch, max_pages] on the cache's device, rows contiguous")
    if lens.dtype != torch.int32 or lens.device != dev or lens.shape != (batch,) or not lens.is_contiguous():
        raise HqqError("lens must be a contiguous int32 tensor [batch] on the cache's device")
    room = pages.shape[1] * cache.page_size
    if max_len is None:
        max_len = room
    elif not 0 <= max_len <= room:
        raise HqqError("max_len must lie between 0 and max_pages * page_size")
    if window < 0:
        raise HqqError("window must not be negative (0: none)")
    if window >= max_len:
        window = 0  # hides nothing, and need not fit the call's 64 bits
    if scale is None:
        scale = dim ** -0.5
    prefix_len = 0
    if prefix is not None:
        prefix_pages, prefix_len = prefix
        if prefix_pages.dtype != torch.int32 or prefix_pages.device != dev or prefix_pages.dim() != 1 \
                or not prefix_pages.is_contiguous():
            raise HqqError("prefix_pages must be a contiguous 1-D int32 tensor on the cache's device")
        if not 0 <= prefix_len <= prefix_pages.shape[0] * cache.page_size:
            raise HqqError("prefix_len must lie between 0 and the tokens of prefix_pages")
    L = lib()
    if workspace is None:
        need = L.hqq_kv_attention_workspace_bytes(cache._ref, batch, nq, heads, max_len, window, prefix_len)
        if need:
            workspace = q.new_empty((need,), dtype=torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise HqqError("workspace must be a contiguous tensor on the cache's device")
    if out is None:
        out = q.new_empty(q.shape)
    else:
        _kv_out("out", out, q.shape, q.dtype, dev)
    lse = q.new_empty((batch, nq, heads), dtype=torch.float32) if return_lse else None
    qs, ps = q.stride(), pages.stride(0)
    ws = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    handle = _kv_stream(dev, stream)
    if prefix is None:
        rc = L.hqq_kv_attention(cache._ref, q.data_ptr(), _KV_DTYPES[q.dtype], batch, nq, heads, qs[0], qs[1], qs[2],
                                pages.data_ptr(), ps, pages.shape[1], lens.data_ptr(), max_len, window, scale,
                                out.data_ptr(), None if lse is None else lse.data_ptr(), ws[0], ws[1], handle)
        _check(rc, "hqq_kv_attention")
    else:
        rc = L.hqq_kv_prefix_attention(cache._ref, q.data_ptr(), _KV_DTYPES[q.dtype], batch, nq, heads, qs[0], qs[1],
                                       qs[2], prefix_pages.data_ptr(), prefix_len, pages.data_ptr(), ps, pages.shape[1],
                                       lens.data_ptr(), max_len, scale, out.data_ptr(),
                                       None if lse is None else lse.data_ptr(), ws[0], ws[1], handle)
        _check(rc, "hqq_kv_prefix_attention")
    return (out, lse) if return_lse else out


@_on_device
def hqq_kv_attention(cache: KVCache, q: torch.Tensor, pages: torch.Tensor, lens: torch.Tensor, *,
                     window: int = 0, scale: float | None = None, max_len: int | None = None,
                     out: torch.Tensor | None = None, return_lse: bool = False,
                     workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Attention of the last nq tokens of each sequence, q [batch, nq, heads, head_dim] (fp16 or bf16,
    strided in all but the last dimension), over its cached context: pages int32 [batch, max_pages],
    lens int32 [batch] with the queries' own tokens counted.  Returns out (and, with return_lse, the
    binary32 log-sum-exp [batch, nq, heads]).  scale defaults to head_dim ** -0.5; max_len bounds lens
    (default: what `pages` has room for) and sizes the launch.  For serving: out and lse require no
    grad, even if q does.  See hqq_kv_attention in the header."""
    return _kv_attend(cache, q, pages, lens, None, window, scale, max_len, out, return_lse,
                      workspace, stream)


@_on_device
def hqq_kv_prefix_attention(cache: KVCache, q: torch.Tensor, prefix_pages: torch.Tensor, prefix_len: int,
                            pages: torch.Tensor, lens: torch.Tensor, *, scale: float | None = None,
                            max_len: int | None = None, out: torch.Tensor | None = None,
                            return_lse: bool = False, workspace: torch.Tensor | None = None,
                            stream: torch.cuda.Stream | None = None):
    """hqq_kv_attention for a batch whose sequences share their first prefix_len tokens, held in
    prefix_pages (int32 [n]) and read once for all; pages and lens are each sequence's own tokens
    behind it.  As there, no gradients.  See hqq_kv_prefix_attention in the header."""
    return _kv_attend(cache, q, pages, lens, (prefix_pages, prefix_len), 0, scale, max_len,
                      out, return_lse, workspace, stream)
