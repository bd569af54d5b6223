"""BinaryAttention forward pass for NVIDIA B200 (sm_100a).

Every step of the path runs in the CUDA kernels of the C-ABI library
``libbinattn.so`` (built from ``csrc/`` by ``build.py``). This module only marshals
arguments: it takes torch CUDA tensors, allocates outputs and workspace with torch,
and passes raw device pointers plus the current stream. There is no CPU fallback: if
the library is missing, every call raises.

Functions mirror the C entry points of ``include/binattn.h``:
``pack_signs``, ``quant_v``, ``attention_fwd``, ``attention_fwd_packed``, and for sequences
that grow ``KVCache`` with ``cache_write``, ``cache_read`` and ``attention_paged``.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbinattn.so")

BA_F16, BA_BF16, BA_F32 = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # BA_NOALLOC_SCRATCH_BYTES of include/binattn.h
BIAS_NONE, BIAS_DENSE, BIAS_RELPOS2D = 0, 1, 2
IMPL_AUTO, IMPL_SIMT, IMPL_TCGEN05 = 0, 1, 2

STATUS = {0: "BA_OK", 1: "BA_ERR_INVALID_ARG", 2: "BA_ERR_UNSUPPORTED", 3: "BA_ERR_ALIGNMENT",
          4: "BA_ERR_WORKSPACE", 5: "BA_ERR_CUDA", 6: "BA_ERR_TIMEOUT"}


class BinAttnError(RuntimeError):
    def __init__(self, status: int, where: str, cuda_error: int = 0):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        if status == 5:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


class CBias(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64),
                ("grid_h", ctypes.c_int), ("grid_w", ctypes.c_int), ("table_h", ctypes.c_int),
                ("table_w", ctypes.c_int), ("n_prefix", ctypes.c_int)]


class CKvCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("d", ctypes.c_int)]


class CPagedSeqs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int64), ("n_heads", ctypes.c_int),
                ("max_q_len", ctypes.c_int), ("max_kv_len", ctypes.c_int64), ("cu_seqlens_q", ctypes.c_void_p),
                ("kv_lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int), ("causal", ctypes.c_int), ("window", ctypes.c_int),
                ("sinks", ctypes.c_int)]


_lib = None

_P, _I, _F, _SZ, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
SIGNATURES = {
    "ba_sign_words": (_I, [_I]),
    "ba_v_row_bytes": (_I, [_I]),
    "ba_kv_block": (_I, []),
    "ba_p_code_threshold": (ctypes.c_double, [_I]),
    "ba_prep_fused": (_I, [_I, _I, _I, _I]),
    "ba_pack_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "ba_quant_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "ba_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "ba_pack_signs": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "ba_quant_v": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "ba_attention_fwd_packed": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.POINTER(CBias), _F, _P,
                                     _I, _P, _P]),
    "ba_attention_fwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(CBias), _F, _P, _I, _P, _SZ,
                              _P, _P]),
    "ba_attention_fwd_debug": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(CBias), _F, _P, _I, _P, _SZ,
                                    _P, _P, _I, _P]),
    "ba_attention_fwd_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, ctypes.POINTER(CBias), _F, _P, _I, _P,
                                      _P]),
    "ba_kv_block_bytes": (_SZ, [_I, _I]),
    "ba_cache_write": (_I, [_P, _I64, _I64, _P, _I64, _I64, _I, _I64, _P, ctypes.POINTER(CKvCache), _P]),
    "ba_cache_read": (_I, [ctypes.POINTER(CKvCache), _P, _I64, _P, _P, _I, _P]),
    "ba_paged_workspace_bytes": (_SZ, [ctypes.POINTER(CKvCache), ctypes.POINTER(CPagedSeqs)]),
    "ba_attention_paged": (_I, [_P, _I64, _I64, _I, ctypes.POINTER(CKvCache), ctypes.POINTER(CPagedSeqs), _F, _P,
                                _I, _P, _P, _SZ, _P]),
    "ba_set_attention_impl": (_I, [_I]),
    "ba_get_attention_impl": (_I, []),
    "ba_last_attention_impl": (_I, []),
    "ba_check_device_status": (_I, [_P]),
    "ba_stage_timing": (_I, [_I]),
    "ba_stage_times": (_I, [ctypes.POINTER(ctypes.c_float), _I, ctypes.POINTER(ctypes.c_int)]),
    "ba_status_string": (ctypes.c_char_p, [_I]),
    "ba_last_cuda_error": (_I, []),
}


def lib(path: Optional[str] = None) -> ctypes.CDLL:
    """The loaded C-ABI library. Raises if it has not been built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libbinattn.so not found at {p}: build it with "
                           "`python -m bit_qk_attention_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = L
    return L


def _check(status: int, where: str):
    if status != 0:
        raise BinAttnError(status, where, lib().ba_last_cuda_error())


# ----------------------------------------------------------------------------- helpers
def _torch():
    import torch
    return torch


def _dt(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return BA_F16
    if t.dtype == torch.bfloat16:
        return BA_BF16
    if t.dtype == torch.float32:
        return BA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _qkv_check(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B,H,N,d]")


@dataclass
class Bias:
    """The additive logit bias (see include/binattn.h, ba_bias)."""
    kind: int = BIAS_NONE
    data: Optional[object] = None  # torch fp32 CUDA tensor
    batch_stride: int = 0
    grid_h: int = 0
    grid_w: int = 0
    table_h: int = 0
    table_w: int = 0
    n_prefix: int = 0

    def c(self) -> CBias:
        b = CBias()
        b.kind = self.kind
        b.data = 0 if self.data is None else self.data.data_ptr()
        b.batch_stride = self.batch_stride
        b.grid_h, b.grid_w = self.grid_h, self.grid_w
        b.table_h, b.table_w, b.n_prefix = self.table_h, self.table_w, self.n_prefix
        return b


def sign_words(d: int) -> int:
    return lib().ba_sign_words(d)


def v_row_bytes(d: int) -> int:
    return lib().ba_v_row_bytes(d)


def kv_block() -> int:
    return lib().ba_kv_block()


def p_code_threshold(k: int) -> float:
    """The least d = s - m (double) whose 8-bit P code exceeds k (0 <= k <= 254), else NaN."""
    return lib().ba_p_code_threshold(int(k))


def prep_fused(B: int, H: int, N: int, d: int) -> bool:
    """Whether attention_fwd prepares q, k, v in one launch for this shape (see ba_prep_fused)."""
    return bool(lib().ba_prep_fused(B, H, N, d))


def workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib().ba_workspace_bytes(B, H, N, d)


def set_attention_impl(impl: int):
    _check(lib().ba_set_attention_impl(impl), "ba_set_attention_impl")


def get_attention_impl() -> int:
    return lib().ba_get_attention_impl()


def last_attention_impl() -> int:
    return lib().ba_last_attention_impl()


def stage_timing(enable: bool):
    """Turn per-stage CUDA-event timing of attention_fwd on or off (measurement only)."""
    _check(lib().ba_stage_timing(1 if enable else 0), "ba_stage_timing")


def stage_times():
    """(ms per stage summed over calls [stream, finalize, quantise, attention], number of calls)."""
    ms = (ctypes.c_float * 4)()
    calls = ctypes.c_int(0)
    _check(lib().ba_stage_times(ms, 4, ctypes.byref(calls)), "ba_stage_times")
    return [float(x) for x in ms], calls.value


def check_device_status(stream=None):
    _check(lib().ba_check_device_status(_stream(stream)), "ba_check_device_status")


# ----------------------------------------------------------------------------- entry points
def pack_signs(x, stream=None) -> Tuple[object, object]:
    """x [B,H,N,d] fp16/bf16 -> (bits uint32-as-int32 [B,H,N,4], mu fp32 [B,H])."""
    torch = _torch()
    _qkv_check(x)
    B, H, N, d = x.shape
    bits = torch.empty((B, H, N, 4), dtype=torch.int32, device=x.device)
    mu = torch.empty((B, H), dtype=torch.float32, device=x.device)
    nws = lib().ba_pack_workspace_bytes(B, H, N, d)
    nws = 0 if nws == ctypes.c_size_t(-1).value else nws
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=x.device)
    _check(lib().ba_pack_signs(_ptr(x), _dt(x), B, H, N, d, _ptr(bits), _ptr(mu), _ptr(ws), nws,
                               _stream(stream)), "ba_pack_signs")
    return bits, mu


def quant_v(v, stream=None) -> Tuple[object, object]:
    """v [B,H,N,d] fp16/bf16 -> (vq int8 [B,H,N,v_row_bytes(d)], v_scale fp32 [B,H,d])."""
    torch = _torch()
    _qkv_check(v)
    B, H, N, d = v.shape
    vq = torch.empty((B, H, N, max(v_row_bytes(d), 1)), dtype=torch.int8, device=v.device)
    vs = torch.empty((B, H, d), dtype=torch.float32, device=v.device)
    nws = lib().ba_quant_workspace_bytes(B, H, N, d)
    nws = 0 if nws == ctypes.c_size_t(-1).value else nws
    ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=v.device)
    _check(lib().ba_quant_v(_ptr(v), _dt(v), B, H, N, d, _ptr(vq), _ptr(vs), _ptr(ws), nws, _stream(stream)),
           "ba_quant_v")
    return vq, vs


def attention_fwd_packed(bits_q, mu_q, bits_k, mu_k, vq, v_scale, d: int, bias: Optional[Bias] = None,
                         softmax_scale: float = 0.0, out=None, out_dtype=None, debug_logits: bool = False,
                         stream=None):
    """Fused step on packed operands. Returns O [B,H,N,d] (and int32 logits [B,H,N,N] if debug_logits)."""
    torch = _torch()
    B, H, N, _ = bits_q.shape
    if out is None:
        out = torch.empty((B, H, N, d), dtype=out_dtype or torch.float32, device=bits_q.device)
    dbg = torch.empty((B, H, N, N), dtype=torch.int32, device=bits_q.device) if debug_logits else None
    cb = (bias or Bias()).c()
    _check(lib().ba_attention_fwd_packed(_ptr(bits_q), _ptr(mu_q), _ptr(bits_k), _ptr(mu_k), _ptr(vq),
                                         _ptr(v_scale), B, H, N, d, ctypes.byref(cb), float(softmax_scale),
                                         _ptr(out), _dt(out), _ptr(dbg), _stream(stream)),
           "ba_attention_fwd_packed")
    return (out, dbg) if debug_logits else out


def attention_fwd(q, k, v, bias: Optional[Bias] = None, softmax_scale: float = 0.0, out=None,
                  out_dtype=None, workspace=None, debug_logits: bool = False, stream=None):
    """The whole forward pass. q, k, v [B,H,N,d] fp16/bf16 CUDA tensors."""
    torch = _torch()
    _qkv_check(q, k, v)
    if q.dtype != k.dtype or q.dtype != v.dtype or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must share dtype and shape")
    B, H, N, d = q.shape
    if out is None:
        out = torch.empty((B, H, N, d), dtype=out_dtype or q.dtype, device=q.device)
    nws = lib().ba_workspace_bytes(B, H, N, d)
    if nws == ctypes.c_size_t(-1).value:  # unsupported size: the call below reports it
        nws = 0
    if workspace is None:
        workspace = torch.empty(max(nws, 1), dtype=torch.uint8, device=q.device)
    dbg = torch.empty((B, H, N, N), dtype=torch.int32, device=q.device) if debug_logits else None
    cb = (bias or Bias()).c()
    _check(lib().ba_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _dt(q), B, H, N, d, ctypes.byref(cb),
                                  float(softmax_scale), _ptr(out), _dt(out), _ptr(workspace),
                                  workspace.numel(), _ptr(dbg), _stream(stream)), "ba_attention_fwd")
    return (out, dbg) if debug_logits else out


def attention_fwd_debug(q, k, v, bias: Optional[Bias] = None, softmax_scale: float = 0.0, out_dtype=None,
                        check_all_codes: bool = False, stream=None):
    """The whole forward pass with its debug outputs: (O, int32 logits [B,H,N,N], uint8 P codes
    [B,H,N,N]). check_all_codes recomputes every near-tie code exactly (see ba_attention_fwd_debug)."""
    torch = _torch()
    _qkv_check(q, k, v)
    B, H, N, d = q.shape
    out = torch.empty((B, H, N, d), dtype=out_dtype or q.dtype, device=q.device)
    nws = lib().ba_workspace_bytes(B, H, N, d)
    nws = 0 if nws == ctypes.c_size_t(-1).value else nws
    workspace = torch.empty(max(nws, 1), dtype=torch.uint8, device=q.device)
    dbg = torch.empty((B, H, N, N), dtype=torch.int32, device=q.device)
    dbg_p = torch.empty((B, H, N, N), dtype=torch.uint8, device=q.device)
    cb = (bias or Bias()).c()
    _check(lib().ba_attention_fwd_debug(_ptr(q), _ptr(k), _ptr(v), _dt(q), B, H, N, d, ctypes.byref(cb),
                                        float(softmax_scale), _ptr(out), _dt(out), _ptr(workspace),
                                        workspace.numel(), _ptr(dbg), _ptr(dbg_p), 1 if check_all_codes else 0,
                                        _stream(stream)), "ba_attention_fwd_debug")
    return out, dbg, dbg_p


# ----------------------------------------------------------------------------- paged cache
def kv_block_bytes(page_size: int, d: int) -> int:
    """Bytes of the cache rows of one page of one KV head (0 for unsupported sizes)."""
    return lib().ba_kv_block_bytes(page_size, d)


class KVCache:
    """A paged cache of binary K and 8-bit V rows (layout: include/binattn.h, ba_kv_cache).

    data: uint8 CUDA tensor [num_pages, n_kv_heads, kv_block_bytes(page_size, d)], contiguous.
    ``KVCache.zeros`` allocates one; any slice of a larger buffer of that shape does as well.
    """

    def __init__(self, data, page_size: int, d: int):
        self._data, self._page_size, self._d = data, page_size, d
        self._c = None  # the C description, checked when it is first asked for

    @classmethod
    def zeros(cls, num_pages: int, n_kv_heads: int, d: int, page_size: int = 64, device="cuda") -> "KVCache":
        nbytes = kv_block_bytes(page_size, d)
        if nbytes == 0:
            raise ValueError("page_size must be a multiple of 16 up to 1024, d between 1 and 128")
        torch = _torch()
        return cls(torch.zeros((num_pages, n_kv_heads, nbytes), dtype=torch.uint8, device=device), page_size, d)

    @property
    def data(self):
        return self._data

    @property
    def page_size(self) -> int:
        return self._page_size

    @property
    def d(self) -> int:
        return self._d

    @property
    def num_pages(self) -> int:
        return self._data.shape[0]

    @property
    def n_kv_heads(self) -> int:
        return self._data.shape[1]

    def _part(self, at: int, width: int):
        return self._data[:, :, self._page_size * at:self._page_size * (at + width)]

    @property
    def v_codes(self):
        """int8 codes of V [num_pages, n_kv_heads, page_size, v_row_bytes(d)] (a view)."""
        dp = v_row_bytes(self._d)
        return self._part(0, dp).view(_torch().int8).unflatten(2, (self._page_size, dp))

    @property
    def k_bits(self):
        """Sign words of K, int32 [num_pages, n_kv_heads, page_size, 4] (a view)."""
        return self._part(v_row_bytes(self._d), 16).view(_torch().int32).unflatten(2, (self._page_size, 4))

    @property
    def k_mu(self):
        """bf16 scales of K [num_pages, n_kv_heads, page_size] (a view)."""
        return self._part(v_row_bytes(self._d) + 16, 2).view(_torch().bfloat16)

    @property
    def v_exp(self):
        """int8 exponents of V [num_pages, n_kv_heads, page_size] (a view)."""
        return self._part(v_row_bytes(self._d) + 18, 1).view(_torch().int8)

    def c(self) -> CKvCache:
        t = self._data
        if self._c is None or self._c.data != t.data_ptr():
            if t.dtype != _torch().uint8 or t.dim() != 3 or not t.is_cuda or not t.is_contiguous():
                raise ValueError("cache data must be a contiguous uint8 CUDA tensor [pages, heads, block bytes]")
            if t.shape[2] != kv_block_bytes(self._page_size, self._d) or t.shape[2] == 0:
                raise ValueError("cache blocks must have kv_block_bytes(page_size, d) bytes")
            self._c = CKvCache(t.data_ptr(), t.shape[0], self._page_size, t.shape[1], self._d)
        return self._c


# The entry points below run many times per second on small tensors, so their checks, allocations and C calls
# are made by a compiled module (csrc/paged_binding.cpp). What they allocate, and their kernels, belong to the
# current stream of the cache's device; a call for another stream, or from another current device, is made
# again inside of it.
_module = None


def _native():
    global _module
    if _module is None:
        L = lib()
        torch = _torch()
        try:
            from . import _paged
            built_for = getattr(_paged, "built_for", "another torch")
        except ImportError:
            built_for = "nothing here"
        if built_for != "torch " + torch.__version__:
            raise RuntimeError(f"the module _paged has been built for {built_for}, and this is torch {torch.__version__}: "
                               "build it with `python -m bit_qk_attention_b200.build`")
        _paged.bind(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "ba_kv_block_bytes", "ba_cache_write", "ba_cache_read", "ba_paged_workspace_bytes", "ba_attention_paged")),
            torch.OutOfMemoryError)
        _module = _paged
    return _module


def _elsewhere(cache, dev: int, stream):
    """The context in which a call has to be made again, or None."""
    torch = _torch()
    if dev < 0:
        raise ValueError("cache data must be a contiguous uint8 CUDA tensor [pages, heads, block bytes]")
    if stream is not None:
        if stream.device != cache.data.device:
            raise ValueError("stream and cache must be on one device")
        return torch.cuda.stream(stream)
    return torch.cuda.device(dev) if dev != torch._C._cuda_getDevice() else None


def cache_write(cache: KVCache, k, v, slots, stream=None) -> None:
    """Quantise new rows k, v [T, n_kv_heads, d] (fp16/bf16; strided views are taken as they are)
    and write them to the tokens at slots (int64 [T], page * page_size + offset; -1 skips a row).
    Slots in range must differ."""
    data = cache._data
    dev = data.get_device()
    other = _elsewhere(cache, dev, stream)
    if other is not None:
        with other:
            return cache_write(cache, k, v, slots)
    _check(_native().write(data, cache._page_size, cache._d, k, v, slots, _torch()._C._cuda_getCurrentRawStream(dev)),
           "ba_cache_write")


def cache_read(cache: KVCache, slots, dtype=None, k_out=None, v_out=None, stream=None) -> Tuple[object, object]:
    """(k, v) [T, n_kv_heads, d]: the rows at slots (int64 [T]) as numbers; rows out of range are 0.
    dtype: fp16, bf16 (default) or fp32, or that of k_out / v_out where they are given."""
    data = cache._data
    dev = data.get_device()
    other = _elsewhere(cache, dev, stream)
    if other is not None:
        with other:
            return cache_read(cache, slots, dtype, k_out, v_out)
    r = _native().read(data, cache._page_size, cache._d, slots, dtype, k_out, v_out,
                       _torch()._C._cuda_getCurrentRawStream(dev))
    if r.__class__ is int:
        _check(r, "ba_cache_read")
    return r


def attention_paged(q, cache: KVCache, page_table, kv_lens, cu_seqlens_q=None, max_q_len: Optional[int] = None,
                    max_kv_len: Optional[int] = None, causal: bool = True, window: int = 0, sinks: int = 0,
                    softmax_scale: float = 0.0, out=None, out_dtype=None, return_lse: bool = False, workspace=None,
                    stream=None):
    """Attention of new tokens over the cache, which holds their own rows too (ba_attention_paged).

    q:            [T, n_heads, d] fp16/bf16, a strided view at will; the new tokens of all sequences.
    page_table:   int32 [B, pages]: page of each page_size tokens of a sequence.
    kv_lens:      int32 [B]: tokens in the cache, the new ones included.
    cu_seqlens_q: int32 [B + 1]: sequence b has rows cu[b] .. cu[b + 1] - 1; None: one row each.
    max_q_len, max_kv_len: host bounds of the lengths (defaults: T, and the page table's tokens).
                  Tight bounds let the launch be chosen well; lengths are read on the device.
    window:       > 0: a token sees itself and the window - 1 tokens before it, and the first `sinks`.
    workspace:    uint8 CUDA tensor of at least the bytes that paged_workspace_bytes tells for the same arguments
                  (default: allocated for the call). Calls that can overlap need one each.
    Returns o [T, n_heads, d] (out_dtype, default q's; rows of no sequence are left as they were in
    `out`), and with return_lse also the fp32 log of the softmax sums [T, n_heads].
    """
    data = cache._data
    dev = data.get_device()
    other = _elsewhere(cache, dev, stream)
    if other is not None:
        with other:
            return attention_paged(q, cache, page_table, kv_lens, cu_seqlens_q, max_q_len, max_kv_len, causal, window,
                                   sinks, softmax_scale, out, out_dtype, return_lse, workspace)
    r = _native().attend(data, cache._page_size, cache._d, q, page_table, kv_lens, cu_seqlens_q, max_q_len, max_kv_len,
                         causal, window, sinks, softmax_scale, out, out_dtype, return_lse, workspace,
                         _torch()._C._cuda_getCurrentRawStream(dev))
    if r.__class__ is int:
        _check(r, "ba_attention_paged")
    return r


def paged_workspace_bytes(q, cache: KVCache, page_table, kv_lens, cu_seqlens_q=None, max_q_len: Optional[int] = None,
                          max_kv_len: Optional[int] = None, causal: bool = True, window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that attention_paged needs for these arguments (ba_paged_workspace_bytes; 0: none). Only
    the tensors' shapes and the bounds count, so that one workspace does for every call with the same ones."""
    T, n_heads, _ = q.shape
    most = 0x7fffffff  # what a C int holds: larger bounds mean the same
    pages = page_table.shape[1]
    if max_q_len is None:
        max_q_len = T if cu_seqlens_q is not None else 1
    keys = pages * cache.page_size
    cu = None if cu_seqlens_q is None else cu_seqlens_q.data_ptr()
    seqs = CPagedSeqs(kv_lens.numel(), T, n_heads, min(max_q_len, most), keys if max_kv_len is None else min(max_kv_len, keys),
                      cu, kv_lens.data_ptr(), page_table.data_ptr(), page_table.stride(0), pages, int(causal),
                      min(window, most), min(sinks, most))
    need = lib().ba_paged_workspace_bytes(ctypes.byref(cache.c()), ctypes.byref(seqs))
    if need == ctypes.c_size_t(-1).value:
        raise ValueError("sizes or bounds that attention_paged refuses")
    return need


def bias_from_workload(w, device) -> Optional[Bias]:
    """Device Bias for a workload of bit_qk_attention_b200.inputs."""
    if w.bias_kind == BIAS_NONE or w.bias is None:
        return None
    return Bias(w.bias_kind, w.bias.to(device=device, dtype=_torch().float32).contiguous(), w.batch_stride,
                w.grid_h, w.grid_w, w.table_h, w.table_w, w.n_prefix)
