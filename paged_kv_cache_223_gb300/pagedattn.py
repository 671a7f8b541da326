"""Python binding of the C ABI in include/pagedattn.h (ctypes; argument marshalling only).

Torch tensors provide device memory and streams; every step of the paged-attention path
runs in the CUDA library. There is no fallback: if the library is missing this module
raises on load.
"""
from __future__ import annotations

import ctypes as C
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpagedattn.so")

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_CUDA, PA_ERR_OOM, PA_ERR_DEVICE_BOUNDS, PA_ERR_TIMEOUT = range(7)
PA_FP16, PA_BF16 = 0, 1
PA_KV_16BIT, PA_KV_FP8_E4M3 = 0, 1
_TORCH_DTYPE = {PA_FP16: torch.float16, PA_BF16: torch.bfloat16}
_PA_DTYPE = {torch.float16: PA_FP16, torch.bfloat16: PA_BF16}


class PaPoolConfig(C.Structure):
    _fields_ = [("num_blocks", C.c_int32), ("block_size", C.c_int32), ("num_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32), ("device", C.c_int32),
                ("partition_tokens", C.c_int32), ("max_seqs", C.c_int32), ("max_q_heads", C.c_int32),
                ("max_q_len", C.c_int32), ("max_context_len", C.c_int32), ("k_cache", C.c_void_p),
                ("v_cache", C.c_void_p), ("kv_format", C.c_int32)]


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


_lock = threading.Lock()
_lib = None


def lib() -> C.CDLL:
    """Load libpagedattn.so (built in-tree by __graft_entry__.build())."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                                   "(run `python -m paged_kv_cache_223_gb300._build`)")
            L = C.CDLL(LIB_PATH)
            P, I32, I64 = C.c_void_p, C.c_int32, C.c_int64
            L.pa_pool_create.argtypes = [C.POINTER(PaPoolConfig), C.POINTER(C.c_void_p)]
            L.pa_destroy.argtypes = [P]
            L.pa_destroy.restype = None
            L.pa_pool_caches.argtypes = [P, C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.POINTER(C.c_uint64)]
            L.pa_cache_write.argtypes = [P, P, P, P, I32, P, P, P]
            L.pa_decode.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, C.c_float, P, P]
            L.pa_prefill.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, C.c_float, P, P]
            L.pa_decode_shared_prefix.argtypes = [P, P, P, P, P, I32, P, I32, I32, I32, C.c_float, I32, P, P]
            L.pa_pool_check.argtypes = [P, P]
            L.pa_pool_selftest_wait.argtypes = [P, C.c_uint64, P]
            L.pa_pool_selftest_wait.restype = C.c_int
            L.pa_decode_launches.argtypes = [P, I32, I32, I32, I32]
            L.pa_decode_launches.restype = I32
            L.pa_status_string.argtypes = [C.c_int]
            L.pa_status_string.restype = C.c_char_p
            for f in ("pa_pool_create", "pa_pool_caches", "pa_cache_write", "pa_decode", "pa_prefill", "pa_decode_shared_prefix",
                      "pa_pool_check"):
                getattr(L, f).restype = C.c_int
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().pa_status_string(status).decode()


def _check(status: int, what: str) -> None:
    if status != PA_OK:
        raise PagedAttnError(status, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    """The CUDA stream handle: the given stream's, else the current device's current stream (read as a raw
    handle where torch offers it: building a torch Stream object costs about 3 us per call)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _dev(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, index: int, shape: tuple) -> None:
    """A contiguous tensor of this type and shape on device `index` (one test of each: this is on every call's path)."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _stream_on(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    """The given stream's handle (a stream of `device`), else that device's current stream."""
    if stream is None:
        return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return stream.cuda_stream


def _new(shape, dtype: torch.dtype, device: torch.device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A tensor that the call writes on `stream`: allocated there, and kept for work queued on the current stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _token_rows(t: torch.Tensor, name: str, dtype: torch.dtype, index: int, n: int, heads: int, d: int) -> int:
    """Token rows [n, heads, d]: heads and dimensions dense, tokens at any stride of whole 16-byte vectors.
    Returns that stride in elements."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n, heads, d):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(n, heads, d)} on cuda:{index}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    st, sh, sd = t.stride()
    if n <= 1:
        st = heads * d
    if (sd != 1 or (sh != d and heads > 1) or st < heads * d or st % 8) and t.numel():
        raise ValueError(f"{name} must have dense heads and a token stride of whole 16-byte vectors, got strides "
                         f"{t.stride()}")
    return st


class Rope:
    """Rotary frequencies on the device (pa_rope_create): pair i turns by position * inv_freq[i] radians.

    inv_freq: rot_dim / 2 frequencies. interleaved: pairs are neighbouring dimensions (2i, 2i + 1) instead of
    (i, i + rot_dim / 2). scale: factor on every cosine and sine."""

    def __init__(self, inv_freq, interleaved: bool = False, scale: float = 1.0, device: int = 0):
        f = [float(x) for x in inv_freq]
        self.rot_dim, self.device = 2 * len(f), torch.device("cuda", device)
        h = C.c_void_p()
        self._h = None
        _check(_serving_lib().pa_rope_create((C.c_double * max(1, len(f)))(*f), self.rot_dim, int(bool(interleaved)),
                                             float(scale), device, C.byref(h)), "pa_rope_create")
        self._h = h

    @classmethod
    def from_base(cls, rot_dim: int, base: float = 10000.0, **kw) -> "Rope":
        """Frequencies base ** (-2i / rot_dim), i < rot_dim / 2."""
        if rot_dim % 2:
            raise ValueError(f"rot_dim must be even, got {rot_dim}")
        return cls([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], **kw)

    @property
    def handle(self) -> C.c_void_p:
        if self._h is None:
            raise RuntimeError("rope is closed")
        return self._h

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            _serving_lib().pa_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_serving_ready = False


class PaLogitsArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("dtype", C.c_int32), ("num_seqs", C.c_int32), ("rows_per_seq", C.c_int32),
                ("num_bias", C.c_int32), ("vocab", C.c_int64), ("seq_stride", C.c_int64), ("row_stride", C.c_int64),
                ("history", C.c_void_p), ("history_stride", C.c_int64), ("history_lens", C.c_void_p),
                ("prompt_lens", C.c_void_p), ("draft", C.c_void_p), ("repetition", C.c_void_p),
                ("presence", C.c_void_p), ("frequency", C.c_void_p), ("bias_tokens", C.c_void_p),
                ("bias_values", C.c_void_p), ("mask", C.c_void_p), ("temperature", C.c_void_p), ("out", C.c_void_p)]


def _serving_lib() -> C.CDLL:
    global _serving_ready
    if _serving_ready:
        return _lib
    L = lib()
    if not _serving_ready:
        P, I32, I64, U64 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64
        L.pa_rope_create.argtypes = [C.POINTER(C.c_double), I32, I32, C.c_float, I32, C.POINTER(C.c_void_p)]
        L.pa_rope_destroy.argtypes = [P]
        L.pa_rope_destroy.restype = None
        L.pa_rope_append.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, I32, I32, P, I64, P, P, P]
        L.pa_prefill_packed_workspace.argtypes = [P, I32, I32, I32, I32, C.POINTER(U64)]
        L.pa_prefill_packed.argtypes = [P, P, P, P, P, P, I32, P, I32, I32, I32, C.c_float, P, U64, P, P]
        L.pa_adjust_logits.argtypes = [C.POINTER(PaLogitsArgs), P]
        L.pa_token_probs.argtypes = [C.POINTER(PaLogitsArgs), P]
        for f in ("pa_rope_create", "pa_rope_append", "pa_prefill_packed_workspace", "pa_prefill_packed",
                  "pa_adjust_logits", "pa_token_probs"):
            getattr(L, f).restype = C.c_int
        _serving_ready = True
    return L


_sparse_fns = None


class PaTablesArgs(C.Structure):
    _fields_ = [("num_seqs", C.c_int32), ("num_tokens", C.c_int32), ("block_table_stride", C.c_int32),
                ("new_lens", C.c_void_p), ("keep_lens", C.c_void_p), ("context_lens", C.c_void_p),
                ("block_tables", C.c_void_p), ("free_blocks", C.c_void_p), ("num_free", C.c_void_p), ("cu_q", C.c_void_p),
                ("positions", C.c_void_p), ("slot_mapping", C.c_void_p)]


def _sparse_lib() -> C.CDLL:
    """The library with the sparse decode step's calls declared (and kept by name: this is on every call's path)."""
    global _sparse_fns
    L = lib()
    if _sparse_fns is None:
        P, I32 = C.c_void_p, C.c_int32
        L.pa_step_tables.argtypes = [P, C.POINTER(PaTablesArgs), P]
        L.pa_key_bounds_size.argtypes = [P, C.POINTER(C.c_uint64)]
        L.pa_key_bounds.argtypes = [P, P, P, P, I32, P, I32, I32, P, P]
        L.pa_select_blocks.argtypes = [P, P, P, P, I32, P, I32, I32, I32, I32, I32, I32, P, P]
        L.pa_decode_selected.argtypes = [P, P, P, P, P, I32, P, I32, P, I32, I32, I32, C.c_float, P, P]
        fns = {f: getattr(L, f) for f in ("pa_step_tables", "pa_key_bounds_size", "pa_key_bounds", "pa_select_blocks",
                                          "pa_decode_selected")}
        for f in fns.values():
            f.restype = C.c_int
        _sparse_fns = fns
    return L


def _sparse_call(name: str, *args) -> None:
    if _sparse_fns is None:
        _sparse_lib()
    status = _sparse_fns[name](*args)
    if status:
        raise PagedAttnError(status, name)


def _int32(x: int, name: str) -> int:
    """A count as the C call takes it: ctypes would drop the bits above 32."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


class Pool:
    """One paged KV pool (pa_pool_create) with its caches.

    The caches are torch tensors, created here unless given; the pool only borrows them.
    16-bit pools: [num_blocks, num_kv_heads, block_size, head_dim] of the model dtype.
    FP8 pools (kv_format=PA_KV_FP8_E4M3): one uint8 buffer each of num_blocks*Hkv*bs*(head_dim + 4)
    bytes (codes, then float32 scales).
    """

    def __init__(self, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                 dtype: torch.dtype = torch.float16, device: int = 0, partition_tokens: int = 0,
                 max_seqs: int = 256, max_q_heads: int = 64, max_q_len: int = 8, max_context_len: int = 8192,
                 k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                 kv_format: int = PA_KV_16BIT):
        self.geometry = (num_blocks, num_kv_heads, block_size, head_dim)
        self.dtype = dtype
        self.kv_format = kv_format
        self.device = torch.device("cuda", device)
        if kv_format == PA_KV_FP8_E4M3:
            shape, cdt = (num_blocks * num_kv_heads * block_size * (head_dim + 4),), torch.uint8
        else:
            shape, cdt = self.geometry, dtype
        if k_cache is None:
            k_cache = torch.empty(shape, dtype=cdt, device=self.device)
            v_cache = torch.empty(shape, dtype=cdt, device=self.device)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            _dev(t, name, cdt)
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} must have shape {tuple(shape)}")
        self.k_cache, self.v_cache = k_cache, v_cache
        cfg = PaPoolConfig(num_blocks, block_size, num_kv_heads, head_dim, _PA_DTYPE[dtype], device,
                           partition_tokens, max_seqs, max_q_heads, max_q_len, max_context_len,
                           k_cache.data_ptr(), v_cache.data_ptr(), kv_format)
        h = C.c_void_p()
        _check(lib().pa_pool_create(C.byref(cfg), C.byref(h)), "pa_pool_create")
        self._h = h

    @property
    def handle(self) -> C.c_void_p:
        if self._h is None:
            raise RuntimeError("pool is closed")
        return self._h

    def close(self) -> None:
        if getattr(self, "_h", None) is not None:
            lib().pa_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check_caches(self, k_cache: Optional[torch.Tensor], v_cache: Optional[torch.Tensor]) -> None:
        """Caches passed per call replace the pool's own: both or neither, each of the pool's shape."""
        if (k_cache is None) != (v_cache is None):
            raise ValueError("pass both k_cache and v_cache, or neither")
        if k_cache is not None:
            for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
                _dev(t, name, self.k_cache.dtype)
                if tuple(t.shape) != tuple(self.k_cache.shape):
                    raise ValueError(f"{name} must have shape {tuple(self.k_cache.shape)}")

    def _attn_args(self, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                   out: Optional[torch.Tensor]) -> torch.Tensor:
        """Checks the shapes the library trusts (it sees only pointers) and returns out."""
        _dev(q, "q", self.dtype)
        _dev(block_tables, "block_tables", torch.int32)
        _dev(context_lens, "context_lens", torch.int32)
        d = self.geometry[3]
        if q.dim() != 4 or q.shape[3] != d:
            raise ValueError(f"q must be [B, q_len, Hq, {d}], got {tuple(q.shape)}")
        B = q.shape[0]
        if block_tables.dim() != 2 or block_tables.shape[0] < B:
            raise ValueError(f"block_tables must be [>= {B}, stride], got {tuple(block_tables.shape)}")
        if context_lens.dim() != 1 or context_lens.shape[0] < B:
            raise ValueError(f"context_lens must hold {B} entries, got {tuple(context_lens.shape)}")
        if out is None:
            out = torch.empty_like(q)
        _dev(out, "out", self.dtype)
        if tuple(out.shape) != tuple(q.shape):
            raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
        return out

    def cache_write(self, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                    k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
        """Scatter k, v [N, Hkv, d] into the slots given by slot_mapping (int64 [N]; -1 = skip)."""
        _dev(k, "k", self.dtype), _dev(v, "v", self.dtype), _dev(slot_mapping, "slot_mapping", torch.int64)
        hd = (self.geometry[1], self.geometry[3])
        if k.dim() != 3 or tuple(k.shape[1:]) != hd or tuple(v.shape) != tuple(k.shape):
            raise ValueError(f"k and v must be [N, {hd[0]}, {hd[1]}], got {tuple(k.shape)} and {tuple(v.shape)}")
        if slot_mapping.dim() != 1 or slot_mapping.shape[0] != k.shape[0]:
            raise ValueError(f"slot_mapping must be [{k.shape[0]}], got {tuple(slot_mapping.shape)}")
        self._check_caches(k_cache, v_cache)
        _check(lib().pa_cache_write(self.handle, _ptr(k), _ptr(v), _ptr(slot_mapping), slot_mapping.numel(),
                                    _ptr(k_cache), _ptr(v_cache), _stream(stream)), "pa_cache_write")

    def decode(self, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
               out: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
               v_cache: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Paged attention for q [B, q_len, Hq, d] -> out [B, q_len, Hq, d] (causal over the q_len rows)."""
        out = self._attn_args(q, block_tables, context_lens, out)
        self._check_caches(k_cache, v_cache)
        B, q_len, Hq, d = q.shape
        _check(lib().pa_decode(self.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               block_tables.shape[1], _ptr(context_lens), B, Hq, q_len, float(scale), _ptr(out),
                               _stream(stream)), "pa_decode")
        return out

    def decode_shared_prefix(self, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                             scale: float, prefix_tokens: int, out: Optional[torch.Tensor] = None,
                             k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """pa_decode_shared_prefix: decode for sequences whose tables share their first prefix_tokens tokens."""
        out = self._attn_args(q, block_tables, context_lens, out)
        self._check_caches(k_cache, v_cache)
        B, q_len, Hq, d = q.shape
        _check(lib().pa_decode_shared_prefix(self.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                             block_tables.shape[1], _ptr(context_lens), B, Hq, q_len, float(scale),
                                             int(prefix_tokens), _ptr(out), _stream(stream)),
               "pa_decode_shared_prefix")
        return out

    def prefill(self, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float,
                out: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                v_cache: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Chunked prefill (pa_prefill): q [B, C, Hq, 128] is a chunk of C new tokens per sequence, causal."""
        out = self._attn_args(q, block_tables, context_lens, out)
        self._check_caches(k_cache, v_cache)
        B, q_len, Hq, d = q.shape
        _check(lib().pa_prefill(self.handle, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                block_tables.shape[1], _ptr(context_lens), B, Hq, q_len, float(scale), _ptr(out),
                                _stream(stream)), "pa_prefill")
        return out

    def rope_append(self, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                    slot_mapping: torch.Tensor, rope: "Rope", q_out: Optional[torch.Tensor] = None,
                    k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
        """Rotate q [N, Hq, d] and k [N, Hkv, d] by positions (int32 [N]) and append k, v to the pool's slots
        (pa_rope_append). Rows may be strided over tokens (slices of one projection's output). Returns the
        rotated q [N, Hq, d] (q_out; may be q itself); q None appends only."""
        _, hkv, _, d = self.geometry
        index, dt = self.device.index, self.dtype
        n = k.shape[0]
        ks = _token_rows(k, "k", dt, index, n, hkv, d)
        vs = _token_rows(v, "v", dt, index, n, hkv, d)
        _need(positions, "positions", torch.int32, index, (n,))
        _need(slot_mapping, "slot_mapping", torch.int64, index, (n,))
        if k_cache is not None or v_cache is not None:
            self._check_caches(k_cache, v_cache)
        hq = qs = os = 0
        if q is not None:
            if q.dim() != 3:
                raise ValueError(f"q must be [{n}, Hq, {d}], got {tuple(q.shape)}")
            hq = q.shape[1]
            qs = _token_rows(q, "q", dt, index, n, hq, d)
            if q_out is None:
                q_out, os = _new((n, hq, d), dt, self.device, stream), hq * d
            else:
                os = _token_rows(q_out, "q_out", dt, index, n, hq, d)
        elif q_out is not None:
            raise ValueError("q_out without q")
        _check(_serving_lib().pa_rope_append(
            self.handle, rope.handle, _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(),
            slot_mapping.data_ptr(), n, hq, _ptr(q_out), os, _ptr(k_cache), _ptr(v_cache),
            _stream_on(stream, self.device)), "pa_rope_append")
        return q_out

    def prefill_packed(self, q: torch.Tensor, cu_q: torch.Tensor, block_tables: torch.Tensor,
                       context_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                       k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Causal attention of packed prompts (pa_prefill_packed): rows cu_q[b]..cu_q[b+1] of q [T, Hq, d] are
        sequence b's newest tokens, their K and V already in the pool. cu_q: int32 [B + 1]. The workspace
        (uint8, packed_workspace() bytes) is allocated for the call unless given; calls that may run at the
        same time need one each."""
        index, dt = self.device.index, self.dtype
        if q.dim() != 3 or cu_q.dim() != 1 or cu_q.shape[0] < 1 or block_tables.dim() != 2 or context_lens.dim() != 1:
            raise ValueError(f"q must be [T, Hq, d], cu_q [B + 1], block_tables [>= B, stride], context_lens [>= B]: got "
                             f"{tuple(q.shape)}, {tuple(cu_q.shape)}, {tuple(block_tables.shape)}, "
                             f"{tuple(context_lens.shape)}")
        (T, Hq, _), B = q.shape, cu_q.shape[0] - 1
        rows, stride = block_tables.shape
        lens = context_lens.shape[0]
        if rows < B or lens < B:
            raise ValueError(f"block_tables and context_lens must hold {B} sequences, got {rows} and {lens}")
        _need(q, "q", dt, index, (T, Hq, self.geometry[3]))
        _need(cu_q, "cu_q", torch.int32, index, (B + 1,))
        _need(block_tables, "block_tables", torch.int32, index, (rows, stride))
        _need(context_lens, "context_lens", torch.int32, index, (lens,))
        if out is None:
            out = _new(q.shape, dt, self.device, stream)
        else:
            _need(out, "out", dt, index, q.shape)
        if k_cache is not None or v_cache is not None:
            self._check_caches(k_cache, v_cache)
        size = 0
        if workspace is not None:
            size = workspace.numel()
            _need(workspace, "workspace", torch.uint8, index, (size,))
        else:
            size = self.packed_workspace(T, B, Hq, stride)
            if size:
                workspace = _new((size,), torch.uint8, self.device, stream)
        _check(_serving_lib().pa_prefill_packed(
            self.handle, q.data_ptr(), _ptr(k_cache), _ptr(v_cache), cu_q.data_ptr(), block_tables.data_ptr(), stride,
            context_lens.data_ptr(), T, B, Hq, float(scale), _ptr(workspace), size, out.data_ptr(),
            _stream_on(stream, self.device)), "pa_prefill_packed")
        return out

    def packed_workspace(self, num_tokens: int, num_seqs: int, num_q_heads: int, block_table_stride: int) -> int:
        """Workspace bytes of prefill_packed for these sizes (pa_prefill_packed_workspace; 0: none is needed)."""
        n = C.c_uint64()
        _check(_serving_lib().pa_prefill_packed_workspace(self.handle, num_tokens, num_seqs, num_q_heads,
                                                          block_table_stride, n), "pa_prefill_packed_workspace")
        return n.value

    def step_tables(self, new_lens: torch.Tensor, context_lens: torch.Tensor, block_tables: torch.Tensor,
                    free_blocks: torch.Tensor, num_free: torch.Tensor, num_tokens: int,
                    keep_lens: Optional[torch.Tensor] = None, cu_q: Optional[torch.Tensor] = None,
                    positions: Optional[torch.Tensor] = None, slot_mapping: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """The tables of a step on the device (pa_step_tables): sequences are cut back to keep_lens, given new_lens
        tokens and the blocks that these need. context_lens [B], block_tables [B, stride], free_blocks
        [num_blocks] (a stack of num_free[0] ids) and num_free [1] are changed in place (all int32). Returns
        cu_q int32 [B + 1], positions int32 and slot_mapping int64 [num_tokens]: 0 and -1 behind the last token."""
        index, i32, num_tokens = self.device.index, torch.int32, _int32(num_tokens, "num_tokens")
        if new_lens.dim() != 1 or block_tables.dim() != 2:
            raise ValueError(f"new_lens must be [B], block_tables [B, stride]: got {tuple(new_lens.shape)}, "
                             f"{tuple(block_tables.shape)}")
        B, stride = new_lens.shape[0], block_tables.shape[1]
        _need(new_lens, "new_lens", i32, index, (B,))
        _need(context_lens, "context_lens", i32, index, (B,))
        _need(block_tables, "block_tables", i32, index, (B, stride))
        _need(free_blocks, "free_blocks", i32, index, (self.geometry[0],))
        _need(num_free, "num_free", i32, index, (1,))
        if keep_lens is not None:
            _need(keep_lens, "keep_lens", i32, index, (B,))
        if num_tokens < 0:
            raise ValueError(f"num_tokens must not be negative, got {num_tokens}")
        if cu_q is None:
            cu_q = _new((B + 1,), i32, self.device, stream)
        else:
            _need(cu_q, "cu_q", i32, index, (B + 1,))
        if positions is None:
            positions = _new((num_tokens,), i32, self.device, stream)
        else:
            _need(positions, "positions", i32, index, (num_tokens,))
        if slot_mapping is None:
            slot_mapping = _new((num_tokens,), torch.int64, self.device, stream)
        else:
            _need(slot_mapping, "slot_mapping", torch.int64, index, (num_tokens,))
        a = PaTablesArgs(B, num_tokens, stride, new_lens.data_ptr(), _ptr(keep_lens), context_lens.data_ptr(),
                         block_tables.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr(), cu_q.data_ptr(),
                         positions.data_ptr(), slot_mapping.data_ptr())
        _sparse_call("pa_step_tables", self.handle, a, _stream_on(stream, self.device))
        return cu_q, positions, slot_mapping

    def bounds_size(self) -> int:
        """Bytes of the bounds of one cache of this pool's geometry (pa_key_bounds_size)."""
        n = C.c_uint64()
        _sparse_call("pa_key_bounds_size", self.handle, n)
        return n.value

    def new_bounds(self) -> torch.Tensor:
        """A bounds buffer for one cache (uint8, zeros: every block scores 0 until key_bounds has seen it)."""
        return torch.zeros(self.bounds_size(), dtype=torch.uint8, device=self.device)

    def _bounds(self, bounds: torch.Tensor) -> torch.Tensor:
        nb, hkv, _, d = self.geometry
        _need(bounds, "bounds", torch.uint8, self.device.index, (nb * hkv * (2 * d + 4),))
        return bounds

    def key_bounds(self, bounds: torch.Tensor, cu_q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                   num_tokens: int, k_cache: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Bounds of the keys of every block that holds one of the newest tokens (pa_key_bounds): sequence b's are
        the cu_q[b + 1] - cu_q[b] tokens up to context_lens[b], num_tokens at most in all. Changes and returns bounds."""
        index = self.device.index
        if cu_q.dim() != 1 or cu_q.shape[0] < 1 or block_tables.dim() != 2 or context_lens.dim() != 1:
            raise ValueError(f"cu_q must be [B + 1], block_tables [>= B, stride], context_lens [>= B]: got "
                             f"{tuple(cu_q.shape)}, {tuple(block_tables.shape)}, {tuple(context_lens.shape)}")
        B, (rows, stride), lens = cu_q.shape[0] - 1, block_tables.shape, context_lens.shape[0]
        if rows < B or lens < B:
            raise ValueError(f"block_tables and context_lens must hold {B} sequences, got {rows} and {lens}")
        self._bounds(bounds)
        _need(cu_q, "cu_q", torch.int32, index, (B + 1,))
        _need(block_tables, "block_tables", torch.int32, index, (rows, stride))
        _need(context_lens, "context_lens", torch.int32, index, (lens,))
        if k_cache is not None:
            _need(k_cache, "k_cache", self.k_cache.dtype, index, self.k_cache.shape)
        _sparse_call("pa_key_bounds", self.handle, _ptr(k_cache), cu_q.data_ptr(), block_tables.data_ptr(), stride,
                     context_lens.data_ptr(), _int32(num_tokens, "num_tokens"), B, bounds.data_ptr(),
                     _stream_on(stream, self.device))
        return bounds

    def _rows(self, q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor) -> tuple:
        """Checks q [B, q_len, Hq, d] and what goes with it; returns (device index, q's shape, the tables' stride)."""
        index, d = self.device.index, self.geometry[3]
        shape, tables, lens = q.shape, block_tables.shape, context_lens.shape
        if len(shape) != 4 or len(tables) != 2 or len(lens) != 1 or tables[0] < shape[0] or lens[0] < shape[0]:
            raise ValueError(f"q must be [B, q_len, Hq, {d}], block_tables [>= B, stride], context_lens [>= B]: got "
                             f"{tuple(shape)}, {tuple(tables)}, {tuple(lens)}")
        _need(q, "q", self.dtype, index, (shape[0], shape[1], shape[2], d))
        _need(block_tables, "block_tables", torch.int32, index, tables)
        _need(context_lens, "context_lens", torch.int32, index, lens)
        return index, shape, tables[1]

    def select_blocks(self, q: torch.Tensor, bounds: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                      budget: int, num_first: int = 1, num_last: int = 2, out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """The budget best blocks for each sequence and KV head of q [B, q_len, Hq, d] by the bounds' scores
        (pa_select_blocks), the first num_first and the last num_last always among them: int32 [B, Hkv, budget],
        ascending, -1 behind the last."""
        (index, (B, q_len, Hq, _), stride), budget = self._rows(q, block_tables, context_lens), _int32(budget, "budget")
        self._bounds(bounds)
        shape = (B, self.geometry[1], max(budget, 0))
        if out is None:
            out = _new(shape, torch.int32, self.device, stream)
        else:
            _need(out, "out", torch.int32, index, shape)
        _sparse_call("pa_select_blocks", self.handle, q.data_ptr(), bounds.data_ptr(), block_tables.data_ptr(), stride,
                     context_lens.data_ptr(), B, Hq, q_len, budget, _int32(num_first, "num_first"),
                     _int32(num_last, "num_last"), out.data_ptr(), _stream_on(stream, self.device))
        return out

    def decode_selected(self, q: torch.Tensor, selected: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
                        k_cache: Optional[torch.Tensor] = None, v_cache: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """decode over the listed blocks only (pa_decode_selected): selected int32 [B, Hkv, budget] names blocks of
        each sequence by their place in its table, negative entries are skipped."""
        index, shape, stride = self._rows(q, block_tables, context_lens)
        if selected.dim() != 3:
            raise ValueError(f"selected must be [B, Hkv, budget], got {tuple(selected.shape)}")
        (B, q_len, Hq, _), budget = shape, selected.shape[2]
        _need(selected, "selected", torch.int32, index, (B, self.geometry[1], budget))
        if out is not None:
            _need(out, "out", self.dtype, index, shape)
        elif stream is None:
            out = torch.empty_like(q)
        else:
            out = _new(shape, self.dtype, self.device, stream)
        if (k_cache is None) != (v_cache is None):
            raise ValueError("pass both k_cache and v_cache, or neither")
        if k_cache is not None:
            _need(k_cache, "k_cache", self.k_cache.dtype, index, self.k_cache.shape)
            _need(v_cache, "v_cache", self.v_cache.dtype, index, self.v_cache.shape)
        _sparse_call("pa_decode_selected", self.handle, q.data_ptr(), _ptr(k_cache), _ptr(v_cache), selected.data_ptr(), budget,
                     block_tables.data_ptr(), stride, context_lens.data_ptr(), B, Hq, q_len, float(scale), out.data_ptr(),
                     _stream_on(stream, self.device))
        return out

    def launches(self, block_table_stride: int, num_seqs: int, num_q_heads: int, q_len: int) -> int:
        return lib().pa_decode_launches(self.handle, block_table_stride, num_seqs, num_q_heads, q_len)

    def selftest_wait(self, limit_ns: int, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Run the bounded-wait self-test kernel (a wait that nothing completes; see pa_pool_selftest_wait)."""
        _check(lib().pa_pool_selftest_wait(self.handle, limit_ns, _stream(stream)), "pa_pool_selftest_wait")

    def check(self, stream: Optional[torch.cuda.Stream] = None) -> int:
        """Synchronise and return (and clear) the device status: PA_OK, PA_ERR_DEVICE_BOUNDS, PA_ERR_TIMEOUT or PA_ERR_OOM (a step
        of step_tables without blocks; beside one of the others the next call tells it)."""
        return lib().pa_pool_check(self.handle, _stream(stream))


def pool_create_status(**cfg) -> int:
    """pa_pool_create's status for a raw config (host-side validation; destroys the pool on success)."""
    c = PaPoolConfig(**cfg)
    h = C.c_void_p()
    st = lib().pa_pool_create(C.byref(c), C.byref(h))
    if st == PA_OK:
        lib().pa_destroy(h)
    return st


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024   # PA_NOALLOC_SCRATCH_BYTES
_noalloc_ready = False


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   context_lens: torch.Tensor, scale: float, out: torch.Tensor, partition_tokens: int = 0,
                   stream: Optional[torch.cuda.Stream] = None) -> int:
    """pa_decode_noalloc: the paged decode for callers that cannot allocate device memory.

    The caches carry the pool geometry ([num_blocks, Hkv, block_size, d]); the split workspace is the
    library's static device array, so nothing is allocated. Returns the pa_status code."""
    global _noalloc_ready
    L = lib()
    if not _noalloc_ready:
        P, I32 = C.c_void_p, C.c_int32
        L.pa_decode_noalloc.argtypes = [P, P, P, I32, I32, I32, I32, I32, P, I32, P, I32, I32, I32, C.c_float, I32,
                                        P, P]
        L.pa_decode_noalloc.restype = C.c_int
        _noalloc_ready = True
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("out", out)):
        _dev(t, name, q.dtype)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(context_lens, "context_lens", torch.int32)
    if k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache must both be [num_blocks, Hkv, block_size, d]")
    NB, Hkv, bs, d = k_cache.shape
    if q.dim() != 4 or q.shape[3] != d or tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"q and out must be [B, q_len, Hq, {d}], got {tuple(q.shape)} and {tuple(out.shape)}")
    B, q_len, Hq, _ = q.shape
    if block_tables.dim() != 2 or block_tables.shape[0] < B or context_lens.dim() != 1 or context_lens.shape[0] < B:
        raise ValueError("block_tables must be [>= B, stride] and context_lens [>= B]")
    return L.pa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), NB, bs, Hkv, d, _PA_DTYPE[q.dtype],
                               _ptr(block_tables), block_tables.shape[1], _ptr(context_lens), B, Hq, q_len,
                               float(scale), partition_tokens, _ptr(out), _stream(stream))


# ------------------------------------------------------------------------------ block manager

_alloc_ready = False


def _alloc_lib() -> C.CDLL:
    global _alloc_ready
    L = lib()
    if not _alloc_ready:
        P, I32 = C.c_void_p, C.c_int32
        L.pa_allocator_create.argtypes = [I32, I32, C.POINTER(C.c_void_p)]
        L.pa_allocator_destroy.argtypes = [P]
        L.pa_allocator_destroy.restype = None
        L.pa_allocator_num_free.argtypes = [P]
        L.pa_allocator_num_free.restype = I32
        L.pa_allocator_ref_count.argtypes = [P, I32]
        L.pa_allocator_ref_count.restype = I32
        L.pa_allocator_alloc.argtypes = [P, I32, P]
        L.pa_allocator_fork.argtypes = [P, P, I32]
        L.pa_allocator_free.argtypes = [P, P, I32]
        L.pa_allocator_cow.argtypes = [P, I32, C.POINTER(C.c_int32), C.POINTER(C.c_int32)]
        L.pa_allocator_append.argtypes = [P, P, I32, C.POINTER(C.c_int32), I32, P, P, C.POINTER(C.c_int32)]
        L.pa_copy_blocks.argtypes = [P, P, I32, P, P, P]
        for f in ("pa_allocator_create", "pa_allocator_alloc", "pa_allocator_fork", "pa_allocator_free",
                  "pa_allocator_cow", "pa_allocator_append", "pa_copy_blocks"):
            getattr(L, f).restype = C.c_int
        _alloc_ready = True
    return L


class BlockAllocator:
    """Host-side free pool with reference counts and copy-on-write (pa_allocator_*). No GPU needed."""

    def __init__(self, num_blocks: int, block_size: int):
        import numpy as np
        self._np = np
        self.block_size = block_size
        h = C.c_void_p()
        _check(_alloc_lib().pa_allocator_create(num_blocks, block_size, C.byref(h)), "pa_allocator_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None:
            _alloc_lib().pa_allocator_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _ids(self, ids):
        return self._np.ascontiguousarray(ids, dtype=self._np.int32)

    @property
    def num_free(self) -> int:
        return _alloc_lib().pa_allocator_num_free(self._h)

    def ref_count(self, block_id: int) -> int:
        return _alloc_lib().pa_allocator_ref_count(self._h, block_id)

    def alloc(self, n: int):
        out = self._np.empty(n, dtype=self._np.int32)
        _check(_alloc_lib().pa_allocator_alloc(self._h, n, out.ctypes.data), "pa_allocator_alloc")
        return out

    def fork(self, ids) -> None:
        a = self._ids(ids)
        _check(_alloc_lib().pa_allocator_fork(self._h, a.ctypes.data, len(a)), "pa_allocator_fork")

    def free(self, ids) -> None:
        a = self._ids(ids)
        _check(_alloc_lib().pa_allocator_free(self._h, a.ctypes.data, len(a)), "pa_allocator_free")

    def cow(self, block_id: int):
        out, copy = C.c_int32(), C.c_int32()
        _check(_alloc_lib().pa_allocator_cow(self._h, block_id, C.byref(out), C.byref(copy)), "pa_allocator_cow")
        return out.value, bool(copy.value)

    def append(self, table_row, length: int, n_new: int):
        """Extend a sequence by n_new tokens. table_row: int32 numpy row, updated in place.
        Returns (slots int64[n_new], new length, copy pair or None)."""
        assert table_row.dtype == self._np.int32 and table_row.flags.c_contiguous
        slots = self._np.empty(n_new, dtype=self._np.int64)
        pair = self._np.empty(2, dtype=self._np.int32)
        ln, nc = C.c_int32(length), C.c_int32()
        _check(_alloc_lib().pa_allocator_append(self._h, table_row.ctypes.data, len(table_row), C.byref(ln), n_new,
                                                slots.ctypes.data, pair.ctypes.data, C.byref(nc)), "pa_allocator_append")
        return slots, ln.value, (tuple(int(x) for x in pair) if nc.value else None)


def copy_blocks(pool: "Pool", pairs: torch.Tensor, k_cache: Optional[torch.Tensor] = None,
                v_cache: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """pa_copy_blocks: copy whole blocks pairs[i, 0] -> pairs[i, 1] (device int32 [n, 2])."""
    _dev(pairs, "pairs", torch.int32)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError(f"pairs must be [n, 2], got {tuple(pairs.shape)}")
    pool._check_caches(k_cache, v_cache)
    _check(_alloc_lib().pa_copy_blocks(pool.handle, _ptr(pairs), pairs.shape[0], _ptr(k_cache), _ptr(v_cache),
                                       _stream(stream)), "pa_copy_blocks")


_spec_ready = False


def spec_verify(p: torch.Tensor, q: torch.Tensor, draft: torch.Tensor, u: torch.Tensor, v: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None):
    """pa_spec_verify: speculative rejection sampling. Returns (out int32 [B, K+1], n_out int32 [B])."""
    global _spec_ready
    L = lib()
    if not _spec_ready:
        P, I32 = C.c_void_p, C.c_int32
        L.pa_spec_verify.argtypes = [P, P, P, P, P, I32, I32, C.c_int64, P, P, P]
        L.pa_spec_verify.restype = C.c_int
        _spec_ready = True
    for name, t, dt in (("p", p, torch.float32), ("q", q, torch.float32), ("draft", draft, torch.int32),
                        ("u", u, torch.float32), ("v", v, torch.float32)):
        _dev(t, name, dt)
    if p.dim() != 3:
        raise ValueError(f"p must be [B, K + 1, V], got {tuple(p.shape)}")
    B, K1, V = p.shape
    for name, t, shape in (("q", q, (B, K1 - 1, V)), ("draft", draft, (B, K1 - 1)), ("u", u, (B, K1 - 1)),
                           ("v", v, (B,))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    out = torch.empty((B, K1), dtype=torch.int32, device=p.device)
    n_out = torch.empty((B,), dtype=torch.int32, device=p.device)
    _check(L.pa_spec_verify(_ptr(p), _ptr(q), _ptr(draft), _ptr(u), _ptr(v), B, K1 - 1, V, _ptr(out), _ptr(n_out),
                            _stream(stream)), "pa_spec_verify")
    return out, n_out


_LOGITS_DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _logits_call(name: str, logits: torch.Tensor, temperature: Optional[torch.Tensor], history, history_lens,
                 prompt_lens, draft, repetition, presence, frequency, bias_tokens, bias_values, mask, out,
                 stream) -> torch.Tensor:
    code, index = _LOGITS_DTYPE.get(logits.dtype), logits.get_device()
    if code is None or index < 0:
        raise ValueError(f"logits must be a CUDA tensor of fp16, bf16 or fp32, got {logits.dtype} on {logits.device}")
    if logits.dim() != 3 or logits.shape[1] < 1 or logits.shape[2] < 1:
        raise ValueError(f"logits must be [B, R, V], got {tuple(logits.shape)}")
    (B, R, V), (sb, sr, sv) = logits.shape, logits.stride()
    if sv != 1 and V > 1:
        raise ValueError("logits must be dense over the vocabulary")
    i32, f32 = torch.int32, torch.float32
    S = NB = 0
    if history is not None:
        if history.dim() != 2 or history_lens is None:
            raise ValueError("history must be [B, S], with history_lens")
        S = history.shape[1]
        _need(history, "history", i32, index, (B, S))
        _need(history_lens, "history_lens", i32, index, (B,))
        if prompt_lens is not None:
            _need(prompt_lens, "prompt_lens", i32, index, (B,))
    elif history_lens is not None or prompt_lens is not None:
        raise ValueError("history_lens or prompt_lens without history")
    if draft is not None:
        _need(draft, "draft", i32, index, (B, R - 1))
    if repetition is not None:
        _need(repetition, "repetition", f32, index, (B,))
    if presence is not None:
        _need(presence, "presence", f32, index, (B,))
    if frequency is not None:
        _need(frequency, "frequency", f32, index, (B,))
    if bias_tokens is not None:
        if bias_tokens.dim() != 2 or bias_values is None:
            raise ValueError("bias_tokens must be [B, NB], with bias_values")
        NB = bias_tokens.shape[1]
        _need(bias_tokens, "bias_tokens", i32, index, (B, NB))
        _need(bias_values, "bias_values", f32, index, (B, NB))
    elif bias_values is not None:
        raise ValueError("bias_values without bias_tokens")
    if mask is not None:
        _need(mask, "mask", i32, index, (B, R, (V + 31) // 32))
    if temperature is not None:
        _need(temperature, "temperature", f32, index, (B,))
    if out is None:
        out = _new((B, R, V), f32, logits.device, stream)
    else:
        _need(out, "out", f32, index, (B, R, V))
    a = PaLogitsArgs(logits.data_ptr(), code, B, R, NB, V, sb if B > 1 else 0, sr if R > 1 else 0, _ptr(history), S,
                     _ptr(history_lens), _ptr(prompt_lens), _ptr(draft), _ptr(repetition), _ptr(presence),
                     _ptr(frequency), _ptr(bias_tokens), _ptr(bias_values), _ptr(mask), _ptr(temperature),
                     out.data_ptr())
    handle, call = _stream_on(stream, logits.device), getattr(_serving_lib(), name)
    if index == torch.cuda.current_device():
        _check(call(a, handle), name)
    else:
        with torch.cuda.device(index):
            _check(call(a, handle), name)
    return out


def adjust_logits(logits: torch.Tensor, history: Optional[torch.Tensor] = None,
                  history_lens: Optional[torch.Tensor] = None, prompt_lens: Optional[torch.Tensor] = None,
                  draft: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                  bias_tokens: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """pa_adjust_logits: penalties, biases and grammar masks on logits [B, R, V] (rows of any stride) -> fp32
    [B, R, V]. history int32 [B, S] (prompt tokens, then outputs), draft int32 [B, R - 1], repetition /
    presence / frequency fp32 [B], bias_tokens / bias_values [B, NB], mask int32 [B, R, ceil(V / 32)]."""
    return _logits_call("pa_adjust_logits", logits, None, history, history_lens, prompt_lens, draft, repetition,
                        presence, frequency, bias_tokens, bias_values, mask, out, stream)


def token_probs(logits: torch.Tensor, temperature: torch.Tensor, history: Optional[torch.Tensor] = None,
                history_lens: Optional[torch.Tensor] = None, prompt_lens: Optional[torch.Tensor] = None,
                draft: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                bias_tokens: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """pa_token_probs: the token distributions of adjusted logits (arguments as adjust_logits; temperature fp32
    [B], 0 = greedy) -> fp32 [B, R, V], the p of spec_verify."""
    if temperature is None:
        raise ValueError("temperature is needed")
    return _logits_call("pa_token_probs", logits, temperature, history, history_lens, prompt_lens, draft, repetition,
                        presence, frequency, bias_tokens, bias_values, mask, out, stream)
