"""Python binding of libll_swa.so (the B200 sink-window attention library).

Argument marshalling only: torch tensors supply device memory and the CUDA
stream; every step of the computation runs in the library's CUDA kernels.
The shared library must have been built (``python -m
sink_window_attention_b200.build`` or ``__graft_entry__.build()``); importing
this package without it raises, there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libll_swa.so")

LL_OK, LL_ERR_INVALID_ARG, LL_ERR_UNSUPPORTED, LL_ERR_CUDA, LL_ERR_TIMEOUT = range(5)
LL_F32, LL_BF16, LL_FP8_E4M3 = 0, 1, 2
MAX_HEADS = 64
LL_ROPE_INTERLEAVED, LL_ROPE_HALF = 0, 1
MAX_TOKEN_HEADS, MAX_TOKEN_PAIRS = 128, 64
ABI_VERSION = 2

EXPORTED = (
    "ll_abi_version", "ll_last_error", "ll_slot_of_frame", "ll_device_error", "ll_rope_apply",
    "ll_kvcache_append", "ll_sink_window_attention_workspace_bytes", "ll_sink_window_attention",
    "ll_kv_recache_workspace_bytes", "ll_kv_recache", "ll_sink_window_attention_noalloc",
    "ll_append_and_attend_workspace_bytes", "ll_append_and_attend", "ll_phase_coherence",
    "ll_selftest_bounded_waits", "ll_sink_window_attention_fp8_mma_workspace_bytes",
    "ll_sink_window_attention_fp8_mma",
    "ll_token_rope_init", "ll_token_rope_apply", "ll_paged_append", "ll_paged_attention_workspace_bytes",
    "ll_paged_attention",
)
NOALLOC_SCRATCH_BYTES = 48 * 1024 * 1024


class LLError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"ll status {status}: {message}")
        self.status = status


class RopeDescC(ctypes.Structure):
    _fields_ = [("pairs_t", ctypes.c_int), ("pairs_h", ctypes.c_int), ("pairs_w", ctypes.c_int),
                ("theta0", ctypes.c_double), ("sigma_t", ctypes.c_double),
                ("eps_h", ctypes.POINTER(ctypes.c_float)), ("grid_h", ctypes.c_int), ("grid_w", ctypes.c_int),
                ("t_offset", ctypes.c_longlong), ("t_scale", ctypes.c_double)]


class KVCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("tokens_per_frame", ctypes.c_int), ("n_sink", ctypes.c_int),
                ("n_local", ctypes.c_int)]


class TokenRopeDescC(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("layout", ctypes.c_int), ("amplitude", ctypes.c_float),
                ("reserved", ctypes.c_int), ("turns", ctypes.c_uint64 * MAX_TOKEN_PAIRS)]


class PagedCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("H", ctypes.c_int), ("D", ctypes.c_int)]


class TokenBatchC(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("B", ctypes.c_int), ("max_pages", ctypes.c_int), ("total_q", ctypes.c_int), ("max_q", ctypes.c_int),
                ("max_kv", ctypes.c_int)]


class ScoreDescC(ctypes.Structure):
    _fields_ = [("softmax_scale", ctypes.c_float), ("soft_cap", ctypes.c_float), ("window", ctypes.c_int),
                ("n_sink", ctypes.c_int), ("prefix_len", ctypes.c_void_p), ("slopes", ctypes.POINTER(ctypes.c_float))]


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with sink_window_attention_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, ll_, f, d, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_double, ctypes.c_size_t
        rp, cp = ctypes.POINTER(RopeDescC), ctypes.POINTER(KVCacheC)
        L.ll_abi_version.restype = i
        L.ll_last_error.restype = ctypes.c_char_p
        L.ll_slot_of_frame.argtypes = [ll_, i, i, ctypes.POINTER(i)]
        L.ll_device_error.argtypes = [ctypes.POINTER(i), vp]
        L.ll_rope_apply.argtypes = [vp, i, i, i, i, i, ll_, rp, vp]
        L.ll_kvcache_append.argtypes = [cp, vp, vp, i, ll_, i, rp, ctypes.POINTER(i), vp]
        L.ll_sink_window_attention_workspace_bytes.argtypes = [cp, i]
        L.ll_sink_window_attention_workspace_bytes.restype = sz
        L.ll_sink_window_attention.argtypes = [vp, i, cp, ll_, i, rp, f, vp, vp, vp, sz, vp]
        L.ll_sink_window_attention_noalloc.argtypes = [vp, i, cp, ll_, i, rp, f, vp, vp, vp]
        L.ll_sink_window_attention_fp8_mma_workspace_bytes.argtypes = [cp, i]
        L.ll_sink_window_attention_fp8_mma_workspace_bytes.restype = sz
        L.ll_sink_window_attention_fp8_mma.argtypes = [vp, i, cp, ll_, i, rp, f, vp, vp, vp, sz, vp]
        L.ll_kv_recache_workspace_bytes.argtypes = [cp, i, i]
        L.ll_kv_recache_workspace_bytes.restype = sz
        L.ll_kv_recache.argtypes = [cp, vp, i, vp, vp, vp, f, ctypes.POINTER(ll_), i, rp, vp, sz, vp]
        L.ll_append_and_attend_workspace_bytes.argtypes = [cp, i]
        L.ll_append_and_attend_workspace_bytes.restype = sz
        L.ll_append_and_attend.argtypes = [cp, vp, vp, vp, i, ll_, i, rp, f, vp, vp, vp, sz, vp]
        L.ll_phase_coherence.argtypes = [rp, i, ll_, i, vp, vp]
        L.ll_selftest_bounded_waits.argtypes = [vp]
        tr, pc, tb = (ctypes.POINTER(c) for c in (TokenRopeDescC, PagedCacheC, TokenBatchC))
        L.ll_token_rope_init.argtypes = [tr, i, i, d, d, d, d, d, d]
        L.ll_token_rope_apply.argtypes = [vp, ll_, vp, ll_, i, vp, i, i, i, tr, i, vp]
        L.ll_paged_append.argtypes = [pc, tb, vp, ll_, vp, ll_, i, tr, vp]
        L.ll_paged_attention_workspace_bytes.argtypes = [pc, tb, i]
        L.ll_paged_attention_workspace_bytes.restype = sz
        L.ll_paged_attention.argtypes = [vp, ll_, i, i, pc, tb, tr, ctypes.POINTER(ScoreDescC), vp, vp, vp, sz, vp]
        for name in EXPORTED[2:]:
            if not name.endswith("_workspace_bytes"):
                getattr(L, name).restype = i
        _lib = L
    return _lib


def last_error() -> str:
    return lib().ll_last_error().decode()


def _check(status: int) -> None:
    if status != LL_OK:
        raise LLError(status, last_error())


def _stream(stream=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return LL_F32
    if t == torch.bfloat16:
        return LL_BF16
    raise ValueError(f"unsupported tensor dtype {t}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Device address of a contiguous CUDA tensor on the current device (the
    library's kernels dereference it there)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"tensors must be CUDA tensors, got one on {t.device}")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors must be on the current CUDA device (cuda:{torch.cuda.current_device()}), "
                         f"got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _expect(t: Optional[torch.Tensor], shape, dtype: torch.dtype, what: str) -> None:
    """Shape and dtype of a buffer the kernels read or write in full."""
    if t is not None and (tuple(t.shape) != tuple(shape) or t.dtype != dtype):
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _cache_c(cache: "KVCache") -> "KVCacheC":
    """The cache descriptor for a launch: its tensors checked like any other."""
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        _ptr(t)
    return cache.to_c()


@dataclass
class Rope:
    """3D RoPE with the LoL per-head jittered temporal base (mirrors ll_rope_desc)."""
    pairs: Sequence[int]
    grid_h: int
    grid_w: int
    theta0: float = 10000.0
    sigma_t: float = 0.0
    eps: Optional[Sequence[float]] = None
    t_offset: int = 0
    t_scale: float = 1.0   # position interpolation of the temporal axis (1: plain RoPE)

    def to_c(self) -> RopeDescC:
        r = RopeDescC()
        r.pairs_t, r.pairs_h, r.pairs_w = (int(x) for x in self.pairs)
        r.theta0 = float(self.theta0)
        r.sigma_t = float(self.sigma_t)
        if self.eps is not None:
            arr = (ctypes.c_float * len(self.eps))(*[float(e) for e in self.eps])
            r._eps_keepalive = arr  # noqa: keep the host array alive with the struct
            r.eps_h = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
        r.grid_h, r.grid_w, r.t_offset = int(self.grid_h), int(self.grid_w), int(self.t_offset)
        r.t_scale = float(self.t_scale)
        return r


def _rope_ref(rope: Optional[Rope]):
    return ctypes.byref(rope.to_c()) if rope is not None else None


class KVCache:
    """One layer's sink + ring KV cache in device memory (mirrors ll_kvcache)."""

    def __init__(self, B: int, H: int, D: int, tokens_per_frame: int, dtype: str = "bf16",
                 n_sink: int = 3, n_local: int = 9, device: str = "cuda"):
        self.B, self.H, self.D, self.N = B, H, D, tokens_per_frame
        self.n_sink, self.n_local = n_sink, n_local
        self.S = n_sink + n_local
        self.dtype = dtype
        shape = (B, self.S * tokens_per_frame, H, D)
        if dtype == "fp8":
            self.k = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.v = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.k_scale = torch.ones(shape[:3], dtype=torch.float32, device=device)
            self.v_scale = torch.ones(shape[:3], dtype=torch.float32, device=device)
            self.code = LL_FP8_E4M3
        else:
            tdt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
            self.k = torch.zeros(shape, dtype=tdt, device=device)
            self.v = torch.zeros(shape, dtype=tdt, device=device)
            self.k_scale = self.v_scale = None
            self.code = _dtype_code(tdt)

    def to_c(self) -> KVCacheC:
        c = KVCacheC()
        c.k, c.v = self.k.data_ptr(), self.v.data_ptr()
        c.k_scale = self.k_scale.data_ptr() if self.k_scale is not None else None
        c.v_scale = self.v_scale.data_ptr() if self.v_scale is not None else None
        c.dtype, c.B, c.H, c.D = self.code, self.B, self.H, self.D
        c.tokens_per_frame, c.n_sink, c.n_local = self.N, self.n_sink, self.n_local
        return c


def abi_version() -> int:
    return lib().ll_abi_version()


def slot_of_frame(frame: int, n_sink: int = 3, n_local: int = 9) -> int:
    s = ctypes.c_int(-1)
    _check(lib().ll_slot_of_frame(frame, n_sink, n_local, ctypes.byref(s)))
    return s.value


def device_error(stream=None) -> int:
    """Synchronise and read (then clear) the library's device error word."""
    code = ctypes.c_int(0)
    st = lib().ll_device_error(ctypes.byref(code), _stream(stream))
    if st not in (LL_OK, LL_ERR_TIMEOUT):
        _check(st)
    return code.value


def rope_apply(x: torch.Tensor, first_frame: int, rope: Rope, stream=None) -> torch.Tensor:
    """In-place 3D RoPE of x [B, F*N, H, D]."""
    if x.dim() != 4:
        raise ValueError(f"x must be [B, F*N, H, D], got shape {tuple(x.shape)}")
    B, T, H, D = x.shape
    N = rope.grid_h * rope.grid_w
    if T % N != 0:
        raise ValueError(f"x holds {T} tokens, not a whole number of {N}-token frames")
    _check(lib().ll_rope_apply(_ptr(x), _dtype_code(x.dtype), B, T // N, H, D, first_frame, _rope_ref(rope),
                               _stream(stream)))
    return x


def _check_shape(cache: "KVCache", t: torch.Tensor, what: str) -> int:
    """[B, F*N, H, D] on the cache's batch, heads and head dim; returns F."""
    if t.dim() != 4 or t.shape[0] != cache.B or t.shape[2] != cache.H or t.shape[3] != cache.D or \
            t.shape[1] % cache.N != 0 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [B={cache.B}, F*{cache.N}, {cache.H}, {cache.D}] tensor, "
                         f"got {tuple(t.shape)}")
    return t.shape[1] // cache.N


def kvcache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, first_frame: int,
                   rope: Optional[Rope], stream=None):
    """Write frames first_frame.. of k, v [B, F*N, H, D] into their slots; returns the slots."""
    F = _check_shape(cache, k, "k")
    if _check_shape(cache, v, "v") != F:
        raise ValueError("k and v must cover the same frames")
    if v.dtype != k.dtype:
        raise ValueError("k and v must have one dtype")
    slots = (ctypes.c_int * F)()
    _check(lib().ll_kvcache_append(ctypes.byref(_cache_c(cache)), _ptr(k), _ptr(v), _dtype_code(k.dtype), first_frame,
                                   F, _rope_ref(rope), slots, _stream(stream)))
    return list(slots)


def attention_workspace_bytes(cache: KVCache, n_query_frames: int) -> int:
    return int(lib().ll_sink_window_attention_workspace_bytes(ctypes.byref(cache.to_c()), n_query_frames))


_workspaces = {}


def workspace_for(nbytes: int, device) -> torch.Tensor:
    """A device scratch buffer of at least nbytes, cached per device. Calls that
    share it must be ordered (one stream); pass your own workspace to run
    attention concurrently on several streams."""
    key = torch.device(device)
    t = _workspaces.get(key)
    if t is None or t.numel() < nbytes:
        t = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=key)
        _workspaces[key] = t
    return t


def sink_window_attention(q: torch.Tensor, cache: KVCache, first_frame: int, rope: Optional[Rope],
                          softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Attention of query frames first_frame.. (q [B, F*N, H, D]) over the cache."""
    F = _check_shape(cache, q, "q")
    if out is None:
        out = torch.empty_like(q)
    _expect(out, q.shape, q.dtype, "out")
    _expect(lse, (cache.B, cache.H, q.shape[1]), torch.float32, "lse")
    if workspace is None:
        workspace = workspace_for(attention_workspace_bytes(cache, F), q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().ll_sink_window_attention(_ptr(q), _dtype_code(q.dtype), ctypes.byref(_cache_c(cache)), first_frame, F,
                                          _rope_ref(rope), float(softmax_scale), _ptr(out), _ptr(lse),
                                          _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def attention_fp8_mma_workspace_bytes(cache: KVCache, n_query_frames: int) -> int:
    return int(lib().ll_sink_window_attention_fp8_mma_workspace_bytes(ctypes.byref(cache.to_c()), n_query_frames))


def sink_window_attention_fp8_mma(q: torch.Tensor, cache: KVCache, first_frame: int, rope: Optional[Rope],
                                  softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                  stream=None) -> torch.Tensor:
    """Attention over an E4M3 cache on the FP8 tensor cores (ll_sink_window_attention_fp8_mma)."""
    F = _check_shape(cache, q, "q")
    if out is None:
        out = torch.empty_like(q)
    _expect(out, q.shape, q.dtype, "out")
    _expect(lse, (cache.B, cache.H, q.shape[1]), torch.float32, "lse")
    if workspace is None:
        workspace = workspace_for(max(attention_fp8_mma_workspace_bytes(cache, F), 256), q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().ll_sink_window_attention_fp8_mma(_ptr(q), _dtype_code(q.dtype), ctypes.byref(_cache_c(cache)),
                                                  first_frame, F, _rope_ref(rope), float(softmax_scale), _ptr(out),
                                                  _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def append_and_attend_workspace_bytes(cache: KVCache, n_frames: int) -> int:
    return int(lib().ll_append_and_attend_workspace_bytes(ctypes.byref(cache.to_c()), n_frames))


def append_and_attend(cache: KVCache, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, first_frame: int,
                      rope: Optional[Rope], softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """ll_append_and_attend: append frames first_frame.. (k, v [B, F*N, H, D])
    and attend with their queries q (one kernel for BF16 / F32 caches; for an
    E4M3 cache the append with the bf16 staging copy, then attention)."""
    F = _check_shape(cache, q, "q")
    if _check_shape(cache, k, "k") != F or _check_shape(cache, v, "v") != F:
        raise ValueError("k, v and q must cover the same frames")
    if not (k.dtype == v.dtype == q.dtype):
        raise ValueError("k, v and q must have one dtype")
    if out is None:
        out = torch.empty_like(q)
    _expect(out, q.shape, q.dtype, "out")
    _expect(lse, (cache.B, cache.H, q.shape[1]), torch.float32, "lse")
    if workspace is None:
        workspace = workspace_for(append_and_attend_workspace_bytes(cache, F), q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().ll_append_and_attend(ctypes.byref(_cache_c(cache)), _ptr(k), _ptr(v), _ptr(q), _dtype_code(q.dtype),
                                      first_frame, F, _rope_ref(rope), float(softmax_scale), _ptr(out), _ptr(lse),
                                      _ptr(workspace), ws_bytes, _stream(stream)))
    return out


def sink_window_attention_noalloc(q: torch.Tensor, cache: KVCache, first_frame: int, rope: Optional[Rope],
                                  softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                                  lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ll_sink_window_attention_noalloc: the same attention with the library's
    static scratch array instead of a caller workspace (allocates nothing)."""
    F = _check_shape(cache, q, "q")
    if out is None:
        out = torch.empty_like(q)
    _expect(out, q.shape, q.dtype, "out")
    _expect(lse, (cache.B, cache.H, q.shape[1]), torch.float32, "lse")
    _check(lib().ll_sink_window_attention_noalloc(_ptr(q), _dtype_code(q.dtype), ctypes.byref(_cache_c(cache)),
                                                  first_frame, F, _rope_ref(rope), float(softmax_scale), _ptr(out),
                                                  _ptr(lse), _stream(stream)))
    return out


def recache_workspace_bytes(cache: KVCache, d_model: int, n_slots: int) -> int:
    return int(lib().ll_kv_recache_workspace_bytes(ctypes.byref(cache.to_c()), d_model, n_slots))


def kv_recache(cache: KVCache, x: torch.Tensor, wk: torch.Tensor, wv: torch.Tensor, gamma: torch.Tensor,
               rms_eps: float, slot_frames: Sequence[int], rope: Rope,
               workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Recompute K/V of slots 0..len(slot_frames)-1 from hidden states x [B, n*N, d_model]."""
    n = len(slot_frames)
    if x.dim() != 3:
        raise ValueError(f"x must be [B, n_slots*N, d_model], got shape {tuple(x.shape)}")
    dm, dout = x.shape[-1], cache.H * cache.D
    _expect(x, (cache.B, n * cache.N, dm), torch.bfloat16, "x")
    _expect(wk, (dm, dout), torch.bfloat16, "wk")
    _expect(wv, (dm, dout), torch.bfloat16, "wv")
    _expect(gamma, (dout,), torch.float32, "gamma")
    frames = (ctypes.c_longlong * n)(*[int(f) for f in slot_frames])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().ll_kv_recache(ctypes.byref(_cache_c(cache)), _ptr(x), dm, _ptr(wk), _ptr(wv), _ptr(gamma),
                               float(rms_eps), frames, n, _rope_ref(rope), _ptr(workspace), ws_bytes,
                               _stream(stream)))


def phase_coherence(rope: Rope, H: int, delta0: int, n_delta: int, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """C_h(D) of the temporal RoPE band for D = delta0 .. delta0 + n_delta - 1
    (ll_phase_coherence): float32 [H, n_delta, 2] (real, imaginary) on the
    current CUDA device."""
    if out is None:
        out = torch.empty((H, n_delta, 2), dtype=torch.float32, device="cuda")
    _expect(out, (H, n_delta, 2), torch.float32, "out")
    _check(lib().ll_phase_coherence(ctypes.byref(rope.to_c()), H, int(delta0), int(n_delta), _ptr(out),
                                    _stream(stream)))
    return out


def selftest_bounded_waits(stream=None) -> int:
    """Launch the bounded-wait self-test (ll_selftest_bounded_waits) and return
    the device error code it leaves (read and cleared by ll_device_error)."""
    _check(lib().ll_selftest_bounded_waits(_stream(stream)))
    return device_error(stream)


# ---------------------------------------------------------------------------
# Streams of single tokens: rotary positions, a paged pool of keys and values,
# and attention of a ragged batch of sequences over it.
# ---------------------------------------------------------------------------
# These calls are made once per layer and token, so the marshalling is kept short:
# one look at the current device, descriptors kept until something they were made of changes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device: int, stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(device)


def _on(t: torch.Tensor, device: int) -> int:
    """_ptr on a device already looked up."""
    if t.get_device() != device or not t.is_contiguous():
        return _ptr(t)
    return t.data_ptr()


def _fits(t: Optional[torch.Tensor], shape, dtype: torch.dtype, what: str) -> None:
    if t is None:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)}, got None")
    _expect(t, shape, dtype, what)


class _Described:
    """Keeps the descriptor of its fields. Setting one drops it; what else can change is a
    tensor in place (its address, size or order), which each call looks at."""
    _kept = (None, None)  # what the descriptor's tensors were, and the descriptor, replaced together

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_kept", (None, None))

    def _keep(self, now, c):
        object.__setattr__(self, "_kept", (now, c))
        return c


class TokenRope:
    """Rotary embedding of token positions (mirrors ll_token_rope_desc; ll_token_rope_init fills it).

    The first rot_dim elements of a head are turned; layout "half" pairs element
    i with i + rot_dim / 2, "interleaved" 2i with 2i + 1. scale < 1 interpolates
    positions, by parts where original_len is given (beta_fast, beta_slow: turns
    within original_len from which on a pair keeps its frequency, and up to
    which it is interpolated in full); rotated elements are multiplied by
    amplitude.
    """

    def __init__(self, rot_dim: int, theta0: float = 10000.0, layout: str = "half", scale: float = 1.0,
                 original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, amplitude: float = 1.0):
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
        self.rot_dim, self.layout = rot_dim, layout
        self._c = TokenRopeDescC()
        _check(lib().ll_token_rope_init(self._c, rot_dim, LL_ROPE_HALF if layout == "half" else LL_ROPE_INTERLEAVED,
                                        theta0, scale, original_len, beta_fast, beta_slow, amplitude))

    def to_c(self) -> TokenRopeDescC:
        return self._c


_POOL_TYPES = {"bf16": (LL_BF16, torch.bfloat16), "fp8": (LL_FP8_E4M3, torch.uint8)}


class PagedKVCache(_Described):
    """One layer's pool of pages in device memory (mirrors ll_paged_cache):
    k, v [n_pages, H, page_size, D]; an "fp8" pool has k_scale, v_scale [n_pages, H]."""

    def __init__(self, n_pages: int, page_size: int, H: int, D: int, dtype: str = "bf16", device: str = "cuda"):
        self.n_pages, self.page_size, self.H, self.D, self.dtype = n_pages, page_size, H, D, dtype
        code, tdt = _POOL_TYPES[dtype]
        shape = (n_pages, H, page_size, D)
        self.k = torch.zeros(shape, dtype=tdt, device=device)
        self.v = torch.zeros(shape, dtype=tdt, device=device)
        self.k_scale = self.v_scale = None
        if dtype == "fp8":
            self.k_scale = torch.zeros(shape[:2], dtype=torch.float32, device=device)
            self.v_scale = torch.zeros(shape[:2], dtype=torch.float32, device=device)
        self.code = code

    def _now(self, device):
        k, v, ks, vs = self.k, self.v, self.k_scale, self.v_scale
        if ks is None:
            return (device, k.data_ptr(), k.numel(), k.is_contiguous(), v.data_ptr(), v.numel(), v.is_contiguous())
        return (device, k.data_ptr(), k.numel(), k.is_contiguous(), v.data_ptr(), v.numel(), v.is_contiguous(),
                ks.data_ptr(), ks.numel(), ks.is_contiguous(), vs.data_ptr(), vs.numel(), vs.is_contiguous())

    def to_c(self, device: Optional[int] = None) -> PagedCacheC:
        """The descriptor, of tensors that fit the pool's sizes and type; with a device,
        they are checked to be there."""
        kept, c = self._kept
        if c is not None and kept == self._now(kept[0] if device is None else device):
            return c
        code, tdt = _POOL_TYPES[self.dtype]
        shape = (self.n_pages, self.H, self.page_size, self.D)
        for t, what in ((self.k, "k"), (self.v, "v")):  # codes may be named by their own type too
            codes = self.dtype == "fp8" and t is not None and t.dtype == torch.float8_e4m3fn
            _fits(t, shape, torch.float8_e4m3fn if codes else tdt, what)
        for t, what in ((self.k_scale, "k_scale"), (self.v_scale, "v_scale")):
            if self.dtype == "fp8":
                _fits(t, shape[:2], torch.float32, what)
            elif t is not None:
                raise ValueError(f"{what} must be None in a {self.dtype} pool")
        at = [t if t is None else (t.data_ptr() if device is None else _on(t, device))
              for t in (self.k, self.v, self.k_scale, self.v_scale)]
        return self._keep(self._now(device), PagedCacheC(*at, code, self.n_pages, self.page_size, self.H,
                                                        self.D))


class TokenBatch(_Described):
    """Which tokens of which sequences a call works on (mirrors ll_token_batch).

    q_start [B+1], kv_len [B], page_table [B, max_pages]: contiguous int32 CUDA
    tensors, read on the device when a call runs, so their contents may change
    between calls (and between replays of a captured graph) as long as max_q and
    max_kv still bound them.
    """

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, max_q: int, max_kv: int):
        if page_table.dim() != 2:
            raise ValueError(f"page_table must be [B, max_pages], got shape {tuple(page_table.shape)}")
        B, max_pages = page_table.shape
        self.q_start, self.kv_len, self.page_table = q_start, kv_len, page_table
        self.B, self.max_pages, self.max_q, self.max_kv = B, max_pages, int(max_q), int(max_kv)
        self._check()

    def _check(self) -> None:
        _fits(self.page_table, (self.B, self.max_pages), torch.int32, "page_table")
        _fits(self.q_start, (self.B + 1,), torch.int32, "q_start")
        _fits(self.kv_len, (self.B,), torch.int32, "kv_len")

    def _now(self, total_q, device):
        q, n, p = self.q_start, self.kv_len, self.page_table
        return (total_q, device, q.data_ptr(), q.numel(), q.is_contiguous(), n.data_ptr(), n.numel(),
                n.is_contiguous(), p.data_ptr(), p.numel(), p.is_contiguous())

    def to_c(self, total_q: int, device: int) -> TokenBatchC:
        kept, c = self._kept
        if c is not None and kept == self._now(total_q, device):
            return c
        self._check()
        # a new structure, not a changed one: another thread may be in a call with the old
        return self._keep(self._now(total_q, device),
                          TokenBatchC(_on(self.q_start, device), _on(self.kv_len, device), _on(self.page_table, device),
                                      self.B, self.max_pages, total_q, self.max_q, self.max_kv))


class Scores:
    """What happens to scores and which keys are seen (mirrors ll_score_desc): see paged_attention.

    prefix_len: int32 CUDA tensor [B]; slopes: one float per query head.
    """

    def __init__(self, softmax_scale: float = 0.0, window: int = 0, n_sink: int = 0,
                 prefix_len: Optional[torch.Tensor] = None, soft_cap: float = 0.0,
                 slopes: Optional[Sequence[float]] = None):
        self.softmax_scale, self.window, self.n_sink, self.soft_cap = softmax_scale, window, n_sink, soft_cap
        self.prefix_len = prefix_len
        self.slopes = None if slopes is None else (ctypes.c_float * len(slopes))(*[float(x) for x in slopes])

    def to_c(self, B: int, Hq: int) -> ScoreDescC:
        _expect(self.prefix_len, (B,), torch.int32, "prefix_len")
        if self.slopes is not None and len(self.slopes) != Hq:
            raise ValueError(f"slopes must have one value for each of the {Hq} query heads, got {len(self.slopes)}")
        c = ScoreDescC(self.softmax_scale, self.soft_cap, self.window, self.n_sink, _ptr(self.prefix_len))
        if self.slopes is not None:
            c.slopes = ctypes.cast(self.slopes, ctypes.POINTER(ctypes.c_float))
        return c


def _rows(t: torch.Tensor, what: str, device: int, H: Optional[int] = None, D: Optional[int] = None):
    """(address, row stride in elements) of a CUDA tensor [T, H, D] whose heads lie
    together; rows may be further apart (a slice of a fused projection)."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [rows, {H or 'heads'}, {D or 'D'}], got shape {tuple(t.shape)}")
    T, h, d = t.shape
    if (H is not None and h != H) or (D is not None and d != D):
        raise ValueError(f"{what} must be [rows, {H or 'heads'}, {D or 'D'}], got shape {tuple(t.shape)}")
    sr, sh, sd = t.stride()
    if T <= 1:
        sr = h * d
    if T > 0 and ((sd != 1 and d > 1) or (sh != d and h > 1)):
        raise ValueError(f"the heads of a row of {what} must be contiguous, got strides {t.stride()}")
    if t.get_device() != device:
        if not t.is_cuda:
            raise ValueError(f"tensors must be CUDA tensors, got one on {t.device}")
        raise ValueError(f"tensors must be on the current CUDA device (cuda:{device}), got one on {t.device}")
    return t.data_ptr(), sr


def _device(t: torch.Tensor) -> int:
    """The current CUDA device, where the call's tensors have to be (none for a host
    tensor, which _rows refuses)."""
    return torch.cuda.current_device() if t.is_cuda else -2


def _empty_rows(like: torch.Tensor, stream) -> torch.Tensor:
    """A contiguous tensor of `like`'s shape that belongs to the stream the kernels run on."""
    if stream is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    with torch.cuda.stream(stream):
        return torch.empty_like(like, memory_format=torch.contiguous_format)


def _workspace(nbytes: int, like: torch.Tensor, stream) -> torch.Tensor:
    with torch.cuda.stream(stream):  # None: the current stream
        return like.new_empty((nbytes,), dtype=torch.uint8)


def _as_rows(g: torch.Tensor) -> torch.Tensor:
    """g, copied where it is no token tensor (an expanded, permuted or unaligned gradient)."""
    T, H, D = g.shape
    sr, sh, sd = g.stride()
    if sd == 1 and sh == D and sr >= H * D and sr % 8 == 0 and g.data_ptr() % 16 == 0:
        return g
    return g.clone(memory_format=torch.contiguous_format)


class _TokenRotation(torch.autograd.Function):
    """The rotation is linear: its gradient is the transposed one's."""

    @staticmethod
    def forward(ctx, x, positions, rope, transpose):
        ctx.save_for_backward(positions)
        ctx.rope, ctx.transpose = rope, transpose
        return token_rope_apply(x.detach(), positions, rope, transpose)

    @staticmethod
    def backward(ctx, g):
        positions, = ctx.saved_tensors
        return token_rope_apply(_as_rows(g), positions, ctx.rope, not ctx.transpose), None, None, None


def token_rope_apply(x: torch.Tensor, positions: torch.Tensor, rope: TokenRope, transpose: bool = False,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotate x [T, H, D] (bf16 or f32) at its tokens' positions (int32 [T]);
    transpose=True applies the transposed rotation: the gradient, which autograd
    takes by itself where x requires grad. out may be x (not where autograd
    tracks either)."""
    if (x.requires_grad or (out is not None and out.requires_grad)) and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where x or out requires grad")
        with torch.cuda.stream(stream):  # None: the current stream
            return _TokenRotation.apply(x, positions, rope, bool(transpose))
    dev = _device(x)
    xp, xs = _rows(x, "x", dev)
    T, H, D = x.shape
    if positions.dtype != torch.int32 or positions.shape != (T,):
        _expect(positions, (T,), torch.int32, "positions")
    if out is None:
        out = _empty_rows(x, stream)
        op, os_ = out.data_ptr(), H * D
    else:
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError(f"out must be a {x.dtype} tensor of shape {tuple(x.shape)}, "
                             f"got {out.dtype} {tuple(out.shape)}")
        op, os_ = _rows(out, "out", dev)
    if T == 0:
        return out
    _check(lib().ll_token_rope_apply(xp, xs, op, os_, _dtype_code(x.dtype), _on(positions, dev), T, H, D, rope._c,
                                     1 if transpose else 0, _stream_of(dev, stream)))
    return out


def _no_gradients(call: str) -> None:
    if torch.is_grad_enabled():
        raise ValueError(f"{call} has no gradients: call it under torch.no_grad(), or detach its inputs")


def paged_append(cache: PagedKVCache, batch: TokenBatch, k: torch.Tensor, v: torch.Tensor,
                 rope: Optional[TokenRope] = None, stream=None) -> None:
    """Write the batch's new tokens, k and v [total_q, H, D] bf16, into their
    pages, K rotated at its positions (ll_paged_append). Rows may be strided. There are
    no gradients: inputs that require them are refused where grad is enabled."""
    if k.requires_grad or v.requires_grad:
        _no_gradients("paged_append")
    dev = _device(k)
    kp, ks = _rows(k, "k", dev, cache.H, cache.D)
    vp, vs = _rows(v, "v", dev, cache.H, cache.D)
    T = k.shape[0]
    if v.shape[0] != T or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    if T == 0:
        return
    _check(lib().ll_paged_append(cache.to_c(dev), batch.to_c(T, dev), kp, ks, vp, vs, _dtype_code(k.dtype),
                                 None if rope is None else rope._c, _stream_of(dev, stream)))


def paged_attention_workspace_bytes(cache: PagedKVCache, batch: TokenBatch, total_q: int, Hq: int) -> int:
    c = TokenBatchC(1 << 12, 1 << 12, 1 << 12, batch.B, batch.max_pages, total_q, batch.max_q, batch.max_kv)
    return int(lib().ll_paged_attention_workspace_bytes(cache.to_c(), c, Hq))


def paged_attention(q: torch.Tensor, cache: PagedKVCache, batch: TokenBatch, rope: Optional[TokenRope] = None,
                    scores: Optional[Scores] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Attention of the batch's rows q [total_q, Hq, D] (bf16, rows may be
    strided; rotated here when rope is given) over the pool, which already holds
    their keys and values (ll_paged_attention). Rows of no sequence are not
    written: they keep what `out` held. There are no gradients: inputs that require them
    are refused where grad is enabled."""
    if q.requires_grad or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad):
        _no_gradients("paged_attention")
    dev = _device(q)
    qp, qs = _rows(q, "q", dev, None, cache.D)
    T, Hq, D = q.shape
    if out is None:
        out = _empty_rows(q, stream)
        op = out.data_ptr()
    else:
        _expect(out, (T, Hq, D), q.dtype, "out")
        op = _on(out, dev)
    lp = None
    if lse is not None:
        _expect(lse, (T, Hq), torch.float32, "lse")
        lp = _on(lse, dev)
    if T == 0:
        return out
    L, pool, tokens = lib(), cache.to_c(dev), batch.to_c(T, dev)
    wp = None
    if workspace is None:
        ws_bytes = L.ll_paged_attention_workspace_bytes(pool, tokens, Hq)
        if ws_bytes:
            workspace = _workspace(ws_bytes, q, stream)
            wp = workspace.data_ptr()
    else:
        wp, ws_bytes = _on(workspace, dev), workspace.numel() * workspace.element_size()
    _check(L.ll_paged_attention(qp, qs, _dtype_code(q.dtype), Hq, pool, tokens, None if rope is None else rope._c,
                                None if scores is None else scores.to_c(batch.B, Hq), op, lp, wp, ws_bytes,
                                _stream_of(dev, stream)))
    return out
