"""Python binding of libhikv, the importance-aware budgeted KV-cache decode step.

Argument marshalling only: every function below takes torch CUDA tensors,
checks their dtype/shape/contiguity, and passes raw device pointers and the
current CUDA stream to the C ABI declared in ``include/hikv.h``.  All
arithmetic of the step runs in the library's CUDA kernels; there is no CPU
or PyTorch fallback, and importing this package fails loudly when
``libhikv.so`` has not been built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import array
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhikv.so")

HIKV_OK, HIKV_ERR_INVALID_ARG, HIKV_ERR_OUT_OF_MEMORY, HIKV_ERR_CAPACITY = 0, 1, 2, 3
HIKV_ERR_CUDA, HIKV_ERR_TIMEOUT, HIKV_ERR_STATE, HIKV_ERR_UNSUPPORTED = 4, 5, 6, 7
STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "OUT_OF_MEMORY", 3: "CAPACITY", 4: "CUDA",
                5: "TIMEOUT", 6: "STATE", 7: "UNSUPPORTED"}
HIKV_F32, HIKV_BF16 = 0, 1

# every entry point of include/hikv.h
ABI_FUNCTIONS = ("hikv_create_cache", "hikv_destroy_cache", "hikv_append", "hikv_score_window",
                 "hikv_decode_step", "hikv_evict", "hikv_gather_retained", "hikv_get_lengths",
                 "hikv_device_status", "hikv_last_error", "hikv_score_window_noalloc",
                 "hikv_decode_step_fused", "hikv_kernel_launches", "hikv_budgets_pyramid",
                 "hikv_budgets_duo", "hikv_selftest_timeout", "hikv_element_rows",
                 "hikv_last_decode_config", "hikv_score_band", "hikv_read_floor",
                 "hikv_read_slot", "hikv_append_packed", "hikv_attend_packed", "hikv_drop",
                 "hikv_device_view")


class HikvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"hikv {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class hikv_config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_sink", ctypes.c_int32), ("recent_window", ctypes.c_int32),
                ("budgets", ctypes.POINTER(ctypes.c_int32)), ("max_tokens", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("pool_pages", ctypes.c_int64),
                ("max_window_queries", ctypes.c_int32), ("scale", ctypes.c_float),
                ("pool_kernel", ctypes.c_int32), ("importance_mode", ctypes.c_int32),
                ("element_budget", ctypes.c_int32), ("band_scoring", ctypes.c_int32)]


class hikv_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class hikv_rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("positions", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class hikv_view(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("pool_pages", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32), ("units", ctypes.c_int32),
                ("importance", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("lengths", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build the CUDA library first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    sig = {
        "hikv_create_cache": ([ctypes.POINTER(hikv_config), ctypes.POINTER(P)], S),
        "hikv_destroy_cache": ([P], S),
        "hikv_append": ([P, I32, I32, I32, P, P, P], S),
        "hikv_score_window": ([P, I32, I32, I32, P, P], S),
        "hikv_score_band": ([P, I32, I32, I32, P, P], S),
        "hikv_decode_step": ([P, I32, I32, P, P, P], S),
        "hikv_evict": ([P, I32, I32, P], S),
        "hikv_gather_retained": ([P, I32, I32, I32, P, P, P, P, P, P], S),
        "hikv_get_lengths": ([P, I32, I32, P], S),
        "hikv_device_status": ([P], S),
        "hikv_last_error": ([], ctypes.c_char_p),
        "hikv_score_window_noalloc": ([I32] * 8 + [ctypes.c_float, P, P, P, P], S),
        "hikv_decode_step_fused": ([P, I32, I32, P, P, P, P, I32, P], S),
        "hikv_kernel_launches": ([P], ctypes.c_int64),
        "hikv_element_rows": ([P, ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
        "hikv_last_decode_config": ([P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
        "hikv_budgets_pyramid": ([I32, I32, I32, I32, I32, P], S),
        "hikv_budgets_duo": ([I32, I32, P, I32, I32, I32, P], S),
        "hikv_selftest_timeout": ([P, I32, P], S),
        "hikv_read_floor": ([P, I64, I32, P, P], S),
        "hikv_read_slot": ([P, I32, I32, P, P, P, P], S),
        "hikv_append_packed": ([P, I32] + [P] * 7, S),
        "hikv_attend_packed": ([P, I32] + [P] * 4, S),
        "hikv_drop": ([P, I32, I32, P, P], S),
        "hikv_device_view": ([P, ctypes.POINTER(hikv_view)], S),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def _check(status: int):
    if status != HIKV_OK:
        raise HikvError(status, _lib.hikv_last_error().decode())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _raw_stream_fn():
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", None)


_RAW_STREAM = None


def _stream_of(t, stream):
    """The stream handle for a call: the given one, else the current stream of
    t's device (read without building a Stream object when torch allows)."""
    global _RAW_STREAM
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _RAW_STREAM is None:
        _RAW_STREAM = _raw_stream_fn() or False
    if _RAW_STREAM:
        return _RAW_STREAM(t.device.index)
    return _stream(None).value


def _ptr_checked(t, name, dtype, shape):
    """One pass of the checks _dev makes, returning the device pointer as an int."""
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dev(t, name, dtype=None, shape=None):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return ctypes.c_void_p(t.data_ptr())


class Rope:
    """Rotation tables for Cache.append_packed: cos and sin [positions][r / 2]
    fp32 on the cache's device, row p for position p; pairs (i, i + r / 2), or
    (2i, 2i + 1) if interleaved.  Form the angles in 64 bits: an fp32
    position x frequency is off by up to 2^-24 of the angle, 0.008 rad at
    position 131072.  Keeps the tables alive."""

    def __init__(self, cos, sin, interleaved: bool = False):
        import torch
        _dev(cos, "cos", torch.float32)
        _dev(sin, "sin", torch.float32, cos.shape)
        if cos.dim() != 2:
            raise ValueError(f"cos has shape {tuple(cos.shape)}, expected [positions][rotated / 2]")
        if cos.device != sin.device:
            raise ValueError("cos and sin are on different devices")
        self.cos, self.sin, self.interleaved = cos, sin, bool(interleaved)
        self.device_index = cos.device.index
        self.c = hikv_rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(self.interleaved))
        self.ref = ctypes.byref(self.c)


class _DeviceArray:
    """Device memory of a cache as a CUDA array; keeps the cache alive."""

    def __init__(self, cache, ptr, shape, typestr):
        self.cache = cache
        self.__cuda_array_interface__ = {"data": (ptr, False), "shape": tuple(shape), "typestr": typestr,
                                         "strides": None, "version": 3}


@dataclass
class CacheConfig:
    num_layers: int
    batch: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    dtype: str                     # "f32" | "bf16"
    num_sink: int
    recent_window: int
    budgets: Sequence[int]         # [num_layers * num_kv_heads]
    max_tokens: int
    page_tokens: int = 64
    pool_pages: int = 0
    max_window_queries: int = 0
    scale: float = 0.0
    pool_kernel: int = 0           # SnapKV max-pool of the prompt scores (0/1: off)
    importance_mode: int = 0       # 0: H2O cumulative, 1: HiKV recent bank only
    element_budget: int = 0        # HiKV Stage II B2 (0 or head_dim: exact attention)
    band_scoring: int = 0          # 1: allow score_band (HiKV banded prefill scores)


def hikv_create_cache(cfg: CacheConfig) -> ctypes.c_void_p:
    b = np.ascontiguousarray(np.asarray(cfg.budgets, dtype=np.int32))
    c = hikv_config(cfg.num_layers, cfg.batch, cfg.num_q_heads, cfg.num_kv_heads, cfg.head_dim,
                    HIKV_BF16 if cfg.dtype == "bf16" else HIKV_F32, cfg.num_sink,
                    cfg.recent_window, b.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                    cfg.max_tokens, cfg.page_tokens, cfg.pool_pages, cfg.max_window_queries,
                    cfg.scale, cfg.pool_kernel, cfg.importance_mode, cfg.element_budget,
                    cfg.band_scoring)
    h = ctypes.c_void_p()
    _check(_lib.hikv_create_cache(ctypes.byref(c), ctypes.byref(h)))
    return h


def hikv_destroy_cache(h) -> None:
    _check(_lib.hikv_destroy_cache(h))


def hikv_append(h, layer0: int, k, v, stream=None) -> None:
    nl, ntok = k.shape[0], k.shape[3]
    _check(_lib.hikv_append(h, layer0, nl, ntok, _dev(k, "k"), _dev(v, "v", k.dtype, k.shape),
                            _stream(stream)))


def hikv_score_window(h, layer0: int, q, stream=None) -> None:
    _check(_lib.hikv_score_window(h, layer0, q.shape[0], q.shape[3], _dev(q, "q"), _stream(stream)))


def hikv_decode_step(h, layer0: int, q, out, stream=None) -> None:
    _check(_lib.hikv_decode_step(h, layer0, q.shape[0], _dev(q, "q"),
                                 _dev(out, "out", q.dtype, q.shape), _stream(stream)))


def hikv_decode_step_fused(h, layer0: int, k, v, q, out, evict: bool = True, stream=None) -> None:
    _check(_lib.hikv_decode_step_fused(h, layer0, q.shape[0], _dev(k, "k"), _dev(v, "v", k.dtype, k.shape),
                                       _dev(q, "q", k.dtype), _dev(out, "out", q.dtype, q.shape),
                                       1 if evict else 0, _stream(stream)))


def budgets_pyramid(num_layers: int, num_kv_heads: int, avg: int, min_budget: int,
                    floor_budget: int = 1) -> np.ndarray:
    """PyramidKV per-layer budgets, [num_layers * num_kv_heads] int32 (C ABI)."""
    out = np.empty(num_layers * num_kv_heads, dtype=np.int32)
    _check(_lib.hikv_budgets_pyramid(num_layers, num_kv_heads, avg, min_budget, floor_budget, out.ctypes.data))
    return out


def budgets_duo(retrieval, full_budget: int, num_sink: int, recent_window: int) -> np.ndarray:
    """DuoAttention budgets from a [num_layers][num_kv_heads] retrieval-head mask (C ABI)."""
    m = np.ascontiguousarray(np.asarray(retrieval, dtype=bool), dtype=np.uint8)
    if m.ndim != 2:
        raise ValueError("retrieval must be [num_layers][num_kv_heads]")
    out = np.empty(m.size, dtype=np.int32)
    _check(_lib.hikv_budgets_duo(m.shape[0], m.shape[1], m.ctypes.data, full_budget, num_sink, recent_window,
                                 out.ctypes.data))
    return out


def hikv_evict(h, layer0: int, nlayers: int, stream=None) -> None:
    _check(_lib.hikv_evict(h, layer0, nlayers, _stream(stream)))


def hikv_gather_retained(h, layer0: int, nlayers: int, cap: int, lengths, positions, importance,
                         k_out=None, v_out=None, stream=None) -> None:
    import torch
    _check(_lib.hikv_gather_retained(
        h, layer0, nlayers, cap, _dev(lengths, "lengths", torch.int32),
        _dev(positions, "positions", torch.int32), _dev(importance, "importance", torch.float32),
        _dev(k_out, "k_out"), _dev(v_out, "v_out"), _stream(stream)))


def hikv_get_lengths(h, layer0: int, nlayers: int, units_per_layer: int) -> np.ndarray:
    out = np.empty(nlayers * units_per_layer, dtype=np.int32)
    _check(_lib.hikv_get_lengths(h, layer0, nlayers, out.ctypes.data))
    return out


def hikv_device_status(h) -> None:
    _check(_lib.hikv_device_status(h))


def hikv_score_window_noalloc(k, q, importance, num_q_heads: int, scale: float = 0.0,
                              stream=None) -> None:
    """Stateless prompt importance on caller-owned buffers (no allocation).

    k: [nl][B][Hkv][ntok][d], q: [nl][B][Hq][nq][d], importance: [nl][B][Hkv][ntok] fp32.
    """
    import torch
    nl, b, hkv, ntok, d = k.shape
    nq = q.shape[3]
    dt = HIKV_BF16 if k.dtype == torch.bfloat16 else HIKV_F32
    _check(_lib.hikv_score_window_noalloc(
        nl, b, num_q_heads, hkv, d, dt, ntok, nq, scale, _dev(k, "k"),
        _dev(q, "q", k.dtype, (nl, b, num_q_heads, nq, d)),
        _dev(importance, "importance", torch.float32, (nl, b, hkv, ntok)), _stream(stream)))


def read_floor(buf, ctas_per_sm: int = 2, sink=None, stream=None) -> None:
    """Measurement aid: one plain streaming read of a CUDA tensor's bytes
    (hikv_read_floor); `sink` a 4-byte CUDA tensor (allocated if None)."""
    import torch
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device=buf.device)
    _check(_lib.hikv_read_floor(_dev(buf, "buf"), buf.numel() * buf.element_size(), ctas_per_sm,
                                _dev(sink, "sink"), _stream(stream)))


def hikv_last_error() -> str:
    return _lib.hikv_last_error().decode()


class Cache:
    """Owning wrapper: one hikv cache on the current CUDA device."""

    def __init__(self, cfg: CacheConfig):
        self.cfg = cfg
        self._step_shapes = {}
        self.units_per_layer = cfg.batch * cfg.num_kv_heads
        self.units = cfg.num_layers * self.units_per_layer
        self.h = hikv_create_cache(cfg)
        import torch
        self.device_index = torch.cuda.current_device()
        self._torch_dtype = self._dtype()
        self._row_args = [hikv_rows() for _ in range(4)]   # k, v, q, q_out / out of a packed call
        self._row_refs = [ctypes.byref(r) for r in self._row_args]

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            hikv_destroy_cache(self.h)
        self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # The C ABI takes raw pointers and cannot see buffer sizes: the binding
    # checks every tensor against the configuration before passing it on.
    def _dtype(self):
        import torch
        return torch.bfloat16 if self.cfg.dtype == "bf16" else torch.float32

    def _check_tensor(self, t, name, shape):
        if t.dtype != self._dtype():
            raise TypeError(f"{name} has dtype {t.dtype}, the cache holds {self._dtype()}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")

    def _layers(self, t, layer0):
        nl = t.shape[0] if t.dim() else 0
        if not (0 <= layer0 and nl >= 1 and layer0 + nl <= self.cfg.num_layers):
            raise ValueError(f"layers [{layer0}, {layer0 + nl}) outside [0, {self.cfg.num_layers})")
        return nl

    def append(self, k, v, layer0=0, stream=None):
        c = self.cfg
        nl = self._layers(k, layer0)
        ntok = k.shape[3] if k.dim() == 5 else -1
        self._check_tensor(k, "k", (nl, c.batch, c.num_kv_heads, ntok, c.head_dim))
        self._check_tensor(v, "v", tuple(k.shape))
        hikv_append(self.h, layer0, k, v, stream)

    def _counts(self, counts, name):
        """HOST int32 [batch] (its address, its sum, what keeps it alive) from
        a list, array or CPU tensor of whole numbers."""
        batch = self.cfg.batch
        if type(counts) in (list, tuple) and len(counts) == batch and set(map(type, counts)) == {int}:
            try:
                a = array.array("i", counts)
            except OverflowError:
                raise ValueError(f"{name} holds values out of range") from None
            low, total, ptr = min(a), sum(a), a.buffer_info()[0]
        else:
            a = np.asarray(counts)
            if a.dtype.kind not in "iu":
                raise TypeError(f"{name} must hold whole numbers")
            if a.shape != (batch,):
                raise ValueError(f"{name} has shape {a.shape}, expected ({batch},)")
            if a.max() > 0x7FFFFFFF or a.min() < -1:
                raise ValueError(f"{name} holds values out of range")
            a = np.ascontiguousarray(a, dtype=np.int32)
            low, total, ptr = int(a.min()), int(a.sum(dtype=np.int64)), a.ctypes.data
        if low < -1:
            raise ValueError(f"{name} holds values out of range")
        return ptr, total, a

    def _rows(self, i, t, name, total, heads):
        """Packed rows [tokens][heads][head_dim] as the C ABI's hikv_rows: a
        reference to the i-th of the structures kept for this cache's calls."""
        try:
            cuda = t.is_cuda
        except AttributeError:
            cuda = False
        if not cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.get_device() != self.device_index:
            raise ValueError(f"{name} is on {t.device}, the cache on cuda:{self.device_index}")
        if t.dtype is not self._torch_dtype or t.shape != (total, heads, self.cfg.head_dim):
            self._check_tensor(t, name, (total, heads, self.cfg.head_dim))
        stride = t.stride()
        if stride[2] != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        r = self._row_args[i]
        r.data, r.token_stride, r.head_stride = t.data_ptr(), stride[0], stride[1]
        return self._row_refs[i]

    def append_packed(self, k, v, ntok, layer=0, q=None, q_out=None, rope=None, stream=None):
        """Append a packed batch to one layer: k, v [sum ntok][Hkv][d] (any
        16-byte strides), sequence b's ntok[b] tokens after those of the
        sequences before it.  With a Rope, k is rotated by position as it
        enters the cache, and q [sum ntok][Hq][d], if given, into q_out (may
        be q itself)."""
        c = self.cfg
        n, total, _keep = self._counts(ntok, "ntok")
        rk, rv = self._rows(0, k, "k", total, c.num_kv_heads), self._rows(1, v, "v", total, c.num_kv_heads)
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        rq = ro = rc = None
        if q is not None:
            rq, ro = self._rows(2, q, "q", total, c.num_q_heads), self._rows(3, q_out, "q_out", total, c.num_q_heads)
        if rope is not None:
            if rope.device_index != self.device_index:
                raise ValueError(f"rope is on {rope.cos.device}, the cache on cuda:{self.device_index}")
            rc = rope.ref
        _check(_lib.hikv_append_packed(self.h, layer, n, rk, rv, rq, ro, rc, self._stream_int(stream)))

    def attend_packed(self, q, out, nq, layer=0, stream=None):
        """Causal attention of the newest nq[b] positions of every sequence
        over everything its units hold up to them: q, out [sum nq][Hq][d]
        (any 16-byte strides that keep their rows apart).  Append the
        positions' tokens first."""
        c = self.cfg
        n, total, _keep = self._counts(nq, "nq")
        rq, ro = self._rows(2, q, "q", total, c.num_q_heads), self._rows(3, out, "out", total, c.num_q_heads)
        _check(_lib.hikv_attend_packed(self.h, layer, n, rq, ro, self._stream_int(stream)))

    def drop(self, counts=None, layer0=0, nlayers=None, stream=None):
        """Drop the newest counts[b] tokens of every unit of batch row b (-1,
        or counts None: all); their positions are free again."""
        n, _, _keep = (None, 0, None) if counts is None else self._counts(counts, "counts")
        nl = self.cfg.num_layers - layer0 if nlayers is None else nlayers
        _check(_lib.hikv_drop(self.h, layer0, nl, n, self._stream_int(stream)))

    def _stream_int(self, stream):
        """The given stream, else the current one of the cache's device."""
        if stream is not None:
            return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        global _RAW_STREAM
        if _RAW_STREAM is None:
            _RAW_STREAM = _raw_stream_fn() or False
        if _RAW_STREAM:
            return _RAW_STREAM(self.device_index)
        import torch
        return torch.cuda.current_stream(self.device_index).cuda_stream

    def device_view(self) -> dict:
        """The cache's own device memory as tensors, without a copy: pages
        [pool_pages][2 (K, V)][page_tokens][d], page_table [units][max_pages],
        importance and positions [units][max_tokens] by slot, lengths
        [units].  Valid until close(); order reads after the calls that write."""
        import torch
        c, w = self.cfg, hikv_view()
        _check(_lib.hikv_device_view(self.h, ctypes.byref(w)))
        pt = c.page_tokens or 64
        bf16 = c.dtype == "bf16"

        def arr(ptr, shape, typestr):
            return torch.as_tensor(_DeviceArray(self, ptr, shape, typestr), device=f"cuda:{self.device_index}")

        pages = arr(w.pool, (w.pool_pages, 2, pt, c.head_dim), "<i2" if bf16 else "<f4")
        return {"pages": pages.view(torch.bfloat16) if bf16 else pages,
                "page_table": arr(w.page_table, (w.units, w.max_pages), "<i4"),
                "importance": arr(w.importance, (w.units, c.max_tokens), "<f4"),
                "positions": arr(w.positions, (w.units, c.max_tokens), "<i4"),
                "lengths": arr(w.lengths, (w.units,), "<i4")}

    def score_window(self, q, layer0=0, stream=None):
        c = self.cfg
        nl = self._layers(q, layer0)
        nq = q.shape[3] if q.dim() == 5 else -1
        self._check_tensor(q, "q", (nl, c.batch, c.num_q_heads, nq, c.head_dim))
        hikv_score_window(self.h, layer0, q, stream)

    def score_band(self, q, band, layer0=0, stream=None):
        """HiKV prefill initialisation: q [nl][B][Hq][n][d] holds the queries
        of every held position; each token's score grows by its attention
        column over the band of queries from its own position."""
        c = self.cfg
        nl = self._layers(q, layer0)
        n = q.shape[3] if q.dim() == 5 else -1
        self._check_tensor(q, "q", (nl, c.batch, c.num_q_heads, n, c.head_dim))
        lens = self.lengths(layer0, nl)
        if lens.size and int(lens[0]) != n:
            raise ValueError(f"q holds {n} positions, the units hold {int(lens[0])} tokens")
        _check(_lib.hikv_score_band(self.h, layer0, nl, int(band), _dev(q, "q"), _stream(stream)))

    def decode_step(self, q, out, layer0=0, stream=None):
        c = self.cfg
        nl = self._layers(q, layer0)
        self._check_tensor(q, "q", (nl, c.batch, c.num_q_heads, c.head_dim))
        self._check_tensor(out, "out", tuple(q.shape))
        hikv_decode_step(self.h, layer0, q, out, stream)

    def selftest_timeout(self, limit_us: int = 20000, stream=None):
        """Enqueue a kernel whose bounded wait runs out (see hikv.h)."""
        _check(_lib.hikv_selftest_timeout(self.h, limit_us, _stream(stream)))

    def kernel_launches(self) -> int:
        """Kernels this cache has launched so far (host counter)."""
        return int(_lib.hikv_kernel_launches(self.h))

    def last_decode_config(self) -> list:
        """The cluster-kernel launches of the latest decode call: units,
        cluster size, clusters and logits placement of each."""
        out = (ctypes.c_int32 * 8)()
        _check(_lib.hikv_last_decode_config(self.h, out))
        return [{"units": out[4 * i], "cluster_size": out[4 * i + 1], "clusters": out[4 * i + 2],
                 "smem_logits": bool(out[4 * i + 3])} for i in range(2) if out[4 * i + 1] > 0]

    def element_rows(self) -> int:
        """V rows the HiKV Stage II decode steps have read so far (synchronous)."""
        r = ctypes.c_int64()
        _check(_lib.hikv_element_rows(self.h, ctypes.byref(r)))
        return int(r.value)

    def step(self, k, v, q, out, evict=True, layer0=0, stream=None):
        """append + decode_step (+ evict) as one call (fused into the attention
        kernel in the steady state).
        The per-step call of a decode loop: each tensor is checked once."""
        import torch
        nl = self._layers(q, layer0)
        shapes = self._step_shapes.get(nl)
        if shapes is None:
            c = self.cfg
            shapes = (torch.Size((nl, c.batch, c.num_kv_heads, 1, c.head_dim)),
                      torch.Size((nl, c.batch, c.num_q_heads, c.head_dim)))
            self._step_shapes[nl] = shapes
        dt = self._dtype()
        kp = _ptr_checked(k, "k", dt, shapes[0])
        vp = _ptr_checked(v, "v", dt, shapes[0])
        qp = _ptr_checked(q, "q", dt, shapes[1])
        op = _ptr_checked(out, "out", dt, shapes[1])
        _check(_lib.hikv_decode_step_fused(self.h, layer0, nl, kp, vp, qp, op, 1 if evict else 0,
                                           _stream_of(q, stream)))

    def evict(self, layer0=0, nlayers=None, stream=None):
        hikv_evict(self.h, layer0, self.cfg.num_layers if nlayers is None else nlayers, stream)

    def lengths(self, layer0=0, nlayers=None) -> np.ndarray:
        nl = self.cfg.num_layers - layer0 if nlayers is None else nlayers
        return hikv_get_lengths(self.h, layer0, nl, self.units_per_layer)

    def gather(self, layer0=0, nlayers=None, cap=None, with_kv=False, stream=None):
        """Retained state of the layers as CUDA tensors (positions ascending)."""
        import torch
        nl = self.cfg.num_layers - layer0 if nlayers is None else nlayers
        nu = nl * self.units_per_layer
        if cap is None:
            cap = max(1, int(self.lengths(layer0, nl).max()))
        dev = torch.device("cuda", torch.cuda.current_device())
        lengths = torch.empty(nu, dtype=torch.int32, device=dev)
        positions = torch.empty(nu, cap, dtype=torch.int32, device=dev)
        importance = torch.empty(nu, cap, dtype=torch.float32, device=dev)
        k_out = v_out = None
        if with_kv:
            dt = torch.bfloat16 if self.cfg.dtype == "bf16" else torch.float32
            k_out = torch.empty(nu, cap, self.cfg.head_dim, dtype=dt, device=dev)
            v_out = torch.empty_like(k_out)
        hikv_gather_retained(self.h, layer0, nl, cap, lengths, positions, importance, k_out, v_out,
                             stream)
        return lengths, positions, importance, k_out, v_out

    def read_slot(self, unit: int, slot: int):
        """Raw contents of one slot (diagnostic, synchronous): K row, V row
        (numpy, bf16 as uint16 bit patterns), importance, position."""
        c = self.cfg
        dt = np.uint16 if c.dtype == "bf16" else np.float32
        k = np.empty(c.head_dim, dt)
        vv = np.empty(c.head_dim, dt)
        imp = ctypes.c_float()
        pos = ctypes.c_int32()
        _check(_lib.hikv_read_slot(self.h, unit, slot, k.ctypes.data, vv.ctypes.data, ctypes.byref(imp),
                                   ctypes.byref(pos)))
        return k, vv, imp.value, pos.value

    def device_status(self):
        hikv_device_status(self.h)
