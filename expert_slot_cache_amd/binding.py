"""ctypes binding of libmoe_pool.so (the C ABI declared in include/moe_pool.h).

Argument marshalling only: every step of the path runs in the library.  Torch
tensors are accepted for convenience and passed as raw device pointers; the
compute stream is a hipStream_t (torch's current stream by default).  The
library must have been built (``python -m expert_slot_cache_amd.build``); a
missing library raises, there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_pool.so")

OK, EINVAL, ENOMEM, EHIP, ERANGE, ESTATE = 0, -1, -2, -3, -4, -5
W_F32, W_BF16, W_INT4_G128 = 0, 1, 2
A_F32, A_BF16 = 0, 1
RULE_DISTINCT, RULE_STATIC = 0, 1
COPY_KERNEL, COPY_DMA = 0, 1
PATH_POOL, PATH_FALLBACK = 0, 1

WTYPES = {"f32": W_F32, "bf16": W_BF16, "int4": W_INT4_G128}
ATYPES = {"f32": A_F32, "bf16": A_BF16}
RULES = {"distinct": RULE_DISTINCT, "static": RULE_STATIC}
COPY_ENGINES = {"dma": COPY_DMA, "kernel": COPY_KERNEL}
POLICY_HOST, POLICY_DEVICE = 0, 1
POLICIES = {"host": POLICY_HOST, "device": POLICY_DEVICE}
EVICT_LRU, EVICT_FIFO, EVICT_LFU, EVICT_SLRU, EVICT_DECAY = 0, 1, 2, 3, 4
EVICTS = {"lru": EVICT_LRU, "fifo": EVICT_FIFO, "lfu": EVICT_LFU, "slru": EVICT_SLRU, "decay": EVICT_DECAY}
ROUTE_SOFTMAX, ROUTE_RENORM = 0, 1
PRODUCT_F32, PRODUCT_BF16, PRODUCT_SWIGLU = 0, 1, 2
SCORES = {"softmax": 0, "sigmoid": 1}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
PREFETCH_AFTER = {"layer": 0, "queued": 1, "previous": 2}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[{status}] {msg}")
        self.status = status


class ExpertRangeError(MoeError):
    pass


class StateError(MoeError):
    pass


class Config(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("n_experts", C.c_int32), ("top_k", C.c_int32),
                ("hidden", C.c_int32), ("inter", C.c_int32), ("n_slots", C.c_int32),
                ("wtype", C.c_int32), ("atype", C.c_int32), ("rule", C.c_int32),
                ("resident", C.c_int32), ("max_tokens", C.c_int32), ("n_copy_streams", C.c_int32),
                ("copy_chunk_bytes", C.c_size_t), ("hbm_budget_bytes", C.c_size_t),
                ("timing", C.c_int32), ("copy_engine", C.c_int32), ("policy", C.c_int32),
                ("read_through", C.c_int32), ("evict", C.c_int32), ("prefetch_slots", C.c_int32)]


class Miss(C.Structure):
    _fields_ = [("expert", C.c_int32), ("slot", C.c_int32), ("evicted", C.c_int32)]


class Stats(C.Structure):
    _fields_ = [("steps", C.c_uint64), ("hits", C.c_uint64), ("misses", C.c_uint64),
                ("fallbacks", C.c_uint64), ("bytes_h2d", C.c_uint64), ("staged", C.c_uint64),
                ("prefetched", C.c_uint64), ("prefetch_bytes", C.c_uint64), ("moves", C.c_uint64)]


class Timing(C.Structure):
    _fields_ = [("copy_ms", C.c_double), ("copy_calls", C.c_uint64), ("copy_bytes", C.c_uint64),
                ("w13_ms", C.c_double), ("w2_ms", C.c_double), ("kernel_calls", C.c_uint64),
                ("sync_wait_ms", C.c_double)]


_P = C.c_void_p
_I32 = C.c_int32
_I64 = C.c_int64
_PI32 = C.POINTER(C.c_int32)

_SIGS = {
    "moe_strerror": (C.c_char_p, [_I32]),
    "moe_last_error": (C.c_char_p, []),
    "moe_expert_bytes": (C.c_size_t, [_I32, _I32, _I32]),
    "moe_pool_create": (_I32, [C.POINTER(Config), _P, C.POINTER(_P)]),
    "moe_pool_destroy": (None, [_P]),
    "moe_pool_load_expert": (_I32, [_P, _I32, _I32, _P, C.c_size_t]),
    "moe_pool_reset": (_I32, [_P]),
    "moe_pool_prepare": (_I32, [_P, _I32, _P, _I32, _P, C.POINTER(Miss), _I32, _PI32, _PI32]),
    "moe_pool_forward": (_I32, [_P, _I32, _P, _P, _P, _P, _I32, _P]),
    "moe_pool_step": (_I32, [_P, _I32, _P, _I32, _P, _P, _P, _P, _P, C.POINTER(Miss), _I32, _PI32,
                             _PI32]),
    "moe_pool_sync": (_I32, [_P]),
    "moe_pool_prefetch": (_I32, [_P, _I32, _P, _I32, _I32]),
    "moe_pool_last_step": (_I32, [_P, _I32, _PI32, C.POINTER(Miss), _I32, _PI32]),
    "moe_pool_get_stats": (_I32, [_P, _I32, C.POINTER(Stats)]),
    "moe_pool_get_state": (_I32, [_P, _I32, _P, _P, _P]),
    "moe_pool_read_slot": (_I32, [_P, _I32, _I32, _P, C.c_size_t]),
    "moe_pool_slot_ptr": (_I32, [_P, _I32, _I32, C.POINTER(_P)]),
    "moe_pool_store_ptr": (_I32, [_P, _I32, _I32, C.POINTER(_P)]),
    "moe_ptr_is_pinned_host": (_I32, [_P, _PI32]),
    "moe_pool_get_timing": (_I32, [_P, C.POINTER(Timing)]),
    "moe_pool_reset_timing": (_I32, [_P]),
    "moe_pool_set_timing": (_I32, [_P, _I32]),
    "moe_read_calibration": (_I32, [_P, C.c_size_t, C.c_size_t, _I32, _P, C.POINTER(C.c_double)]),
    "moe_link_calibration": (_I32, [C.c_size_t, _I32, _I32, _I32, _P, C.POINTER(C.c_double)]),
    "moe_pool_set_slots": (_I32, [_P, _I32]),
    "moe_pool_set_eviction": (_I32, [_P, _I32]),
    "moe_forward_slots": (_I32, [_I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _I32, _P, _P]),
    "moe_route": (_I32, [_I32, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_route_backward": (_I32, [_I32, _P, _I64, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _I64, _P]),
    "moe_sort_tokens": (_I32, [_I32, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "moe_sort_workspace_bytes": (C.c_size_t, [_I32, _I32, _I32]),
    "moe_combine_rows": (_I32, [_I32, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P]),
    "moe_combine_rows_backward": (_I32, [_I32, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_scaled_product": (_I32, [_P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_route_groups": (_I32, [_I32, _P, _I64, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, C.c_float, _P, _P, _P]),
    "moe_route_groups_backward": (_I32, [_I32, _P, _I64, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, C.c_float, _P, _I64, _P]),
    "moe_expert_product": (_I32, [_I32, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _P]),
    "moe_activation_backward": (_I32, [_I32, _P, _I32, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, C.c_size_t, _P]),
    "moe_activation_backward_workspace_bytes": (C.c_size_t, [_I32, _I32, _I32]),
    "moe_expert_product_backward": (_I32, [_I32, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _I32, _P, _P, C.c_size_t, _P]),
    "moe_expert_product_backward_workspace_bytes": (C.c_size_t, [_I32, _I32, _I32, _I32, _I32]),
    "moe_lru_create": (_I32, [_I32, _I32, _I32, C.POINTER(_P)]),
    "moe_lru_destroy": (None, [_P]),
    "moe_lru_step": (_I32, [_P, _P, _I32, _I32, _P, C.POINTER(Miss), _I32, _PI32, _PI32]),
    "moe_lru_get_state": (_I32, [_P, _P, _P, _P]),
    "moe_lru_get_stats": (_I32, [_P, C.POINTER(Stats)]),
}

_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m expert_slot_cache_amd.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return sorted(_SIGS)


def _check(status: int):
    if status == OK:
        return
    msg = lib().moe_last_error().decode(errors="replace")
    if status == ERANGE:
        raise ExpertRangeError(status, msg)
    if status == ESTATE:
        raise StateError(status, msg)
    raise MoeError(status, msg)


def forward_slots(*, wtype: str, atype: str, hidden: int, inter: int, top_k: int, slots, n_slots: int,
                  slot_ids, x, topk_w, out, n_tokens: int, resid=None, stream=None):
    """moe_forward_slots: the fused MoE over caller-held slots, scratch in the library's
    static device array (no allocation)."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    _check(lib().moe_forward_slots(WTYPES[wtype], ATYPES[atype], hidden, inter, top_k, _ptr(slots), n_slots,
                                   _ptr(slot_ids), _ptr(x), _ptr(topk_w), _ptr(resid), n_tokens, _ptr(out),
                                   C.c_void_p(stream)))


def expert_bytes(wtype: str, hidden: int, inter: int) -> int:
    return int(lib().moe_expert_bytes(WTYPES[wtype], hidden, inter))


def _ptr(t) -> int:
    """Device/host address of a torch tensor, a numpy array, or an int."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _misses(buf, n):
    return [(buf[i].expert, buf[i].slot, buf[i].evicted) for i in range(n)]


class MoePool:
    """One pool object: n_layers layers of n_slots HBM slots over a pinned store."""

    def __init__(self, *, layers: int, experts: int, top_k: int, hidden: int, inter: int,
                 slots: int, wtype: str = "bf16", atype: str = "bf16", rule: str = "distinct",
                 resident: bool = False, max_tokens: int = 1, copy_streams: int = 1,
                 copy_chunk_bytes: int = 0, hbm_budget_bytes: int = 0, timing: int = 0,
                 copy_engine: str = "kernel", policy: str = "host", read_through: bool = False,
                 evict: str = "lru", prefetch_slots: int = 0, stream=None):
        self._h = None
        cfg = Config(layers, experts, top_k, hidden, inter, slots, WTYPES[wtype], ATYPES[atype],
                     RULES[rule], int(bool(resident)), max_tokens, copy_streams,
                     copy_chunk_bytes, hbm_budget_bytes, int(timing), COPY_ENGINES[copy_engine],
                     POLICIES[policy], int(bool(read_through)), EVICTS[evict], int(prefetch_slots))
        if stream is None:
            import torch
            stream = torch.cuda.current_stream().cuda_stream
        h = C.c_void_p()
        _check(lib().moe_pool_create(C.byref(cfg), C.c_void_p(stream), C.byref(h)))
        self._h = h
        self.cfg = cfg
        self.layers, self.experts, self.top_k = layers, experts, top_k
        self.hidden, self.inter, self.slots = hidden, inter, slots
        self.wtype, self.atype, self.resident = wtype, atype, resident
        self.policy = policy
        self.evict = evict
        self.read_through = bool(read_through)
        self.max_tokens = max_tokens
        self.expert_nbytes = expert_bytes(wtype, hidden, inter)
        self._miss_buf = (Miss * max(1, experts))()

    # -- lifetime ----------------------------------------------------------------
    def close(self):
        if self._h is not None and self._h.value:
            lib().moe_pool_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # -- store -------------------------------------------------------------------
    def load_expert(self, layer: int, expert: int, data: np.ndarray):
        b = np.ascontiguousarray(data).view(np.uint8).ravel()
        _check(lib().moe_pool_load_expert(self._h, layer, expert, b.ctypes.data, b.size))

    def reset(self):
        _check(lib().moe_pool_reset(self._h))

    def set_slots(self, n_slots: int):
        """Slots per layer from now on (<= the count at create); the pool goes cold."""
        _check(lib().moe_pool_set_slots(self._h, n_slots))
        self.slots = n_slots

    def set_eviction(self, evict: str):
        """Eviction policy from now on ("lru", "fifo", "lfu", "slru", "decay"); the pool
        goes cold."""
        _check(lib().moe_pool_set_eviction(self._h, EVICTS[evict]))
        self.evict = evict

    # -- the step ------------------------------------------------------------------
    def prepare(self, layer: int, topk_ids, n_tokens: int, slot_ids):
        """topk_ids/slot_ids: int32 [n_tokens, top_k] on the device (tensor or address).
        Returns (path, misses) with misses a list of (expert, slot, evicted)."""
        nm, path = C.c_int32(0), C.c_int32(0)
        _check(lib().moe_pool_prepare(self._h, layer, _ptr(topk_ids), n_tokens, _ptr(slot_ids),
                                      self._miss_buf, len(self._miss_buf), C.byref(nm),
                                      C.byref(path)))
        return path.value, _misses(self._miss_buf, min(nm.value, len(self._miss_buf)))

    def prepare_raw(self, layer: int, ids_ptr: int, n_tokens: int, slot_ptr: int) -> int:
        """prepare() without building the miss list; returns the path."""
        path = C.c_int32(0)
        _check(lib().moe_pool_prepare(self._h, layer, ids_ptr, n_tokens, slot_ptr, None, 0, None,
                                      C.byref(path)))
        return path.value

    def forward(self, layer: int, x, slot_ids, topk_w, out, n_tokens: int, resid=None):
        _check(lib().moe_pool_forward(self._h, layer, _ptr(x), _ptr(slot_ids), _ptr(topk_w),
                                      _ptr(resid), n_tokens, _ptr(out)))
        return out

    def step(self, layer: int, topk_ids, n_tokens: int, slot_ids, x, topk_w, out, resid=None):
        """prepare + forward in one call; returns (path, misses)."""
        nm, path = C.c_int32(0), C.c_int32(0)
        _check(lib().moe_pool_step(self._h, layer, _ptr(topk_ids), n_tokens, _ptr(slot_ids), _ptr(x),
                                   _ptr(topk_w), _ptr(resid), _ptr(out), self._miss_buf,
                                   len(self._miss_buf), C.byref(nm), C.byref(path)))
        return path.value, _misses(self._miss_buf, min(nm.value, len(self._miss_buf)))

    def sync(self):
        _check(lib().moe_pool_sync(self._h))

    def prefetch(self, layer: int, predicted_ids, n_tokens: int, after: str = "queued"):
        """Hint: the next step of `layer` will use these ids (int32 [n_tokens, top_k] on
        the device); predicted experts the layer does not hold are copied into its
        prefetch buffer on a copy stream, starting after everything queued on the compute
        stream ("queued"), after the layer's last step ("layer") or after the previous
        prefetch ("previous")."""
        _check(lib().moe_pool_prefetch(self._h, layer, _ptr(predicted_ids), n_tokens, PREFETCH_AFTER[after]))

    def last_step(self, layer: int):
        """(path, misses) of the layer's last prepare/step (waits for it under the
        device policy)."""
        nm, path = C.c_int32(0), C.c_int32(0)
        _check(lib().moe_pool_last_step(self._h, layer, C.byref(path), self._miss_buf, len(self._miss_buf),
                                        C.byref(nm)))
        return path.value, _misses(self._miss_buf, min(nm.value, len(self._miss_buf)))

    # -- introspection ---------------------------------------------------------------
    def stats(self, layer: int = -1) -> dict:
        s = Stats()
        _check(lib().moe_pool_get_stats(self._h, layer, C.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in Stats._fields_}

    def state(self, layer: int):
        m = np.empty(self.experts, np.int32)
        n = max(1, self.slots)
        o = np.empty(n, np.int32)
        l = np.empty(n, np.int32)
        _check(lib().moe_pool_get_state(self._h, layer, m.ctypes.data, o.ctypes.data, l.ctypes.data))
        k = self.slots if not self.resident else 0
        return m, o[:k], l[:k]

    def read_slot(self, layer: int, slot: int, n: int | None = None) -> np.ndarray:
        n = self.expert_nbytes if n is None else n
        buf = np.empty(n, np.uint8)
        _check(lib().moe_pool_read_slot(self._h, layer, slot, buf.ctypes.data, n))
        return buf

    def read_staging(self, rank: int, n: int | None = None) -> np.ndarray:
        return self.read_slot(0, -rank - 1, n)

    def slot_ptr(self, layer: int, slot: int) -> int:
        p = C.c_void_p()
        _check(lib().moe_pool_slot_ptr(self._h, layer, slot, C.byref(p)))
        return p.value

    def store_ptr(self, layer: int, expert: int) -> int:
        p = C.c_void_p()
        _check(lib().moe_pool_store_ptr(self._h, layer, expert, C.byref(p)))
        return p.value

    def store_view(self, layer: int, expert: int) -> np.ndarray:
        """numpy view of an expert's bytes in the pinned store (for bulk filling)."""
        addr = self.store_ptr(layer, expert)
        buf = (C.c_uint8 * self.expert_nbytes).from_address(addr)
        return np.frombuffer(buf, dtype=np.uint8)

    def timing(self) -> dict:
        t = Timing()
        _check(lib().moe_pool_get_timing(self._h, C.byref(t)))
        return {f: (float(getattr(t, f)) if "ms" in f else int(getattr(t, f)))
                for f, _ in Timing._fields_}

    def reset_timing(self):
        _check(lib().moe_pool_reset_timing(self._h))

    def set_timing(self, every: int):
        """Event-timing period from now on (0 = off, e.g. before a graph capture)."""
        _check(lib().moe_pool_set_timing(self._h, int(every)))


def read_calibration(buf, bytes_per_launch: int, reps: int = 20, stream=None) -> float:
    """Mean event-timed duration (us) of a plain streaming read of bytes_per_launch,
    rotating over the device buffer `buf` (a torch tensor)."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    us = C.c_double(0)
    _check(lib().moe_read_calibration(_ptr(buf), buf.numel() * buf.element_size(), bytes_per_launch, reps,
                                      C.c_void_p(stream), C.byref(us)))
    return us.value


def link_calibration(nbytes: int, engine: str = "kernel", reps: int = 8, streams: int = 1, stream=None) -> float:
    """Mean event-timed duration (us) of one pinned host -> HBM copy of nbytes with
    the given engine ("kernel" or "dma"), split over `streams` streams."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    us = C.c_double(0)
    _check(lib().moe_link_calibration(nbytes, reps, COPY_ENGINES[engine], streams, C.c_void_p(stream),
                                      C.byref(us)))
    return us.value


def is_pinned_host(addr: int) -> bool:
    v = C.c_int32(0)
    _check(lib().moe_ptr_is_pinned_host(addr, C.byref(v)))
    return bool(v.value)


# ---- the operators around the experts ------------------------------------------------
# On torch tensors of the current device, whose shapes give the sizes; every output is the
# caller's buffer.  include/moe_pool.h documents each operator.


def _bad(what: str):
    raise MoeError(EINVAL, what)


def _check_tensor(name: str, t, dtype, shape, dev: int):
    """t lies on device `dev`, is contiguous and of this dtype and shape."""
    if t is not None and t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return
    if t is None:
        _bad(f"{name} is missing")
    if t.get_device() != dev:
        _bad(f"{name} is not on the current device, cuda:{dev}")
    if t.dtype is not dtype:
        _bad(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        _bad(f"{name} is {tuple(t.shape)}, not {tuple(shape)}")
    _bad(f"{name} is not contiguous")


def _sizes(name: str, t, dims: int):
    """The shape of t, every size of which the library's int32 holds."""
    if t is None:
        _bad(f"{name} is missing")
    shape = t.shape
    if len(shape) != dims:
        _bad(f"{name} has {len(shape)} dimensions, not {dims}")
    for n in shape:
        if n > 0x7fffffff:
            _bad(f"{name} is {tuple(shape)}: sizes above 2^31 - 1")
    return shape


def _array(name: str, t, dtype, dev: int, dims: int = 2):
    """The shape of a contiguous array of this dtype on device `dev`."""
    shape = _sizes(name, t, dims)
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous():
        _check_tensor(name, t, dtype, shape, dev)
    return shape


def _rows(name: str, t, dev: int):
    """(rows, values of a row, elements from one row to the next) of a matrix on device `dev`
    whose rows may be apart."""
    n, h = _sizes(name, t, 2)
    stride, one = t.stride()
    if t.get_device() != dev:
        _bad(f"{name} is not on the current device, cuda:{dev}")
    if one != 1 and h > 1:
        _bad(f"the values of a row of {name} are not contiguous")
    return n, h, stride if n > 1 else h


def _atype(torch, name: str, t) -> int:
    if t is None:
        _bad(f"{name} is missing")
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return A_BF16
    if dtype is torch.float32:
        return A_F32
    _bad(f"{name} is {dtype}, not float32 or bfloat16")


def _place(torch, stream):
    """The current device and the stream to use on it (torch's current one by default)."""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream


def route(logits, topk_ids, topk_w, *, renorm: bool = True, stream=None):
    """moe_route: logits [T, E] (fp32 or bf16, rows may be apart) -> topk_ids int32 [T, K] and
    topk_w fp32 [T, K]; renorm: the weights of a token sum to one."""
    import torch
    dev, s = _place(torch, stream)
    T, E, stride = _rows("logits", logits, dev)
    shape = _array("topk_ids", topk_ids, torch.int32, dev)
    if shape[0] != T:
        _bad(f"topk_ids has {shape[0]} rows, logits {T}")
    _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    _check(lib().moe_route(_atype(torch, "logits", logits), logits.data_ptr(), stride, T, E, shape[1],
                           ROUTE_RENORM if renorm else ROUTE_SOFTMAX, topk_ids.data_ptr(), topk_w.data_ptr(), s))


def route_backward(logits, topk_ids, topk_w, d_topk_w, d_logits, *, renorm: bool = True, stream=None):
    """moe_route_backward: d_topk_w fp32 [T, K] -> d_logits [T, E] in the logits' type, for what
    route gave on these logits (with renorm they are not read and may be None)."""
    import torch
    dev, s = _place(torch, stream)
    T, E, d_stride = _rows("d_logits", d_logits, dev)
    stride = E
    if logits is not None:
        n, e, stride = _rows("logits", logits, dev)
        if (n, e) != (T, E) or logits.dtype is not d_logits.dtype:
            _bad(f"logits are {logits.dtype} {(n, e)}, d_logits {d_logits.dtype} {(T, E)}")
    shape = _array("topk_ids", topk_ids, torch.int32, dev)
    if shape[0] != T:
        _bad(f"topk_ids has {shape[0]} rows, d_logits {T}")
    _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    _check_tensor("d_topk_w", d_topk_w, torch.float32, shape, dev)
    _check(lib().moe_route_backward(_atype(torch, "d_logits", d_logits), _ptr(logits),
                                    stride, topk_ids.data_ptr(), topk_w.data_ptr(), d_topk_w.data_ptr(), T, E, shape[1],
                                    ROUTE_RENORM if renorm else ROUTE_SOFTMAX, d_logits.data_ptr(), d_stride, s))


def _named(what: str, names: dict, name) -> int:
    if name not in names:
        _bad(f"{what} {name!r}: one of {', '.join(names)}")
    return names[name]


def route_groups(logits, topk_ids, topk_w, *, bias=None, score: str = "softmax", renorm: bool = True, n_groups: int = 1,
                 kept_groups: int | None = None, group_top: int = 1, scale: float = 1.0, stream=None):
    """moe_route_groups: logits [T, E] (fp32 or bf16, rows may be apart) -> topk_ids int32 [T, K] and
    topk_w fp32 [T, K], chosen by score ("softmax" or "sigmoid") plus bias fp32 [E] among the
    kept_groups (None: all) of n_groups groups whose group_top largest choices sum highest."""
    import torch
    dev, s = _place(torch, stream)
    T, E, stride = _rows("logits", logits, dev)
    shape = _array("topk_ids", topk_ids, torch.int32, dev)
    if shape[0] != T:
        _bad(f"topk_ids has {shape[0]} rows, logits {T}")
    _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    if bias is not None:
        _check_tensor("bias", bias, torch.float32, (E,), dev)
    at, code = _atype(torch, "logits", logits), _named("score", SCORES, score)
    _check(lib().moe_route_groups(at, logits.data_ptr(), stride, _ptr(bias), T, E, shape[1], code,
                                  ROUTE_RENORM if renorm else ROUTE_SOFTMAX, n_groups,
                                  n_groups if kept_groups is None else kept_groups, group_top, scale, topk_ids.data_ptr(),
                                  topk_w.data_ptr(), s))


def route_groups_backward(logits, topk_ids, topk_w, d_topk_w, d_logits, *, score: str = "softmax", renorm: bool = True,
                          scale: float = 1.0, stream=None):
    """moe_route_groups_backward: d_topk_w fp32 [T, K] -> d_logits [T, E] in the logits' type, for
    what route_groups gave on these logits with this score, renorm and scale (softmax with renorm
    does not read them: they may be None)."""
    import torch
    dev, s = _place(torch, stream)
    T, E, d_stride = _rows("d_logits", d_logits, dev)
    stride = E
    if logits is not None:
        n, e, stride = _rows("logits", logits, dev)
        if (n, e) != (T, E) or logits.dtype is not d_logits.dtype:
            _bad(f"logits are {logits.dtype} {(n, e)}, d_logits {d_logits.dtype} {(T, E)}")
    shape = _array("topk_ids", topk_ids, torch.int32, dev)
    if shape[0] != T:
        _bad(f"topk_ids has {shape[0]} rows, d_logits {T}")
    _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    _check_tensor("d_topk_w", d_topk_w, torch.float32, shape, dev)
    at, code = _atype(torch, "d_logits", d_logits), _named("score", SCORES, score)
    _check(lib().moe_route_groups_backward(at, _ptr(logits), stride, topk_ids.data_ptr(), topk_w.data_ptr(),
                                           d_topk_w.data_ptr(), T, E, shape[1], code, ROUTE_RENORM if renorm else ROUTE_SOFTMAX,
                                           scale, d_logits.data_ptr(), d_stride, s))


def sort_workspace_bytes(n_tokens: int, top_k: int, experts: int) -> int:
    if max(n_tokens, top_k, experts) > 0x7fffffff:
        return 0
    return int(lib().moe_sort_workspace_bytes(n_tokens, top_k, experts))


def sort_tokens(x, topk_ids, sorted_x, offsets, rows, *, scales=None, workspace=None, stream=None):
    """moe_sort_tokens: x [T, H] (fp32 or bf16, rows may be apart) and topk_ids int32 [T, K] ->
    sorted_x [T*K, H] (x's type, or float8_e4m3fn with scales fp32 [T*K, ceil(H/128)]), offsets
    int32 [experts + 1] and rows int32 [T, K].  x and sorted_x None: the places only.
    workspace: uint8, sort_workspace_bytes(T, K, experts) of them; None: taken from torch's
    allocator for this call (on torch's current stream only)."""
    import torch
    dev, s = _place(torch, stream)
    shape = T, K = _array("topk_ids", topk_ids, torch.int32, dev)
    _check_tensor("rows", rows, torch.int32, shape, dev)
    E = _sizes("offsets", offsets, 1)[0] - 1
    _check_tensor("offsets", offsets, torch.int32, (E + 1,), dev)
    H = at = f8 = stride = 0
    if x is None:
        if sorted_x is not None or scales is not None:
            _bad("sorted rows need x")
    else:
        n, H, stride = _rows("x", x, dev)
        if n != T:
            _bad(f"x has {n} rows, topk_ids {T}")
        at = _atype(torch, "x", x)
        f8 = int(scales is not None)
        _check_tensor("sorted_x", sorted_x, torch.float8_e4m3fn if f8 else x.dtype, (T * K, H), dev)
        if f8:
            _check_tensor("scales", scales, torch.float32, (T * K, -(-H // 128)), dev)
    L = lib()
    need = L.moe_sort_workspace_bytes(T, K, E)
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, workspace.shape, dev)
        need = workspace.numel()
    elif need:
        if stream is not None and stream != torch.cuda.current_stream(dev).cuda_stream:
            _bad("a sort on a stream that is not torch's current one needs its workspace from the caller")
        workspace = torch.empty(need, dtype=torch.uint8, device=topk_ids.device)
    _check(L.moe_sort_tokens(at, _ptr(x), stride, topk_ids.data_ptr(), T, K, E, H, f8, _ptr(sorted_x), _ptr(scales),
                             offsets.data_ptr(), rows.data_ptr(), _ptr(workspace), need, s))


def combine_rows(ys, rows, out, *, topk_w=None, resid=None, stream=None):
    """moe_combine_rows: ys [T*K, H] (fp32 or bf16) at rows int32 [T, K], times topk_w fp32 [T, K]
    (None: ones), summed with resid [T, H] (optional) into out [T, H].  Without weights it is
    the gradient of sort_tokens."""
    import torch
    dev, s = _place(torch, stream)
    shape = T, K = _array("rows", rows, torch.int32, dev)
    at = _atype(torch, "out", out)
    n, H = _array("out", out, out.dtype, dev)
    if n != T:
        _bad(f"out has {n} rows, rows {T}")
    _check_tensor("ys", ys, out.dtype, (T * K, H), dev)
    if topk_w is not None:
        _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    if resid is not None:
        _check_tensor("resid", resid, out.dtype, (T, H), dev)
    _check(lib().moe_combine_rows(at, ys.data_ptr(), rows.data_ptr(), _ptr(topk_w), _ptr(resid),
                                  T, K, H, out.data_ptr(), s))


def combine_rows_backward(d_out, ys, rows, topk_w, d_ys, d_topk_w, *, stream=None):
    """moe_combine_rows_backward: d_out [T, H] -> d_ys [T*K, H] (rows that no pair has are left as
    they are) and d_topk_w fp32 [T, K], for what combine_rows took."""
    import torch
    dev, s = _place(torch, stream)
    shape = T, K = _array("rows", rows, torch.int32, dev)
    at = _atype(torch, "d_out", d_out)
    n, H = _array("d_out", d_out, d_out.dtype, dev)
    if n != T:
        _bad(f"d_out has {n} rows, rows {T}")
    _check_tensor("ys", ys, d_out.dtype, (T * K, H), dev)
    _check_tensor("d_ys", d_ys, d_out.dtype, (T * K, H), dev)
    _check_tensor("topk_w", topk_w, torch.float32, shape, dev)
    _check_tensor("d_topk_w", d_topk_w, torch.float32, shape, dev)
    _check(lib().moe_combine_rows_backward(at, d_out.data_ptr(), ys.data_ptr(), rows.data_ptr(), topk_w.data_ptr(),
                                           T, K, H, d_ys.data_ptr(), d_topk_w.data_ptr(), s))


def scaled_product(x, x_scales, w, w_scales, out, *, offsets=None, swiglu_scales=None, stream=None):
    """moe_scaled_product: rows x [M, K] (float8_e4m3fn, x_scales fp32 [M, ceil(K/128)]), sorted by
    group as offsets int32 [G + 1] says (None: one group), times w [G, N, K] (float8_e4m3fn,
    w_scales fp32 [G, ceil(N/128), ceil(K/128)]) into out [M, N], fp32 or bf16.  With
    swiglu_scales fp32 [M, N/256]: out is float8_e4m3fn [M, N/2], silu(gate) * up rounded."""
    import torch
    dev, s = _place(torch, stream)
    f8, f32 = torch.float8_e4m3fn, torch.float32
    M, K = _array("x", x, f8, dev)
    G, N, depth = _array("w", w, f8, dev, 3)
    if depth != K:
        _bad(f"rows of w have {depth} values, of x {K}")
    kb = -(-K // 128)
    _check_tensor("x_scales", x_scales, f32, (M, kb), dev)
    _check_tensor("w_scales", w_scales, f32, (G, -(-N // 128), kb), dev)
    if offsets is not None:
        _check_tensor("offsets", offsets, torch.int32, (G + 1,), dev)
    if swiglu_scales is not None:
        ep = PRODUCT_SWIGLU
        _check_tensor("out", out, f8, (M, N // 2), dev)
        _check_tensor("swiglu_scales", swiglu_scales, f32, (M, N // 256), dev)
    else:
        ep = PRODUCT_BF16 if _atype(torch, "out", out) == A_BF16 else PRODUCT_F32
        _check_tensor("out", out, out.dtype, (M, N), dev)
    _check(lib().moe_scaled_product(x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), _ptr(offsets),
                                    M, G, N, K, ep, out.data_ptr(), _ptr(swiglu_scales), s))


def _workspace(torch, what: str, workspace, need: int, dev: int, like, stream):
    """The caller's workspace, or one of torch's allocator for this call; and its bytes."""
    if workspace is not None:
        _check_tensor("workspace", workspace, torch.uint8, workspace.shape, dev)
        return workspace, workspace.numel()
    if need == 0:
        return None, 0
    if stream is not None and stream != torch.cuda.current_stream(dev).cuda_stream:
        _bad(f"{what} on a stream that is not torch's current one needs its workspace from the caller")
    return torch.empty(need, dtype=torch.uint8, device=like.device), need


def _same_or_f32(torch, name: str, t, kind) -> int:
    at = _atype(torch, name, t)
    if t.dtype is not kind and at != A_F32:
        _bad(f"{name} is {t.dtype}, not float32 or {kind}")
    return at


def expert_product(x, w, out, *, bias=None, resid=None, pre=None, act: str = "none", offsets=None, stream=None):
    """moe_expert_product: rows x [M, K] (fp32 or bf16), sorted by group as offsets int32 [G + 1] says
    (None: one group), times w [G, N, K] of their type; with bias fp32 [G, N], act ("none", "relu",
    "gelu", "silu" or "swiglu") and resid into out [M, N] ("swiglu": [M, N/2]), fp32 or x's type.
    pre [M, N] in x's type gets the values before the activation."""
    import torch
    dev, s = _place(torch, stream)
    at = _atype(torch, "x", x)
    M, K = _array("x", x, x.dtype, dev)
    G, N, depth = _array("w", w, x.dtype, dev, 3)
    if depth != K:
        _bad(f"rows of w have {depth} values, of x {K}")
    code = _named("act", ACTS, act)
    ot = _same_or_f32(torch, "out", out, x.dtype)
    cols = N // 2 if act == "swiglu" else N
    _check_tensor("out", out, out.dtype, (M, cols), dev)
    if bias is not None:
        _check_tensor("bias", bias, torch.float32, (G, N), dev)
    if resid is not None:
        _check_tensor("resid", resid, out.dtype, (M, cols), dev)
    if pre is not None:
        _check_tensor("pre", pre, x.dtype, (M, N), dev)
    if offsets is not None:
        _check_tensor("offsets", offsets, torch.int32, (G + 1,), dev)
    _check(lib().moe_expert_product(at, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(offsets), _ptr(resid), M, G, N, K, code,
                                    ot, out.data_ptr(), _ptr(pre), s))


def activation_backward(d_out, pre, d_pre=None, *, d_bias=None, act: str = "none", offsets=None, workspace=None, stream=None):
    """moe_activation_backward: d_out [M, N] ("swiglu": [M, N/2]), fp32 or pre's type, and pre [M, N]
    ("none": not read, may be None) -> d_pre [M, N] in pre's type and d_bias fp32 [G, N] (each
    optional), for what expert_product took.  workspace: uint8, moe_activation_backward_
    workspace_bytes(M, G, N) of them where d_bias is given; None: taken from torch's allocator
    for this call (on torch's current stream only)."""
    import torch
    dev, s = _place(torch, stream)
    code = _named("act", ACTS, act)
    ot = _atype(torch, "d_out", d_out)
    M, cols = _array("d_out", d_out, d_out.dtype, dev)
    N = 2 * cols if act == "swiglu" else cols
    like = pre if pre is not None else d_pre if d_pre is not None else d_out
    at, kind = _atype(torch, "pre" if like is pre else "d_pre", like), like.dtype
    if act != "none" or pre is not None:
        _check_tensor("pre", pre, kind, (M, N), dev)
    _same_or_f32(torch, "d_out", d_out, kind)
    if d_pre is not None:
        _check_tensor("d_pre", d_pre, kind, (M, N), dev)
    G = 1
    if offsets is not None:
        G = _sizes("offsets", offsets, 1)[0] - 1
        _check_tensor("offsets", offsets, torch.int32, (G + 1,), dev)
    need = 0
    if d_bias is not None:
        _check_tensor("d_bias", d_bias, torch.float32, (G, N), dev)
        need = lib().moe_activation_backward_workspace_bytes(M, G, N) if N <= 0x7fffffff else 0
    workspace, size = _workspace(torch, "a bias' gradient", workspace, need, dev, d_out, stream)
    _check(lib().moe_activation_backward(at, d_out.data_ptr(), ot, _ptr(pre), _ptr(offsets), M, G, N, code, _ptr(d_pre),
                                         _ptr(d_bias), _ptr(workspace), size, s))


def activation_backward_workspace_bytes(n_rows: int, n_groups: int, n_cols: int) -> int:
    if max(n_rows, n_groups, n_cols) > 0x7fffffff:
        return 0
    return int(lib().moe_activation_backward_workspace_bytes(n_rows, n_groups, n_cols))


def expert_product_backward(d_pre, x, w, *, d_x=None, d_w=None, offsets=None, workspace=None, stream=None):
    """moe_expert_product_backward: d_pre [M, N] (fp32 or bf16), x [M, K] and w [G, N, K] of its type ->
    d_x [M, K] in their type and d_w [G, N, K], fp32 or their type (each optional; w is read for
    d_x alone and x for d_w alone: the other may be None).  workspace: uint8,
    expert_product_backward_workspace_bytes(...) of them; None: taken from torch's allocator for
    this call (on torch's current stream only)."""
    import torch
    dev, s = _place(torch, stream)
    at = _atype(torch, "d_pre", d_pre)
    kind = d_pre.dtype
    M, N = _array("d_pre", d_pre, kind, dev)
    if d_x is None and d_w is None:
        _bad("d_x and d_w are missing")
    wt, G, K = A_F32, 1, 0
    if d_w is not None:
        wt = _same_or_f32(torch, "d_w", d_w, kind)
        G, n, K = _array("d_w", d_w, d_w.dtype, dev, 3)
        if n != N:
            _bad(f"d_w has {n} rows a matrix, d_pre {N} columns")
        _check_tensor("x", x, kind, (M, K), dev)
    if d_x is not None:
        if d_w is None:
            G, n, K = _array("w", w, kind, dev, 3)
            if n != N:
                _bad(f"w has {n} rows a matrix, d_pre {N} columns")
        else:
            _check_tensor("w", w, kind, (G, N, K), dev)
        _check_tensor("d_x", d_x, kind, (M, K), dev)
    if offsets is not None:
        _check_tensor("offsets", offsets, torch.int32, (G + 1,), dev)
    need = lib().moe_expert_product_backward_workspace_bytes(at, M, G, N, K) if d_w is not None else 0
    workspace, size = _workspace(torch, "a matrix' gradient", workspace, need, dev, d_pre, stream)
    _check(lib().moe_expert_product_backward(at, d_pre.data_ptr(), x.data_ptr() if d_w is not None else None,
                                             w.data_ptr() if d_x is not None else None, _ptr(offsets), M, G, N, K, _ptr(d_x),
                                             wt, _ptr(d_w), _ptr(workspace), size, s))


def expert_product_backward_workspace_bytes(kind: str, n_rows: int, n_groups: int, n_cols: int, depth: int) -> int:
    """kind: "f32" or "bf16", the type of the rows."""
    if max(n_rows, n_groups, n_cols, depth) > 0x7fffffff:
        return 0
    return int(lib().moe_expert_product_backward_workspace_bytes(ATYPES[kind], n_rows, n_groups, n_cols, depth))


class SlotLRU:
    """The library's slot manager on host ids (no GPU)."""

    def __init__(self, experts: int, slots: int, rule: str = "distinct"):
        self._h = None
        h = C.c_void_p()
        _check(lib().moe_lru_create(experts, slots, RULES[rule], C.byref(h)))
        self._h = h
        self.experts, self.slots = experts, slots
        self._miss_buf = (Miss * max(1, experts))()

    def close(self):
        if self._h is not None and self._h.value:
            lib().moe_lru_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step(self, ids: np.ndarray):
        ids = np.ascontiguousarray(ids, dtype=np.int32)
        T, K = ids.shape
        out = np.empty_like(ids)
        nm, path = C.c_int32(0), C.c_int32(0)
        _check(lib().moe_lru_step(self._h, ids.ctypes.data, T, K, out.ctypes.data, self._miss_buf,
                                  len(self._miss_buf), C.byref(nm), C.byref(path)))
        return out, path.value, _misses(self._miss_buf, min(nm.value, len(self._miss_buf)))

    def state(self):
        m = np.empty(self.experts, np.int32)
        o = np.empty(max(1, self.slots), np.int32)
        l = np.empty(max(1, self.slots), np.int32)
        _check(lib().moe_lru_get_state(self._h, m.ctypes.data, o.ctypes.data, l.ctypes.data))
        return m, o[:self.slots], l[:self.slots]

    def stats(self) -> dict:
        s = Stats()
        _check(lib().moe_lru_get_stats(self._h, C.byref(s)))
        return {f: int(getattr(s, f)) for f, _ in Stats._fields_}
