"""Thin ctypes binding of libmoe_fp4 (include/moe_fp4.h).

Argument marshalling only: torch provides device memory and streams, every
step of the layer runs in the library's CUDA kernels.  Loading fails loudly
when the library is missing; there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmoe_fp4.so")
SYNTH_PATH = os.path.join(_PKG, "lib", "libmoe_synth.so")

OK, EINVAL, ENOMEM, ECUDA, ESLOT, ETIMEOUT = 0, 1, 2, 3, 4, 5
STATUS_NAMES = {0: "OK", 1: "EINVAL", 2: "ENOMEM", 3: "ECUDA", 4: "ESLOT", 5: "ETIMEOUT"}
PATH_AUTO, PATH_GEMV, PATH_TC = 0, 1, 2
OPT_PATH, OPT_PROFILE, OPT_WAIT_LIMIT_US = 1, 2, 3

# every symbol include/moe_fp4.h declares
EXPORTS = ("moe_fp4_slot_bytes", "moe_fp4_create", "moe_fp4_destroy", "moe_fp4_arena",
           "moe_fp4_set_option", "moe_fp4_profile_read", "moe_fp4_load_expert_slot", "moe_fp4_route",
           "moe_fp4_forward", "moe_fp4_route_forward", "moe_fp4_last_error", "moe_fp4_forward_noalloc",
           "moe_fp4_saliency", "moe_fp4_stream_experts", "moe_fp4_residency_stats", "moe_fp4_expert_outputs",
           "moe_fp4_combine", "moe_fp4_linear", "moe_fp4_linear_backward")

# element types and activations of the 16-bit products (moe_fp4_linear)
BF16, F16, F32 = 0, 1, 2
_TYPES = {torch.bfloat16: BF16, torch.int16: BF16, torch.uint16: BF16, torch.float16: F16, torch.float32: F32}
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "swiglu": 4}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_layers", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32)]


class LinearArgs(ctypes.Structure):
    """moe_fp4_linear_args."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "in_features", "out_features", "type", "act", "n_groups")] + \
        [(n, ctypes.c_void_p) for n in ("offsets", "x_rows", "y_rows")] + \
        [(n, ctypes.c_int32) for n in ("x_total", "y_total")] + \
        [(n, ctypes.c_void_p) for n in ("x", "w", "w_up")] + \
        [(n, ctypes.c_int64) for n in ("ldx", "ldw", "w_group_stride")] + \
        [(n, ctypes.c_void_p) for n in ("bias", "bias_up")] + \
        [(n, ctypes.c_int32) for n in ("bias_type", "residual_type")] + \
        [("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64), ("y", ctypes.c_void_p),
         ("ldy", ctypes.c_int64), ("y_type", ctypes.c_int32), ("reserved", ctypes.c_int32),
         ("z", ctypes.c_void_p), ("z_up", ctypes.c_void_p), ("ldz", ctypes.c_int64)]


class LinearGradArgs(ctypes.Structure):
    """moe_fp4_linear_grads."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "in_features", "out_features", "type", "act", "n_groups")] + \
        [(n, ctypes.c_void_p) for n in ("offsets", "x_rows", "y_rows", "dx_rows")] + \
        [(n, ctypes.c_int32) for n in ("x_total", "y_total", "dx_total", "dy_type")] + \
        [("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("z", ctypes.c_void_p), ("z_up", ctypes.c_void_p),
         ("ldz", ctypes.c_int64)] + \
        [(n, ctypes.c_void_p) for n in ("x", "w", "w_up")] + \
        [(n, ctypes.c_int64) for n in ("ldx", "ldw", "w_group_stride")] + \
        [("dz", ctypes.c_void_p), ("dz_up", ctypes.c_void_p), ("lddz", ctypes.c_int64), ("dx", ctypes.c_void_p),
         ("lddx", ctypes.c_int64), ("dx_type", ctypes.c_int32), ("dw_type", ctypes.c_int32),
         ("dw", ctypes.c_void_p), ("dw_up", ctypes.c_void_p), ("lddw", ctypes.c_int64),
         ("dw_group_stride", ctypes.c_int64), ("db", ctypes.c_void_p), ("db_up", ctypes.c_void_p),
         ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


@dataclass
class LinearGrads:
    """What linear_backward and grouped_linear_backward return (None for what was not asked for)."""
    dx: torch.Tensor | None
    dw: torch.Tensor | None
    dw_up: torch.Tensor | None
    db: torch.Tensor | None
    db_up: torch.Tensor | None


_lib = None
_synth = None


def load(path: str = LIB_PATH):
    """Load libmoe_fp4.so (raises if it is missing: no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} not built: run python -m fp4_routed_expert_router_b200.build")
        L = ctypes.CDLL(path)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_fp4_slot_bytes.restype = SZ
        L.moe_fp4_slot_bytes.argtypes = [ctypes.POINTER(Config)]
        L.moe_fp4_create.restype = I32
        L.moe_fp4_create.argtypes = [ctypes.POINTER(Config), I32, P, SZ, ctypes.POINTER(P)]
        L.moe_fp4_destroy.restype = None
        L.moe_fp4_destroy.argtypes = [P]
        L.moe_fp4_arena.restype = P
        L.moe_fp4_arena.argtypes = [P]
        L.moe_fp4_set_option.restype = I32
        L.moe_fp4_set_option.argtypes = [P, I32, I32]
        L.moe_fp4_profile_read.restype = I32
        L.moe_fp4_profile_read.argtypes = [P, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float), I32]
        L.moe_fp4_load_expert_slot.restype = I32
        L.moe_fp4_load_expert_slot.argtypes = [P, I32, I32, I32, P, P, P, P, P, P, P]
        L.moe_fp4_route.restype = I32
        L.moe_fp4_route.argtypes = [P, I32, P, P, I32, P, P, P, P, P, P]
        L.moe_fp4_forward.restype = I32
        L.moe_fp4_forward.argtypes = [P, I32, P, I32, P, P, P, P, P, P, P, P]
        L.moe_fp4_route_forward.restype = I32
        L.moe_fp4_route_forward.argtypes = [P, I32, P, P, P, I32, P, P, P, P, P, P, P, P]
        L.moe_fp4_saliency.restype = I32
        L.moe_fp4_saliency.argtypes = [P, I32, P, P, P, P, P]
        L.moe_fp4_stream_experts.restype = I32
        L.moe_fp4_stream_experts.argtypes = [P, I32, P, I32, P, P, P]
        L.moe_fp4_residency_stats.restype = I32
        L.moe_fp4_residency_stats.argtypes = [P, P]
        L.moe_fp4_expert_outputs.restype = I32
        L.moe_fp4_expert_outputs.argtypes = [P, I32, P, I32, P, P, P]
        L.moe_fp4_combine.restype = I32
        L.moe_fp4_combine.argtypes = [P, I32, P, P, P, P, P, P]
        L.moe_fp4_last_error.restype = I32
        L.moe_fp4_last_error.argtypes = [P, ctypes.c_char_p, SZ]
        L.moe_fp4_forward_noalloc.restype = I32
        L.moe_fp4_forward_noalloc.argtypes = [ctypes.POINTER(Config), P, P, I32, P, I32, P, P, P, P, P, P, P]
        L.moe_fp4_linear.restype = I32
        L.moe_fp4_linear.argtypes = [P, ctypes.POINTER(LinearArgs), P]
        L.moe_fp4_linear_backward.restype = I32
        L.moe_fp4_linear_backward.argtypes = [P, ctypes.POINTER(LinearGradArgs), P]
        _lib = L
    return _lib


def load_synth(path: str = SYNTH_PATH):
    global _synth
    if _synth is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} not built")
        S = ctypes.CDLL(path)
        S.moe_synth_expert_bytes.restype = ctypes.c_size_t
        S.moe_synth_expert_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
        S.moe_synth_l2_discard.restype = ctypes.c_int
        S.moe_synth_l2_discard.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        S.moe_synth_fill_expert.restype = ctypes.c_int
        S.moe_synth_fill_expert.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_void_p]
        _synth = S
    return _synth


def _ptr(t) -> ctypes.c_void_p | None:
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def synth_fill_expert(dst: torch.Tensor, seed: int, layer: int, expert: int, hidden: int, inter: int,
                      scale_lo: int, scale_hi: int, stream=None) -> None:
    """Write the synthetic expert (seed, layer, expert) into ``dst`` (uint8, device)
    in checkpoint layout, bit-identical to ``synth.expert_object``."""
    rc = load_synth().moe_synth_fill_expert(_ptr(dst), seed & ((1 << 64) - 1), layer, expert, hidden, inter,
                                            scale_lo, scale_hi, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"moe_synth_fill_expert failed: cuda error {rc}")


def l2_flush(buf: torch.Tensor, value: float = 0.0, stream=None) -> None:
    """Push every earlier line out of L2 by writing ``buf`` (larger than L2),
    then drop ``buf``'s own lines without write-back: the next kernel starts
    with a cold, clean L2."""
    if stream is None:
        buf.fill_(value)
    else:
        with torch.cuda.stream(stream):
            buf.fill_(value)
    n = buf.numel() * buf.element_size() // 128 * 128
    rc = load_synth().moe_synth_l2_discard(_ptr(buf), n, _stream(stream))
    if rc != 0:
        raise RuntimeError(f"moe_synth_l2_discard failed: cuda error {rc}")


@dataclass
class Routing:
    ids: torch.Tensor       # int32 [T, k]
    weights: torch.Tensor   # fp32 [T, k]
    counts: torch.Tensor    # int32 [E]
    offsets: torch.Tensor   # int32 [E+1]
    perm: torch.Tensor      # int32 [T*k]


class Context:
    """One moe_fp4 context: arena + slot table + workspace on one device."""

    def __init__(self, hidden: int, inter: int, n_experts: int, top_k: int, n_layers: int, n_slots: int,
                 max_tokens: int, device: int = 0, arena: torch.Tensor | None = None):
        self.lib = load()
        self.cfg = Config(hidden, inter, n_experts, top_k, n_layers, n_slots, max_tokens)
        self.device = device
        self._arena_ref = arena
        h = ctypes.c_void_p()
        nbytes = arena.numel() * arena.element_size() if arena is not None else 0
        rc = self.lib.moe_fp4_create(ctypes.byref(self.cfg), device, _ptr(arena), nbytes, ctypes.byref(h))
        if rc != OK:
            raise MoeError(rc, "moe_fp4_create failed")
        self.h = h

    # ------------------------------------------------------------------ basics
    @property
    def slot_bytes(self) -> int:
        return self.lib.moe_fp4_slot_bytes(ctypes.byref(self.cfg))

    def arena_ptr(self) -> int:
        return self.lib.moe_fp4_arena(self.h)

    def close(self) -> None:
        if getattr(self, "h", None):
            self.lib.moe_fp4_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, rc: int, what: str) -> None:
        if rc != OK:
            buf = ctypes.create_string_buffer(256)
            self.lib.moe_fp4_last_error(self.h, buf, 256)
            raise MoeError(rc, f"{what}: {buf.value.decode()}")

    def last_error(self) -> tuple[int, str]:
        buf = ctypes.create_string_buffer(256)
        rc = self.lib.moe_fp4_last_error(self.h, buf, 256)
        return rc, buf.value.decode()

    def set_path(self, path: int) -> None:
        self._check(self.lib.moe_fp4_set_option(self.h, OPT_PATH, path), "set_option")

    def set_wait_limit_us(self, us: int) -> None:
        """Limit of every bounded device-side wait (0 restores the default, 1 s)."""
        self._check(self.lib.moe_fp4_set_option(self.h, OPT_WAIT_LIMIT_US, int(us)), "set_option")

    def set_profile(self, on: bool) -> None:
        self._check(self.lib.moe_fp4_set_option(self.h, OPT_PROFILE, 1 if on else 0), "set_option")

    def profile_read(self, max_records: int = 65536) -> list[tuple[str, float]]:
        """[(kernel name, device ms)] of the profiled launches since the last read."""
        names = (ctypes.c_char_p * max_records)()
        ms = (ctypes.c_float * max_records)()
        n = self.lib.moe_fp4_profile_read(self.h, names, ms, max_records)
        if n < 0:
            raise MoeError(ECUDA, "moe_fp4_profile_read failed")
        return [(names[i].decode(), float(ms[i])) for i in range(n)]

    # ------------------------------------------------------------------ calls
    def load_expert_slot(self, layer: int, expert: int, slot: int, t: dict | None, stream=None) -> None:
        """``t``: w1, s1, w3, s3, w2, s2 tensors in checkpoint layout (host or device),
        or None with slot = -1 to unmap."""
        if t is None:
            ptrs = [None] * 6
        else:
            ptrs = [ctypes.c_void_p(_data_ptr(t[n])) for n in ("w1", "s1", "w3", "s3", "w2", "s2")]
        rc = self.lib.moe_fp4_load_expert_slot(self.h, layer, expert, slot, *ptrs, _stream(stream))
        self._check(rc, "load_expert_slot")

    def load_expert_object(self, layer: int, expert: int, slot: int, obj: torch.Tensor, stream=None) -> None:
        """Load from one contiguous expert object (w1, w3, w2 codes, s1, s3, s2 scales)."""
        H, I = self.cfg.hidden, self.cfg.inter
        c13, c2, s13 = I * H // 2, H * I // 2, I * H // 32
        base = obj.data_ptr()
        offs = {"w1": 0, "w3": c13, "w2": 2 * c13, "s1": 2 * c13 + c2, "s3": 2 * c13 + c2 + s13,
                "s2": 2 * c13 + c2 + 2 * s13}
        ptrs = [ctypes.c_void_p(base + offs[n]) for n in ("w1", "s1", "w3", "s3", "w2", "s2")]
        rc = self.lib.moe_fp4_load_expert_slot(self.h, layer, expert, slot, *ptrs, _stream(stream))
        self._check(rc, "load_expert_slot")

    def alloc_routing(self, T: int) -> Routing:
        dev = torch.device("cuda", self.device)
        k, E = self.cfg.top_k, self.cfg.n_experts
        return Routing(torch.empty((T, k), dtype=torch.int32, device=dev),
                       torch.empty((T, k), dtype=torch.float32, device=dev),
                       torch.empty(E, dtype=torch.int32, device=dev),
                       torch.empty(E + 1, dtype=torch.int32, device=dev),
                       torch.empty(T * k, dtype=torch.int32, device=dev))

    def route(self, layer: int, logits: torch.Tensor, keep: torch.Tensor | None = None,
              out: Routing | None = None, stream=None) -> Routing:
        T = logits.shape[0]
        r = out if out is not None else self.alloc_routing(T)
        rc = self.lib.moe_fp4_route(self.h, layer, _ptr(logits), _ptr(keep), T, _ptr(r.ids), _ptr(r.weights),
                                    _ptr(r.counts), _ptr(r.offsets), _ptr(r.perm), _stream(stream))
        self._check(rc, "route")
        return r

    def forward(self, layer: int, x: torch.Tensor, r: Routing, y: torch.Tensor | None = None,
                x_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x: uint16/bf16 [T, H] bf16 bits.  Returns y fp32 [T, H]."""
        T = x.shape[0]
        if y is None:
            y = torch.empty((T, self.cfg.hidden), dtype=torch.float32, device=x.device)
        rc = self.lib.moe_fp4_forward(self.h, layer, _ptr(x), T, _ptr(r.ids), _ptr(r.weights), _ptr(r.counts),
                                      _ptr(r.offsets), _ptr(r.perm), _ptr(y), _ptr(x_out), _stream(stream))
        self._check(rc, "forward")
        return y

    def route_forward(self, layer: int, logits: torch.Tensor, x: torch.Tensor, keep: torch.Tensor | None = None,
                      out: Routing | None = None, y: torch.Tensor | None = None,
                      x_out: torch.Tensor | None = None, stream=None) -> tuple[Routing, torch.Tensor]:
        """Route + forward in one call (one kernel for decode batches)."""
        T = x.shape[0]
        r = out if out is not None else self.alloc_routing(T)
        if y is None:
            y = torch.empty((T, self.cfg.hidden), dtype=torch.float32, device=x.device)
        rc = self.lib.moe_fp4_route_forward(self.h, layer, _ptr(logits), _ptr(keep), _ptr(x), T, _ptr(r.ids),
                                            _ptr(r.weights), _ptr(r.counts), _ptr(r.offsets), _ptr(r.perm),
                                            _ptr(y), _ptr(x_out), _stream(stream))
        self._check(rc, "route_forward")
        return r, y

    def expert_outputs(self, layer: int, x: torch.Tensor, experts: torch.Tensor, o: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
        """o[i] = expert experts[i] applied to x[i] (fp32 [n, H]); x bf16 bits [n, H]."""
        n = x.shape[0]
        if o is None:
            o = torch.empty((n, self.cfg.hidden), dtype=torch.float32, device=x.device)
        rc = self.lib.moe_fp4_expert_outputs(self.h, layer, _ptr(x), n, _ptr(experts), _ptr(o), _stream(stream))
        self._check(rc, "expert_outputs")
        return o

    def combine(self, o: torch.Tensor, weights: torch.Tensor, x: torch.Tensor | None = None,
                y: torch.Tensor | None = None, x_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y[t] = sum_j weights[t, j] * o[t*k + j] (+ x_out = bf16(x + y))."""
        T = weights.shape[0]
        if y is None:
            y = torch.empty((T, self.cfg.hidden), dtype=torch.float32, device=o.device)
        rc = self.lib.moe_fp4_combine(self.h, T, _ptr(o), _ptr(weights), _ptr(x), _ptr(y), _ptr(x_out),
                                      _stream(stream))
        self._check(rc, "combine")
        return y

    def stream_experts(self, layer: int, experts, objects, stream=None) -> list[int]:
        """Make the listed distinct experts of ``layer`` resident (LRU slots).
        ``objects``: per expert a contiguous checkpoint-layout object (pinned
        host or device uint8 tensor, or numpy array), or None if resident.
        Returns the slot of each expert."""
        n = len(experts)
        ids = (ctypes.c_int32 * n)(*[int(e) for e in experts])
        ptrs = (ctypes.c_void_p * n)(*[(_data_ptr(o) if o is not None else None) for o in objects])
        slots = (ctypes.c_int32 * n)()
        rc = self.lib.moe_fp4_stream_experts(self.h, layer, ids, n, ptrs, slots, _stream(stream))
        self._check(rc, "stream_experts")
        return list(slots)

    def residency_stats(self) -> tuple[int, int, int]:
        """(hits, misses, bytes copied) of stream_experts since create."""
        out = (ctypes.c_int64 * 3)()
        rc = self.lib.moe_fp4_residency_stats(self.h, out)
        self._check(rc, "residency_stats")
        return out[0], out[1], out[2]

    def saliency(self, r: Routing, sal: torch.Tensor, stream=None) -> torch.Tensor:
        """Accumulate per-expert saliency (fp64 [E] device tensor) of the last
        forward on this context: sal[e] += sum of weight * ||expert output||_2
        over the entries routed to e.  Call after forward, same stream."""
        T = r.ids.shape[0]
        rc = self.lib.moe_fp4_saliency(self.h, T, _ptr(r.weights), _ptr(r.offsets), _ptr(r.perm), _ptr(sal),
                                       _stream(stream))
        self._check(rc, "saliency")
        return sal

    # ------------------------------------------------------------------ 16-bit products
    def linear(self, x: torch.Tensor, w: torch.Tensor, w_up: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, bias_up: torch.Tensor | None = None, act: str = "none",
               residual: torch.Tensor | None = None, y: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, save: bool = False, stream=None):
        """y = act(x w^T + bias) + residual for x [R, K] and w [N, K], both bf16 (or its bits) or fp16.

        act: "none", "relu", "silu", "gelu" or "swiglu" (silu(x w^T + bias) *
        (x w_up^T + bias_up)).  bias [N], residual [R, N] and y may be of
        either 16-bit type or fp32; y is x's type unless out_dtype or y says
        otherwise, and residual may be y itself.  Rows may be strided, the last
        dimension is contiguous.  save: also return z (and z_up, else None), the
        pre-activations that linear_backward takes.  Work runs on ``stream``
        (default: the current one of the context's device)."""
        return self._linear("linear", x, w, None, w_up, bias, bias_up, act, residual, y, out_dtype, save, None, None,
                            stream)

    def grouped_linear(self, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                       w_up: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                       bias_up: torch.Tensor | None = None, act: str = "none",
                       residual: torch.Tensor | None = None, x_rows: torch.Tensor | None = None,
                       y_rows: torch.Tensor | None = None, y: torch.Tensor | None = None,
                       out_dtype: torch.dtype | None = None, save: bool = False, stream=None):
        """linear with a weight per group: w [E, N, K], bias [E, N]; rows offsets[e] .. offsets[e+1]
        (int32 [E+1] on the device, as Routing.offsets) take weight e.

        x_rows (int32 [R]): row i reads x[x_rows[i]], e.g. Routing.perm // k.
        y_rows (int32 [R], distinct): row i goes to y[y_rows[i]] (and takes
        residual[y_rows[i]]), e.g. Routing.perm for rows in entry order.  Rows
        of y outside every group are left as they were; z is in grouped order."""
        return self._linear("grouped_linear", x, w, offsets, w_up, bias, bias_up, act, residual, y, out_dtype, save,
                            x_rows, y_rows, stream)

    def _linear(self, what, x, w, offsets, w_up, bias, bias_up, act, residual, y, out_dtype, save, x_rows, y_rows,
                stream):
        chk = _Check(self, what)
        E, N, K, wdt = chk.weights(w, offsets, w_up)
        R = chk.rows(x, x_rows, K, wdt)
        lead = () if offsets is None else (E,)
        y_total = R if y_rows is None else (y.shape[0] if y is not None else
                                            (residual.shape[0] if residual is not None else R))
        act_id = chk.act(act, w_up)
        a = LinearArgs(rows=R, in_features=K, out_features=N, type=wdt, act=act_id,
                       n_groups=0 if offsets is None else E, x_total=x.shape[0], y_total=y_total)
        a.offsets, a.x_rows, a.y_rows = _addr(offsets), chk.index(x_rows, "x_rows", R), chk.index(y_rows, "y_rows", R)
        a.x, a.ldx = chk.matrix(x, "x", (x.shape[0], K), (wdt,))
        a.w, a.ldw, a.w_group_stride = chk.weight_layout(w)
        if w_up is not None:
            if chk.weight_layout(w_up)[1:] != (a.ldw, a.w_group_stride):
                chk.fail("w and w_up differ in their strides")
            a.w_up = w_up.data_ptr()
        for t, name in ((bias, "bias"), (bias_up, "bias_up")):
            if t is not None:
                setattr(a, name, chk.dense(t, name, lead + (N,)))
                if bias is not None and t.dtype != bias.dtype:
                    chk.fail("bias and bias_up differ in type")
                a.bias_type = _TYPES[t.dtype]
        if residual is not None:
            a.residual, a.ld_residual = chk.matrix(residual, "residual", (y_total, N))
            a.residual_type = _TYPES[residual.dtype]
        with chk.on(stream) as s:
            if y is None:
                y = torch.empty((y_total, N), dtype=out_dtype or chk.plain(x.dtype), device=x.device)
            a.y, a.ldy = chk.matrix(y, "y", (y_total, N))
            a.y_type = _TYPES[y.dtype]
            z = z_up = None
            if save:
                z = torch.empty((R, N), dtype=chk.plain(x.dtype), device=x.device)
                z_up = torch.empty_like(z) if w_up is not None else None
                a.z, a.z_up, a.ldz = _addr(z), _addr(z_up), N
            chk.keep(s, x, w, w_up, offsets, bias, bias_up, residual, x_rows, y_rows, y, z, z_up)
            self._check(self.lib.moe_fp4_linear(self.h, ctypes.byref(a), ctypes.c_void_p(s.cuda_stream)), what)
        return (y, z, z_up) if save else y

    def linear_backward(self, dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, w_up: torch.Tensor | None = None,
                        z: torch.Tensor | None = None, z_up: torch.Tensor | None = None, act: str = "none",
                        need_dx: bool = True, need_dw: bool = True, need_db: bool = False,
                        dx: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                        dw_up: torch.Tensor | None = None, db: torch.Tensor | None = None,
                        db_up: torch.Tensor | None = None, dw_dtype: torch.dtype | None = None,
                        accumulate: bool = False, stream=None) -> LinearGrads:
        """Gradients of ``linear`` (the residual's is dy itself): dz = dy act'(z), dx = dz w (+ dz_up w_up),
        dw = dz^T x, db = sum of dz (fp32).

        dy [R, N] has x's type or fp32; z (and z_up) are what linear(save=True)
        returned.  dz is rounded to x's type for the products.  dx, dw, dw_up,
        db, db_up may be given as outputs (dx and dw of any of the three
        types); accumulate adds to the given dw and db instead of overwriting
        them (micro-batches)."""
        return self._linear_backward("linear_backward", dy, x, w, None, w_up, z, z_up, act, need_dx, need_dw, need_db,
                                     dx, dw, dw_up, db, db_up, dw_dtype, accumulate, None, None, None, stream)

    def grouped_linear_backward(self, dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                                w_up: torch.Tensor | None = None, z: torch.Tensor | None = None,
                                z_up: torch.Tensor | None = None, act: str = "none",
                                x_rows: torch.Tensor | None = None, y_rows: torch.Tensor | None = None,
                                dx_rows: torch.Tensor | None = None, need_dx: bool = True, need_dw: bool = True,
                                need_db: bool = False, dx: torch.Tensor | None = None,
                                dw: torch.Tensor | None = None, dw_up: torch.Tensor | None = None,
                                db: torch.Tensor | None = None, db_up: torch.Tensor | None = None,
                                dw_dtype: torch.dtype | None = None, accumulate: bool = False,
                                stream=None) -> LinearGrads:
        """Gradients of ``grouped_linear``, dw and db per group (zero for an empty one).

        x and dy are read through x_rows and y_rows as in the forward; dx has a
        row per grouped row, at dx_rows[i] (int32 [R], distinct) when given, else
        at i.  With dx_rows = Routing.perm and an fp32 dx, ``combine`` with
        weights of one sums the k rows of each token."""
        return self._linear_backward("grouped_linear_backward", dy, x, w, offsets, w_up, z, z_up, act, need_dx,
                                     need_dw, need_db, dx, dw, dw_up, db, db_up, dw_dtype, accumulate, x_rows, y_rows,
                                     dx_rows, stream)

    def _linear_backward(self, what, dy, x, w, offsets, w_up, z, z_up, act, need_dx, need_dw, need_db, dx, dw, dw_up,
                         db, db_up, dw_dtype, accumulate, x_rows, y_rows, dx_rows, stream) -> LinearGrads:
        chk = _Check(self, what)
        E, N, K, wdt = chk.weights(w, offsets, w_up)
        R = chk.rows(x, x_rows, K, wdt)
        lead = () if offsets is None else (E,)
        two = w_up is not None
        act_id = chk.act(act, w_up)
        if act_id and z is None or two and z_up is None:
            chk.fail("z (and z_up) of the forward pass are needed")
        if not two and any(t is not None for t in (z_up, dw_up, db_up)):
            chk.fail("z_up, dw_up and db_up go with w_up")
        if (not need_dx and dx is not None) or (not need_dw and (dw is not None or dw_up is not None)) or \
                (not need_db and (db is not None or db_up is not None)):
            chk.fail("an output was given for a gradient that is not needed")
        if accumulate and ((need_dw and (dw is None or two and dw_up is None)) or
                           (need_db and (db is None or two and db_up is None))):
            chk.fail("accumulate adds to given outputs")
        dy_total = R if y_rows is None else dy.shape[0]
        dx_total = R if dx_rows is None else (dx.shape[0] if dx is not None else R)
        a = LinearGradArgs(rows=R, in_features=K, out_features=N, type=wdt, act=act_id,
                           n_groups=0 if offsets is None else E, x_total=x.shape[0], y_total=dy_total,
                           dx_total=dx_total, accumulate=int(accumulate))
        a.offsets, a.x_rows = _addr(offsets), chk.index(x_rows, "x_rows", R)
        a.y_rows, a.dx_rows = chk.index(y_rows, "y_rows", R), chk.index(dx_rows, "dx_rows", R)
        a.dy, a.lddy = chk.matrix(dy, "dy", (dy_total, N), (wdt, F32))
        a.dy_type = _TYPES[dy.dtype]
        a.x, a.ldx = chk.matrix(x, "x", (x.shape[0], K), (wdt,))
        a.w, a.ldw, a.w_group_stride = chk.weight_layout(w)
        if two:
            if chk.weight_layout(w_up)[1:] != (a.ldw, a.w_group_stride):
                chk.fail("w and w_up differ in their strides")
            a.w_up = w_up.data_ptr()
        if act_id:
            a.z, a.ldz = chk.matrix(z, "z", (R, N), (wdt,))
            if two:
                a.z_up, ld_up = chk.matrix(z_up, "z_up", (R, N), (wdt,))
                if ld_up != a.ldz:
                    chk.fail("z and z_up differ in their strides")
        t16 = chk.plain(x.dtype)
        with chk.on(stream) as s:
            def new(shape, dtype):
                return torch.empty(shape, dtype=dtype, device=x.device)

            dz = dz_up = None
            if (act_id or _TYPES[dy.dtype] == F32 or y_rows is not None) and (need_dx or need_dw):
                dz = new((R, N), t16)
                dz_up = new((R, N), t16) if two else None
                a.dz, a.dz_up, a.lddz = _addr(dz), _addr(dz_up), N
            if need_dx:
                dx = new((dx_total, K), t16) if dx is None else dx
                a.dx, a.lddx = chk.matrix(dx, "dx", (dx_total, K))
                a.dx_type = _TYPES[dx.dtype]
            if need_dw:
                dw = new(lead + (N, K), dw_dtype or t16) if dw is None else dw
                a.dw, a.lddw, a.dw_group_stride = chk.grad_layout(dw, "dw", lead + (N, K))
                a.dw_type = _TYPES[dw.dtype]
                if two:
                    dw_up = torch.empty_like(dw) if dw_up is None else dw_up
                    if dw_up.dtype != dw.dtype or \
                            chk.grad_layout(dw_up, "dw_up", lead + (N, K))[1:] != (a.lddw, a.dw_group_stride):
                        chk.fail("dw and dw_up differ in type or strides")
                    a.dw_up = dw_up.data_ptr()
            if need_db:
                db = new(lead + (N,), torch.float32) if db is None else db
                a.db = chk.dense(db, "db", lead + (N,), (F32,))
                if two:
                    db_up = torch.empty_like(db) if db_up is None else db_up
                    a.db_up = chk.dense(db_up, "db_up", lead + (N,), (F32,))
            chk.keep(s, dy, x, w, w_up, offsets, z, z_up, x_rows, y_rows, dx_rows, dz, dz_up, dx, dw, dw_up, db,
                     db_up)
            self._check(self.lib.moe_fp4_linear_backward(self.h, ctypes.byref(a), ctypes.c_void_p(s.cuda_stream)),
                        what)
        return LinearGrads(dx, dw, dw_up, db, db_up)


def _addr(t):
    return None if t is None else t.data_ptr()


class _Check:
    """Argument checks of the 16-bit products: what the C call cannot see (devices, shapes, tensor types)."""

    def __init__(self, ctx: Context, what: str):
        self.ctx, self.what = ctx, what

    def fail(self, why: str):
        raise MoeError(EINVAL, f"{self.what}: {why}")

    def tensor(self, t, name: str, types=(BF16, F16, F32)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda" or t.device.index != self.ctx.device:
            self.fail(f"{name} is not a tensor on the context's device {self.ctx.device}")
        if t.dtype not in _TYPES or _TYPES[t.dtype] not in types:
            self.fail(f"{name} has type {t.dtype}")

    def matrix(self, t, name: str, shape, types=(BF16, F16, F32)):
        """(address, row stride) of a 2-D tensor with contiguous rows."""
        self.tensor(t, name, types)
        if tuple(t.shape) != tuple(shape):
            self.fail(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if t.shape[1] > 1 and t.stride(1) != 1:
            self.fail(f"{name} needs a contiguous last dimension")
        ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
        if ld < t.shape[1]:
            self.fail(f"{name}'s rows overlap")
        return t.data_ptr(), ld

    def dense(self, t, name: str, shape, types=(BF16, F16, F32)):
        self.tensor(t, name, types)
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            self.fail(f"{name} has to be a contiguous tensor of shape {tuple(shape)}")
        return t.data_ptr()

    def grad_layout(self, t, name: str, shape, types=(BF16, F16, F32)):
        """(address, row stride, group stride) of [N, K] or [E, N, K] with contiguous rows."""
        self.tensor(t, name, types)
        if tuple(t.shape) != tuple(shape):
            self.fail(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        if shape[-1] > 1 and t.stride(-1) != 1:
            self.fail(f"{name} needs a contiguous last dimension")
        ld = t.stride(-2) if shape[-2] > 1 else shape[-1]
        gs = t.stride(0) if len(shape) == 3 and shape[0] > 1 else shape[-2] * ld
        if ld < shape[-1] or (len(shape) == 3 and gs < (shape[-2] - 1) * ld + shape[-1]):
            self.fail(f"{name}'s rows overlap")
        return t.data_ptr(), ld, gs

    def weight_layout(self, w):
        return self.grad_layout(w, "w", tuple(w.shape))

    def weights(self, w, offsets, w_up):
        self.tensor(w, "w", (BF16, F16))
        want = 2 if offsets is None else 3
        if w.dim() != want or min(w.shape) < 1:
            self.fail(f"w has shape {tuple(w.shape)}, not {want} dimensions of one or more")
        if w_up is not None:
            self.tensor(w_up, "w_up", (_TYPES[w.dtype],))
            if w_up.shape != w.shape:
                self.fail("w and w_up differ in shape")
        E = 1
        if offsets is not None:
            E = w.shape[0]
            if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or \
                    tuple(offsets.shape) != (E + 1,) or not offsets.is_contiguous() or \
                    offsets.device != w.device:
                self.fail(f"offsets has to be a contiguous int32 [{E + 1}] on w's device")
        return E, w.shape[-2], w.shape[-1], _TYPES[w.dtype]

    def rows(self, x, x_rows, K, wdt):
        self.tensor(x, "x", (wdt,))
        if x.dim() != 2 or x.shape[1] != K:
            self.fail(f"x has shape {tuple(x.shape)}, not [rows, {K}]")
        return x.shape[0] if x_rows is None else x_rows.numel()

    def act(self, act, w_up):
        if act not in ACTS:
            self.fail(f"act {act!r} is not one of {', '.join(ACTS)}")
        if (act == "swiglu") != (w_up is not None):
            self.fail("w_up goes with act='swiglu'")
        return ACTS[act]

    def index(self, t, name: str, n: int):
        if t is None:
            return None
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or tuple(t.shape) != (n,) or \
                not t.is_contiguous() or t.device.type != "cuda" or t.device.index != self.ctx.device:
            self.fail(f"{name} has to be a contiguous int32 [{n}] on the context's device")
        return t.data_ptr()

    @staticmethod
    def plain(dtype):
        """The float type of a tensor that may hold bf16 bits."""
        return torch.bfloat16 if dtype in (torch.int16, torch.uint16) else dtype

    @contextlib.contextmanager
    def on(self, stream):
        """The context's device and the call's stream, so that outputs are allocated for that stream."""
        with torch.cuda.device(self.ctx.device):
            self.home = torch.cuda.current_stream()
            s = stream if stream is not None else self.home
            with torch.cuda.stream(s):
                yield s

    def keep(self, s, *tensors):
        """Tell the allocator of tensors used on another stream than the current one, so that memory a caller
        frees right after the call is not given away before the work is done."""
        if s == self.home or torch.cuda.is_current_stream_capturing():
            return
        for t in tensors:
            if t is not None:
                t.record_stream(s)


def _data_ptr(t) -> int:
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return t.ctypes.data   # numpy array (host memory)


def forward_noalloc(cfg: Config, arena_ptr: int, slot_table: torch.Tensor, layer: int, x: torch.Tensor,
                    r: Routing, y: torch.Tensor, x_out: torch.Tensor | None = None,
                    err: torch.Tensor | None = None, stream=None) -> int:
    """moe_fp4_forward_noalloc: the decode forward with library-owned static
    scratch, for callers that may not allocate device memory.  Returns the
    status code (EINVAL when T exceeds the scratch limit)."""
    return load().moe_fp4_forward_noalloc(ctypes.byref(cfg), ctypes.c_void_p(arena_ptr), _ptr(slot_table), layer,
                                          _ptr(x), x.shape[0], _ptr(r.weights), _ptr(r.offsets), _ptr(r.perm),
                                          _ptr(y), _ptr(x_out), _ptr(err), _stream(stream))
