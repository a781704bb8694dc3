"""Python binding of liblmoe.so, the B200 Stable-LatentMoE layer with Quantile Balancing.

Argument marshalling only: every step of the layer runs in the CUDA kernels behind the C ABI
(include/lmoe.h).  torch supplies device memory and streams.  If the library is not built the
import of the binding still works, but the first call raises: there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from ctypes import POINTER, c_float, c_int, c_int32, c_size_t, c_uint32, c_void_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblmoe.so")

F32, BF16 = 0, 1
EXPERTS_BF16, EXPERTS_MXFP8, EXPERTS_MXFP4 = 0, 1, 4
RECORD_STATS = 1
UPDATE_BIAS = 4
ASYNC_OUTPUT = 8
QB_LITERAL = 1
BIAS_SIGN = 2
MX4_SWIGLU = 1
MX4_ZERO_REST = 2
STATUS_NAN_SCORE, STATUS_WATCHDOG, STATUS_BAD_INDEX = 1, 2, 4
NBINS = 4096

EXPORTED = (
    "lmoe_create", "lmoe_destroy", "lmoe_workspace_bytes", "lmoe_forward", "lmoe_forward_host", "lmoe_host_wait",
    "lmoe_qb_update", "lmoe_set_update", "lmoe_route_scores", "lmoe_get_routing", "lmoe_get_bias", "lmoe_set_bias",
    "lmoe_get_hist", "lmoe_set_hist", "lmoe_get_load", "lmoe_set_load", "lmoe_get_status", "lmoe_strerror", "lmoe_gemm_bf16",
    "lmoe_profile_enable", "lmoe_profile_read", "lmoe_stage_name", "lmoe_launch_count",
    "lmoe_route_noalloc", "lmoe_watchdog_selftest", "lmoe_gemm_bf16_ex", "lmoe_forward_backward",
    "lmoe_mx4_bytes", "lmoe_mx4_quant", "lmoe_mx4_quant_w13", "lmoe_mx4_dequant", "lmoe_mx4_gemm",
    "lmoe_balance_scratch_bytes", "lmoe_balance_loss", "lmoe_set_balance", "lmoe_set_balance_total",
    "lmoe_get_balance",
)
NUM_STAGES = 14


class LmoeError(RuntimeError):
    pass


class lmoe_config(ctypes.Structure):
    _fields_ = [("d", c_int32), ("l", c_int32), ("E", c_int32), ("k", c_int32), ("h", c_int32),
                ("hs", c_int32), ("dtype", c_int32), ("nbins", c_int32), ("rms_eps", c_float),
                ("max_tokens", c_int32), ("experts", c_int32)]


class lmoe_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("rms_gain", "w_down", "w_router", "router_bias", "w1", "w3",
                                         "w2", "w_up", "ws1", "ws3", "ws2")]


class lmoe_grads(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("dx", "rms_gain", "w_down", "w_router", "router_bias", "w1", "w3", "w2",
                                         "w_up", "ws1", "ws3", "ws2")]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LmoeError(f"{LIB_PATH} is missing: build it with `python -m latent_routing_quantile_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, i64 = c_void_p, c_int32, c_uint32, ctypes.c_int64
        sig = {
            "lmoe_create": [POINTER(lmoe_config), POINTER(lmoe_weights), vp, POINTER(vp)],
            "lmoe_destroy": [vp],
            "lmoe_workspace_bytes": [POINTER(lmoe_config), POINTER(c_size_t)],
            "lmoe_forward": [vp, vp, vp, i32, u32, vp],
            "lmoe_forward_host": [vp, vp, vp, i32, u32, vp],
            "lmoe_host_wait": [vp, vp],
            "lmoe_qb_update": [vp, c_float, u32, vp],
            "lmoe_set_update": [vp, c_float, u32],
            "lmoe_route_scores": [vp, vp, i32, u32, vp],
            "lmoe_get_routing": [vp, vp, vp, vp, vp, vp, vp, vp, vp],
            "lmoe_get_bias": [vp, vp, vp],
            "lmoe_set_bias": [vp, vp, vp],
            "lmoe_get_hist": [vp, vp, vp, vp],
            "lmoe_set_hist": [vp, vp, vp, vp],
            "lmoe_get_load": [vp, vp, vp],
            "lmoe_set_load": [vp, vp, vp],
            "lmoe_get_status": [vp, POINTER(u32)],
            "lmoe_gemm_bf16": [vp, vp, vp, i32, i32, i32, vp],
            "lmoe_gemm_bf16_ex": [vp, i32, vp, i32, vp, i32, i32, i32, i32, vp],
            "lmoe_forward_backward": [vp, POINTER(lmoe_weights), vp, vp, vp, i32, u32, POINTER(lmoe_grads), vp],
            "lmoe_profile_enable": [vp, i32],
            "lmoe_profile_read": [vp, POINTER(c_float), i32, POINTER(i32)],
            "lmoe_launch_count": [vp, POINTER(ctypes.c_int64)],
            "lmoe_route_noalloc": [vp, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp],
            "lmoe_watchdog_selftest": [vp, i32, vp],
            "lmoe_mx4_bytes": [i64, i32, i32, i32, POINTER(c_size_t), POINTER(c_size_t)],
            "lmoe_mx4_quant": [vp, i32, i64, vp, i64, i64, i32, i32, vp, vp, vp, vp, vp],
            "lmoe_mx4_quant_w13": [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp],
            "lmoe_mx4_dequant": [vp, vp, i64, i32, i32, vp, vp, i32, i64, u32, vp, vp],
            "lmoe_mx4_gemm": [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, i64, u32, vp, vp],
            "lmoe_balance_scratch_bytes": [POINTER(c_size_t)],
            "lmoe_set_balance": [vp, c_float, vp, i32],
            "lmoe_set_balance_total": [vp, vp, vp],
            "lmoe_get_balance": [vp, vp, vp, vp],
            "lmoe_balance_loss": [vp, vp, i32, i32, i32, vp, i32, c_float, vp, vp, vp, vp, vp, vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = c_int
        L.lmoe_strerror.argtypes = [c_int]
        L.lmoe_strerror.restype = ctypes.c_char_p
        L.lmoe_stage_name.argtypes = [c_int32]
        L.lmoe_stage_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        raise LmoeError(f"{what}: {lib().lmoe_strerror(rc).decode()} ({rc})")


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype=None, shape=None, name="tensor"):
    if not t.is_cuda or not t.is_contiguous():
        raise LmoeError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise LmoeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise LmoeError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


class Layer:
    """One LatentMoE layer handle (lmoe_create ... lmoe_destroy).

    weights: dict of CUDA tensors named as in lmoe_weights (rms_gain, w_down, w_router,
    router_bias, w1, w3, w2, w_up, ws1, ws3, ws2), layouts (out, in).
    """

    def __init__(self, d, l, E, k, h, hs, dtype, max_tokens, weights, rms_eps=1e-6, stream=None,
                 experts=EXPERTS_BF16):
        self.cfg = lmoe_config(d, l, E, k, h, hs, dtype, NBINS, rms_eps, max_tokens, experts)
        self.dtype = torch.float32 if dtype == F32 else torch.bfloat16
        dt = self.dtype
        shapes = {"rms_gain": ((d,), dt), "w_down": ((l, d), dt), "w_router": ((E, l), torch.float32),
                  "router_bias": ((E,), torch.float32), "w1": ((E, h, l), dt), "w3": ((E, h, l), dt),
                  "w2": ((E, l, h), dt), "w_up": ((d, l), dt)}
        if hs:
            shapes.update({"ws1": ((hs, d), dt), "ws3": ((hs, d), dt), "ws2": ((d, hs), dt)})
        w = lmoe_weights()
        for name, (shape, tdt) in shapes.items():
            t = weights.get(name)
            if t is not None:
                _dev(t, tdt, shape, name)
                setattr(w, name, t.data_ptr())
        self._keep = dict(weights)
        self.handle = c_void_p()
        _check(lib().lmoe_create(ctypes.byref(self.cfg), ctypes.byref(w), _stream(stream),
                                 ctypes.byref(self.handle)), "lmoe_create")
        (torch.cuda.current_stream() if stream is None else stream).synchronize()
        self._keep = None
        self._balance = None  # (bounds, sequences) of the balance loss while it is on
        self.last_T = 0

    # ---------------------------------------------------------------- forward
    @staticmethod
    def _fwd_flags(record_stats, update_bias):
        # update_bias records this forward's statistics too (the update counts them)
        return (RECORD_STATS if (record_stats or update_bias) else 0) | (UPDATE_BIAS if update_bias else 0)

    def forward(self, x, y=None, record_stats=False, update_bias=False, stream=None):
        """update_bias=True also runs the bias update set by set_update inside this forward."""
        T = x.shape[0]
        _dev(x, self.dtype, (T, self.cfg.d), "x")
        if y is None:
            y = torch.empty_like(x)
        _dev(y, self.dtype, (T, self.cfg.d), "y")
        _check(lib().lmoe_forward(self.handle, _ptr(x), _ptr(y), T, self._fwd_flags(record_stats, update_bias),
                                  _stream(stream)), "lmoe_forward")
        self.last_T = T
        return y

    GRAD_NAMES = ("x", "rms_gain", "w_down", "w_router", "router_bias", "w1", "w3", "w2", "w_up", "ws1", "ws3",
                  "ws2")

    def forward_backward(self, x, dy, weights, y=None, record_stats=False, grads=None, stream=None):
        """One training step's layer work (lmoe_forward_backward): y = forward(x) and the fp32
        gradients of sum(y * dy) with respect to x and every weight, returned as a dict keyed like
        the weights (plus "x").  `weights` are the device tensors the layer was created from.
        `grads` may pass preallocated fp32 buffers."""
        c = self.cfg
        T = x.shape[0]
        _dev(x, self.dtype, (T, c.d), "x")
        _dev(dy, self.dtype, (T, c.d), "dy")
        if y is None:
            y = torch.empty_like(x)
        _dev(y, self.dtype, (T, c.d), "y")
        shapes = {"x": (T, c.d), "rms_gain": (c.d,), "w_down": (c.l, c.d), "w_router": (c.E, c.l),
                  "router_bias": (c.E,), "w1": (c.E, c.h, c.l), "w3": (c.E, c.h, c.l), "w2": (c.E, c.l, c.h),
                  "w_up": (c.d, c.l)}
        if c.hs:
            shapes.update({"ws1": (c.hs, c.d), "ws3": (c.hs, c.d), "ws2": (c.d, c.hs)})
        g = dict(grads or {})
        for n, shp in shapes.items():
            if n not in g:
                g[n] = torch.empty(shp, dtype=torch.float32, device=x.device)
            _dev(g[n], torch.float32, shp, "grad " + n)
        w = lmoe_weights()
        for n in ("rms_gain", "w_down", "w_router", "router_bias", "w1", "w3", "w2", "w_up", "ws1", "ws3", "ws2"):
            t = weights.get(n)
            if t is not None:
                setattr(w, n, _dev(t, None, None, n).data_ptr())
        gs = lmoe_grads()
        for n in shapes:
            setattr(gs, "dx" if n == "x" else n, g[n].data_ptr())
        _check(lib().lmoe_forward_backward(self.handle, ctypes.byref(w), _ptr(x), _ptr(dy), _ptr(y), T,
                                           self._fwd_flags(record_stats, False), ctypes.byref(gs), _stream(stream)),
               "lmoe_forward_backward")
        self.last_T = T
        return y, g

    def forward_host(self, x_host, y_host, record_stats=False, update_bias=False, async_output=False,
                     stream=None):
        """Host tensors (pinned for asynchronous copies); y_host is valid after the stream syncs,
        or with async_output=True after host_wait() and a sync of that stream."""
        T = x_host.shape[0]
        if x_host.is_cuda or y_host.is_cuda or x_host.dtype != self.dtype or y_host.dtype != self.dtype:
            raise LmoeError("forward_host takes host tensors of the layer dtype")
        _check(lib().lmoe_forward_host(self.handle, c_void_p(x_host.data_ptr()), c_void_p(y_host.data_ptr()), T,
                                       self._fwd_flags(record_stats, update_bias) | (ASYNC_OUTPUT if async_output else 0),
                                       _stream(stream)),
               "lmoe_forward_host")
        self.last_T = T
        return y_host

    def host_wait(self, stream=None):
        """Makes the stream wait for every async_output copy enqueued so far."""
        _check(lib().lmoe_host_wait(self.handle, _stream(stream)), "lmoe_host_wait")

    def route_scores(self, scores, record_stats=False, stream=None):
        T = scores.shape[0]
        _dev(scores, torch.float32, (T, self.cfg.E), "scores")
        _check(lib().lmoe_route_scores(self.handle, _ptr(scores), T, RECORD_STATS if record_stats else 0,
                                       _stream(stream)), "lmoe_route_scores")
        self.last_T = T

    def qb_update(self, beta, literal=False, sign_rule=False, stream=None):
        """Bias update from the recorded statistics: Quantile Balancing, or with sign_rule=True the
        aux-loss-free rule b_e += beta * sign(mean load - load_e)."""
        flags = (QB_LITERAL if literal else 0) | (BIAS_SIGN if sign_rule else 0)
        _check(lib().lmoe_qb_update(self.handle, float(beta), flags, _stream(stream)), "lmoe_qb_update")

    def set_update(self, beta, literal=False, sign_rule=False):
        """Step and rule of the update that forward(..., update_bias=True) runs after its routing."""
        flags = (QB_LITERAL if literal else 0) | (BIAS_SIGN if sign_rule else 0)
        _check(lib().lmoe_set_update(self.handle, float(beta), flags), "lmoe_set_update")

    def set_balance(self, coef, cu_seqlens=None):
        """The router's balance loss in every later forward_backward (weight coef; 0 takes it out), sequence
        by sequence for bounds cu_seqlens (int32 [S + 1] on the device, read at each step; None: the
        step's tokens are one sequence).  The loss is a mean over the step's own sequences; dp_train_step
        makes it one over all ranks'."""
        S = 1
        if cu_seqlens is not None:
            S = _offsets(cu_seqlens, "cu_seqlens").numel() - 1
            if S > _INT_MAX:
                _too_large(S=S)
            _dev(cu_seqlens, name="cu_seqlens")
        _check(lib().lmoe_set_balance(self.handle, float(coef), _ptr(cu_seqlens), S), "lmoe_set_balance")
        # the bounds stay alive as long as the steps read them
        self._balance = (cu_seqlens, S) if float(coef) != 0 else None

    def balance_sequences(self, T):
        """Sequences with tokens of a training step of T tokens (int32 [1] on the bounds' device), None while
        the balance loss is off."""
        if self._balance is None:
            return None
        cu, _ = self._balance
        if cu is None:
            return torch.full((1,), int(T > 0), dtype=torch.int32, device="cuda")
        return (cu[1:] > cu[:-1]).sum(dtype=torch.int32).view(1)

    def set_balance_total(self, total=None, stream=None):
        """The number of sequences (int32 [1] on the device, copied) that the balance loss of later steps is a
        mean over: those of all ranks.  None: each step's own again."""
        if total is not None:
            _dev(total, torch.int32, (1,), "total")
        _check(lib().lmoe_set_balance_total(self.handle, _ptr(total), _stream(stream)), "lmoe_set_balance_total")
        if total is not None and stream is not None:
            total.record_stream(stream)

    def balance(self, stream=None):
        """(loss [1], counts [S, E]) of the last training step since set_balance; zeros before the first."""
        S = 1 if self._balance is None else self._balance[1]
        with _current(stream):  # the results belong to the stream that writes them
            loss = torch.empty(1, dtype=torch.float32, device="cuda")
            counts = torch.empty((S, self.cfg.E), dtype=torch.int32, device="cuda")
        _check(lib().lmoe_get_balance(self.handle, _ptr(loss), _ptr(counts), _stream(stream)), "lmoe_get_balance")
        return loss, counts

    # ---------------------------------------------------------------- introspection
    def routing(self, stream=None):
        T, k, E = self.last_T, self.cfg.k, self.cfg.E
        dev = torch.device("cuda")
        out = dict(idx=torch.empty((T, k), dtype=torch.int32, device=dev),
                   gates=torch.empty((T, k), dtype=torch.float32, device=dev),
                   scores=torch.empty((T, E), dtype=torch.float32, device=dev),
                   counts=torch.empty(E, dtype=torch.int32, device=dev),
                   offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm=torch.empty(T * k, dtype=torch.int32, device=dev),
                   inv=torch.empty(T * k, dtype=torch.int32, device=dev))
        _check(lib().lmoe_get_routing(self.handle, *(_ptr(out[n]) for n in
                                                     ("idx", "gates", "scores", "counts", "offsets", "perm", "inv")),
                                      _stream(stream)), "lmoe_get_routing")
        return out

    def bias(self, stream=None):
        b = torch.empty(self.cfg.E, dtype=torch.float32, device="cuda")
        _check(lib().lmoe_get_bias(self.handle, _ptr(b), _stream(stream)), "lmoe_get_bias")
        return b

    def set_bias(self, b, stream=None):
        _dev(b, torch.float32, (self.cfg.E,), "b")
        _check(lib().lmoe_set_bias(self.handle, _ptr(b), _stream(stream)), "lmoe_set_bias")

    def hist(self, stream=None):
        hist = torch.empty((self.cfg.E, NBINS), dtype=torch.int32, device="cuda")
        n = torch.empty(1, dtype=torch.int64, device="cuda")
        _check(lib().lmoe_get_hist(self.handle, _ptr(hist), _ptr(n), _stream(stream)), "lmoe_get_hist")
        return hist, n

    def set_hist(self, hist, ntok, stream=None):
        _dev(hist, torch.int32, (self.cfg.E, NBINS), "hist")
        _dev(ntok, torch.int64, (1,), "ntok")
        _check(lib().lmoe_set_hist(self.handle, _ptr(hist), _ptr(ntok), _stream(stream)), "lmoe_set_hist")

    def load(self, stream=None):
        load = torch.empty(self.cfg.E, dtype=torch.int64, device="cuda")
        _check(lib().lmoe_get_load(self.handle, _ptr(load), _stream(stream)), "lmoe_get_load")
        return load

    def set_load(self, load, stream=None):
        _dev(load, torch.int64, (self.cfg.E,), "load")
        _check(lib().lmoe_set_load(self.handle, _ptr(load), _stream(stream)), "lmoe_set_load")

    def profile(self, enable: bool = True):
        _check(lib().lmoe_profile_enable(self.handle, 1 if enable else 0), "lmoe_profile_enable")

    def profile_read(self):
        """(per-stage milliseconds summed over the recorded calls, number of recorded forwards)."""
        ms = (c_float * NUM_STAGES)()
        calls = c_int32(0)
        _check(lib().lmoe_profile_read(self.handle, ms, NUM_STAGES, ctypes.byref(calls)), "lmoe_profile_read")
        return {stage_name(i): ms[i] for i in range(NUM_STAGES)}, calls.value

    def launches(self) -> int:
        n = ctypes.c_int64(0)
        _check(lib().lmoe_launch_count(self.handle, ctypes.byref(n)), "lmoe_launch_count")
        return n.value

    def status(self) -> int:
        v = c_uint32(0)
        _check(lib().lmoe_get_status(self.handle, ctypes.byref(v)), "lmoe_get_status")
        return v.value

    def close(self):
        if self.handle:
            _check(lib().lmoe_destroy(self.handle), "lmoe_destroy")
            self.handle = c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def watchdog_selftest(limit_us: int = 20000, stream=None) -> int:
    """Runs the bounded-wait check (a wait on a barrier nothing completes) and returns the status word."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(lib().lmoe_watchdog_selftest(_ptr(st), int(limit_us), _stream(stream)), "lmoe_watchdog_selftest")
    torch.cuda.synchronize()
    return int(st.item()) & 0xffffffff


def stage_name(i: int) -> str:
    return lib().lmoe_stage_name(i).decode()


def workspace_bytes(d, l, E, k, h, hs, dtype, max_tokens, rms_eps=1e-6, experts=EXPERTS_BF16) -> int:
    cfg = lmoe_config(d, l, E, k, h, hs, dtype, NBINS, rms_eps, max_tokens, experts)
    n = c_size_t(0)
    _check(lib().lmoe_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)), "lmoe_workspace_bytes")
    return n.value


def gemm_bf16(a, b, stream=None):
    """C = A B^T on the tensor-core engine (fp32 result), for checks of the engine itself."""
    M, K = a.shape
    N = b.shape[0]
    _dev(a, torch.bfloat16, (M, K), "a")
    _dev(b, torch.bfloat16, (N, K), "b")
    c = torch.empty((M, N), dtype=torch.float32, device=a.device)
    _check(lib().lmoe_gemm_bf16(_ptr(a), _ptr(b), _ptr(c), M, N, K, _stream(stream)), "lmoe_gemm_bf16")
    return c


def gemm_bf16_ex(a, b, a_mn=False, b_mn=False, k_split=1, stream=None):
    """C = op(A) op(B)^T with op(A) = A ([M, K]) or, a_mn, A^T of A stored [K, M]; likewise B
    ([N, K], or stored [K, N] with b_mn).  k_split > 1 adds K-range partial products by TMA
    reductions.  For checks of the engine's MN-major operands and split K."""
    M, K = (a.shape[1], a.shape[0]) if a_mn else a.shape
    N = b.shape[1] if b_mn else b.shape[0]
    _dev(a, torch.bfloat16, None, "a")
    _dev(b, torch.bfloat16, None, "b")
    if (b.shape[0] if b_mn else b.shape[1]) != K:
        raise LmoeError("A and B disagree on K")
    c = torch.empty((M, N), dtype=torch.float32, device=a.device)
    _check(lib().lmoe_gemm_bf16_ex(_ptr(a), int(a_mn), _ptr(b), int(b_mn), _ptr(c), M, N, K, k_split,
                                   _stream(stream)), "lmoe_gemm_bf16_ex")
    return c


def _current(stream):
    """Makes `stream` (None: no change) the current one, which collectives are ordered by."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def sum_qb_statistics(hist, ntok, load=None, group=None):
    """The data-parallel exchange step of the bias update: sums the integer histograms [E, 4096],
    token counts and (for the sign rule) expert loads [E] of all ranks in place (torch.distributed
    all-reduce), so every rank then applies the same bias update as one device that saw every
    token."""
    import torch.distributed as dist
    dist.all_reduce(hist, group=group)
    dist.all_reduce(ntok, group=group)
    if load is not None:
        dist.all_reduce(load, group=group)
    return hist, ntok, load


def dp_qb_update(layer, beta, literal=False, sign_rule=False, group=None, stream=None):
    """The data-parallel bias update, on every rank of `group`: read this rank's statistics
    recorded since the last update (histogram, token count and, for the sign rule, expert loads),
    sum them over the ranks with sum_qb_statistics, set the sums back, and run the update.  Every
    rank then applies the update one device would apply after seeing every rank's tokens, and all
    ranks keep the same bias ("Pretraining a Mini Kimi K3", capsule 27, Bug 2: the all-reduce
    comes before the update)."""
    with _current(stream):
        hist, n = layer.hist(stream)
        load = layer.load(stream) if sign_rule else None
        sum_qb_statistics(hist, n, load, group)
        layer.set_hist(hist, n, stream)
        if load is not None:
            layer.set_load(load, stream)
        layer.qb_update(beta, literal=literal, sign_rule=sign_rule, stream=stream)


def dp_train_step(layer, x, dy, weights, beta=None, literal=False, sign_rule=False, group=None, grads=None,
                  stream=None):
    """One data-parallel training step's layer work on every rank of `group`: forward_backward of
    this rank's tokens (QB statistics recorded), then the exchange: every weight gradient summed
    over the ranks with one all-reduce each (the loss is the sum over all ranks' tokens, so its
    gradient is the sum of the ranks' own; dL/dx stays per rank), and, when beta is given, the
    ranks' QB statistics summed and the bias updated (dp_qb_update).  A balance loss (set_balance, on
    every rank or on none) is a mean over all ranks' sequences, whose number is summed before the
    step; layer.balance() is then this rank's share of the loss.  Returns (y, grads)."""
    import torch.distributed as dist
    sequences = getattr(layer, "balance_sequences", None)  # stand-ins may come without the balance loss
    with _current(stream):
        total = sequences(x.shape[0]) if sequences else None
        if total is not None:
            dist.all_reduce(total, group=group)
            layer.set_balance_total(total, stream)
        try:
            y, g = layer.forward_backward(x, dy, weights, record_stats=True, grads=grads, stream=stream)
        finally:
            if total is not None:
                layer.set_balance_total(None, stream)
        for name, t in g.items():
            if name != "x":
                dist.all_reduce(t, group=group)
    if beta is not None:
        dp_qb_update(layer, beta, literal=literal, sign_rule=sign_rule, group=group, stream=stream)
    return y, g


def route_noalloc(scores, bias, k, out=None, stream=None):
    """Routing of fp32 scores [T, E] with bias [E] through lmoe_route_noalloc, which allocates no
    device memory (its scratch is a static array in the library).  `out` may pass preallocated
    buffers (idx, gates, counts, offsets, perm, inv, status); missing ones are allocated here by
    torch.  out["status"] (one int32 word) holds the call's fault bits once the stream syncs."""
    T, E = scores.shape
    _dev(scores, torch.float32, (T, E), "scores")
    _dev(bias, torch.float32, (E,), "bias")
    dev = scores.device
    shapes = dict(idx=((T, k), torch.int32), gates=((T, k), torch.float32), counts=((E,), torch.int32),
                  offsets=((E + 1,), torch.int32), perm=((T * k,), torch.int32), inv=((T * k,), torch.int32),
                  status=((1,), torch.int32))
    out = dict(out or {})
    for n, (shp, dt) in shapes.items():
        if n not in out:
            out[n] = torch.empty(shp, dtype=dt, device=dev)
        _dev(out[n], dt, shp, n)
    _check(lib().lmoe_route_noalloc(_ptr(scores), _ptr(bias), T, E, k,
                                    *(_ptr(out[n]) for n in ("idx", "gates", "counts", "offsets", "perm", "inv",
                                                             "status")),
                                    _stream(stream)), "lmoe_route_noalloc")
    return out


# --------------------------------------------------------------------------- operators on the caller's tensors
# Small calls last a few microseconds on the GPU, so their host side is kept short: plain integers to
# ctypes, sizes worked out here, one look at the current device and stream.
_status_words = {}  # device index -> (tensor, address)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _status_word(index: int) -> int:
    """Address of the device word that the operators below OR their fault bits into (one a device)."""
    w = _status_words.get(index)
    if w is None:
        if torch.cuda.is_current_stream_capturing():
            raise LmoeError("the first operator call on a device cannot be captured: make one before the capture, "
                            "or pass a status word")
        word = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
        torch.cuda.synchronize(index)
        w = _status_words.setdefault(index, (word, word.data_ptr()))  # of two threads' words the first stays
    return w[1]


def _status_at(status, index: int) -> int:
    """Address of a call's status word: the caller's own, or the device's."""
    if status is None:
        return _status_word(index)
    return _dev(status, torch.int32, (1,), "status").data_ptr()


def op_status(device=None) -> int:
    """Fault bits (STATUS_*) of the mx4_* and balance_loss calls on `device` since the last read;
    synchronises the device and clears the bits it returns.  Every thread's and stream's calls share
    them, but for calls with a word of their own (status=, int32 [1] on the device: the call ORs its
    bits in and never clears them)."""
    index = None if device is None else torch.device(device).index
    index = torch.cuda.current_device() if index is None else index
    if index not in _status_words:
        return 0
    word = _status_words[index][0]
    torch.cuda.synchronize(index)
    v = int(word.item())
    word.bitwise_and_(~v)  # a bit that another thread's call set in between stays
    torch.cuda.synchronize(index)
    return v & 0xffffffff


def _device_of(*tensors) -> int:
    """The one CUDA device of the tensors (None entries are skipped)."""
    index = tensors[0].get_device()
    if index < 0:
        raise LmoeError("tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise LmoeError(f"tensors on different devices ({tensors[0].device} and {t.device})")
    return index


class _Elsewhere:
    """The rare form of an operator call, on a stream the caller names or on a device that is not the
    current one: makes the device and stream current around the call (new tensors then belong to
    that stream) and tells torch which tensors are in use there."""

    def __init__(self, index, stream, *tensors):
        if stream is not None and stream.device.index != index:
            raise LmoeError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        self.named = stream is not None
        self.stream = stream if self.named else torch.cuda.current_stream(index)
        self.tensors = tensors
        self.ctx = torch.cuda.stream(self.stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.named:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        self.ctx.__exit__(*exc)
        return False


_INT_MAX = 0x7fffffff


def _too_large(**sizes):
    """Raises for sizes that the C entries' 32-bit arguments do not hold (ctypes would drop their upper bits)."""
    names = ", ".join(f"{n} = {v}" for n, v in sizes.items() if v > _INT_MAX)
    raise LmoeError(f"unsupported shape: {names} is more than {_INT_MAX}")


_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _dtype(dtype, name):
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise LmoeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")
    return dt


def _offsets(offsets, name="offsets"):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise LmoeError(f"{name} must be a contiguous int32 tensor of one dimension and at least two entries")
    return offsets


class Mx4:
    """A matrix in MXFP4 (see lmoe.h): `rows` x `cols` in `groups` groups of rows, equal ones or those
    of `offsets` (int32 [groups + 1], kept, not copied).  elems holds two codes a byte, row after
    row; scales the blocks' scale bytes in the tensor core's order.  `stacked`: made from a tensor
    of three dimensions [groups, rows / groups, cols].  `glu`: gate and linear rows interleaved by
    mx4_quant_w13."""

    __slots__ = ("buf", "rows", "cols", "groups", "offsets", "stacked", "glu", "_scales_at")

    def __init__(self, rows, cols, groups, offsets, stacked, like, glu=False):
        if cols % 32 or cols == 0:
            raise LmoeError(f"columns must be a positive multiple of 32, got {cols}")
        self.rows, self.cols, self.groups, self.offsets = rows, cols, groups, offsets
        self.stacked, self.glu = stacked, glu
        # one buffer: the scales (the sizes of lmoe_mx4_bytes; a multiple of 1024 bytes), the elements
        tiles = (rows // groups + 127) // 128 * groups if offsets is None else (rows + 127) // 128 + groups
        self._scales_at = tiles * ((cols + 255) // 256) * 1024
        self.buf = torch.empty(self._scales_at + rows * (cols // 2), dtype=torch.uint8, device=like.device)

    @property
    def scales(self):
        return self.buf[:self._scales_at]

    @property
    def elems(self):
        return self.buf[self._scales_at:].view(self.rows, self.cols // 2)

    def _ptrs(self):
        p = self.buf.data_ptr()
        return p + self._scales_at, p

    def _match(self, rows, cols, groups, offsets, stacked, glu):
        if (self.rows, self.cols, self.groups, self.stacked, self.glu) != (rows, cols, groups, stacked, glu) or \
                (self.offsets is None) != (offsets is None):
            raise LmoeError("out was made for a matrix of another shape")
        self.offsets = offsets


def mx4_quant(x, offsets=None, index=None, out=None, stream=None, status=None) -> Mx4:
    """x in MXFP4: [rows, cols] (fp32 or bf16, cols a multiple of 32, any row stride), or stacked
    matrices [groups, rows, cols].  index (int32 [n]): the n rows x[index] instead, as routing's perm
    names them.  offsets (int32 [groups + 1]): the rows' groups, for the grouped product.  out: an
    Mx4 of an earlier call with the same shapes, to write into.  status: see op_status."""
    dt = _dtype(x.dtype, "x")
    shape = x.shape
    x_rows = 0
    if len(shape) == 2:
        rows, cols = shape
        groups, stacked = 1, False
        ld, step = x.stride()
        if rows <= 1:
            ld = cols
        if (step != 1 and rows and cols > 1) or ld < cols:
            raise LmoeError("x's columns must be contiguous and its rows must not overlap")
        if index is not None:
            if index.dtype != torch.int32 or index.dim() != 1 or not index.is_contiguous():
                raise LmoeError("index must be a contiguous int32 tensor of one dimension")
            x_rows, rows = rows, index.numel()
        if offsets is not None:
            groups = _offsets(offsets).numel() - 1
    elif len(shape) == 3 and offsets is None and index is None:
        if not x.is_contiguous():
            raise LmoeError("stacked matrices must be contiguous")
        groups, stacked = shape[0], True
        if groups == 0:
            raise LmoeError("x must hold at least one matrix")
        rows, cols, ld = groups * shape[1], shape[2], shape[2]
    else:
        raise LmoeError("x must be [rows, cols], or [groups, rows, cols] without offsets and index")
    if cols > _INT_MAX or groups > _INT_MAX:
        _too_large(cols=cols, groups=groups)
    dev = _device_of(x, offsets, index, None if out is None else out.buf, status)
    if stream is not None or dev != _current_device():
        with _Elsewhere(dev, stream, x, offsets, index, None if out is None else out.buf, status):
            return mx4_quant(x, offsets, index, out, status=status)
    if out is None:
        out = Mx4(rows, cols, groups, offsets, stacked, x)
    else:
        out._match(rows, cols, groups, offsets, stacked, False)
    elems, scales = out._ptrs()
    rc = lib().lmoe_mx4_quant(x.data_ptr(), dt, ld, None if index is None else index.data_ptr(), x_rows, rows, cols,
                              groups, None if offsets is None else offsets.data_ptr(), elems, scales,
                              _status_at(status, dev), _raw_stream(dev))
    if rc:
        _check(rc, "lmoe_mx4_quant")
    return out


def mx4_quant_w13(w1, w3, out=None, stream=None, status=None) -> Mx4:
    """A SwiGLU's gate and linear projections w1, w3 ([h, cols] or stacked [groups, h, cols], h a
    multiple of 64) as one MXFP4 matrix for mx4_gemm(..., swiglu=True)."""
    dt = _dtype(w1.dtype, "w1")
    if w1.dim() not in (2, 3) or w1.numel() == 0:
        raise LmoeError("w1 must be [h, cols] or [groups, h, cols]")
    _dev(w1, None, None, "w1")
    _dev(w3, w1.dtype, w1.shape, "w3")
    stacked = w1.dim() == 3
    groups = w1.shape[0] if stacked else 1
    h, cols = w1.shape[-2:]
    if max(groups, h, cols) > _INT_MAX:
        _too_large(groups=groups, h=h, cols=cols)
    dev = _device_of(w1, w3, None if out is None else out.buf, status)
    if stream is not None or dev != _current_device():
        with _Elsewhere(dev, stream, w1, w3, None if out is None else out.buf, status):
            return mx4_quant_w13(w1, w3, out, status=status)
    if out is None:
        out = Mx4(2 * groups * h, cols, groups, None, stacked, w1, glu=True)
    else:
        out._match(2 * groups * h, cols, groups, None, stacked, True)
    elems, scales = out._ptrs()
    _check(lib().lmoe_mx4_quant_w13(w1.data_ptr(), w3.data_ptr(), dt, groups, h, cols, elems, scales,
                                    _status_at(status, dev), _raw_stream(dev)), "lmoe_mx4_quant_w13")
    return out


def mx4_dequant(q: Mx4, dtype=torch.bfloat16, out=None, stream=None, status=None):
    """The values q stands for, [rows, cols] (stacked matrices: [groups, rows / groups, cols]).
    Rows of q that belong to no group: zeros, or left as they are in a given `out`."""
    dt = _dtype(dtype if out is None else out.dtype, "dtype")
    shape = (q.groups, q.rows // q.groups, q.cols) if q.stacked else (q.rows, q.cols)
    if out is not None and (tuple(out.shape) != shape or not out.is_contiguous()):
        raise LmoeError(f"out must be contiguous and have shape {shape}")
    offsets = q.offsets
    dev = _device_of(q.buf, offsets, out, status)
    if stream is not None or dev != _current_device():
        with _Elsewhere(dev, stream, q.buf, offsets, out, status):
            return mx4_dequant(q, dtype, out, status=status)
    flags = 0
    if out is None:
        out, flags = torch.empty(shape, dtype=dtype, device=q.buf.device), MX4_ZERO_REST
    elems, scales = q._ptrs()
    rc = lib().lmoe_mx4_dequant(elems, scales, q.rows, q.cols, q.groups, None if offsets is None else offsets.data_ptr(),
                                out.data_ptr(), dt, q.cols, flags, _status_at(status, dev), _raw_stream(dev))
    if rc:
        _check(rc, "lmoe_mx4_dequant")
    return out


def mx4_gemm(a: Mx4, b: Mx4, swiglu=False, dtype=torch.bfloat16, out=None, stream=None, status=None):
    """a b^T of MXFP4 matrices with fp32 sums: [M, N] in fp32 or bf16.  b stacked [groups, N, K]: a
    quantised with offsets, its rows of group g times matrix g.  swiglu=True: b from mx4_quant_w13,
    the result bf16 silu(gate) * linear [M, N / 2].  Rows of a that belong to no group: zeros, or
    left as they are in a given `out`."""
    if a.stacked or a.glu:
        raise LmoeError("a must be one matrix of rows")
    if a.cols != b.cols:
        raise LmoeError(f"a and b disagree on K ({a.cols} and {b.cols})")
    offsets = a.offsets
    if b.offsets is not None or (offsets is None) == b.stacked or a.groups != b.groups:
        raise LmoeError("a product takes a plain matrix b, or a with offsets and as many stacked matrices b")
    if bool(swiglu) != b.glu:
        raise LmoeError("swiglu=True goes with a matrix from mx4_quant_w13")
    M, N = a.rows, b.rows // b.groups
    cols = N // 2 if swiglu else N
    dt = _dtype(dtype if out is None else out.dtype, "dtype")
    if out is not None and (tuple(out.shape) != (M, cols) or (cols > 1 and out.stride(1) != 1) or
                            (M > 1 and out.stride(0) < cols)):
        raise LmoeError(f"out must have shape {(M, cols)}, contiguous columns and rows that do not overlap")
    dev = _device_of(a.buf, offsets, b.buf, out, status)
    if stream is not None or dev != _current_device():
        with _Elsewhere(dev, stream, a.buf, offsets, b.buf, out, status):
            return mx4_gemm(a, b, swiglu, dtype, out, status=status)
    flags = MX4_SWIGLU if swiglu else 0
    ld = cols
    if out is None:
        out, flags = torch.empty((M, cols), dtype=dtype, device=a.buf.device), flags | MX4_ZERO_REST
    elif M > 1:
        ld = out.stride(0)
    ae, asc = a._ptrs()
    be, bsc = b._ptrs()
    rc = lib().lmoe_mx4_gemm(ae, asc, be, bsc, M, N, a.cols, a.groups, None if offsets is None else offsets.data_ptr(),
                             out.data_ptr(), dt, ld, flags, _status_at(status, dev), _raw_stream(dev))
    if rc:
        _check(rc, "lmoe_mx4_gemm")
    return out


@functools.lru_cache(None)
def _balance_floats() -> int:
    """fp32 values that hold a call's loss (the first 64 bytes) and scratch."""
    n = c_size_t(0)
    _check(lib().lmoe_balance_scratch_bytes(ctypes.byref(n)), "lmoe_balance_scratch_bytes")
    return 16 + (n.value + 3) // 4


def balance_loss(scores, idx, coef, cu_seqlens=None, grad=True, out=None, stream=None, status=None):
    """Balance loss of a router (lmoe_balance_loss): scores [T, E] fp32 and the choice idx [T, k] int32,
    as Layer.routing() gives them; cu_seqlens (int32 [S + 1]) bounds the sequences (None: one).
    Returns dict(loss [1] fp32, counts [S, E] int32, dscores [T, E] fp32): the gradient of the loss
    in the scores, left out with grad=False.  `out` may pass preallocated buffers.  status: see op_status."""
    if scores.dim() != 2 or idx.dim() != 2:
        raise LmoeError("scores must be [T, E] and idx [T, k]")
    T, E = scores.shape
    k = idx.shape[1]
    S = 1
    if cu_seqlens is not None:
        S = _offsets(cu_seqlens, "cu_seqlens").numel() - 1
    if max(T, E, k, S) > _INT_MAX:
        _too_large(T=T, E=E, k=k, S=S)
    dev = _device_of(scores, idx, cu_seqlens, status)
    _dev(scores, torch.float32, None, "scores")
    _dev(idx, torch.int32, (T, k), "idx")
    given = () if out is None else tuple(out.values())
    if stream is not None or dev != _current_device():
        with _Elsewhere(dev, stream, scores, idx, cu_seqlens, status, *given):
            return balance_loss(scores, idx, coef, cu_seqlens, grad, out, status=status)
    if given:
        _device_of(scores, *given)
    device = scores.device
    # the loss and the call's scratch share a buffer
    buf = torch.empty(_balance_floats(), dtype=torch.float32, device=device)
    res = dict(out or ())
    if "loss" in res:
        _dev(res["loss"], torch.float32, (1,), "loss")
    else:
        res["loss"] = buf[:1]
    if "counts" in res:
        _dev(res["counts"], torch.int32, (S, E), "counts")
    else:
        res["counts"] = torch.empty((S, E), dtype=torch.int32, device=device)
    dscores = None
    if grad:
        if "dscores" in res:
            _dev(res["dscores"], torch.float32, (T, E), "dscores")
        else:
            res["dscores"] = torch.empty_like(scores)
        dscores = res["dscores"].data_ptr()
    else:
        res.pop("dscores", None)  # a given one is not this call's
    rc = lib().lmoe_balance_loss(scores.data_ptr(), idx.data_ptr(), T, E, k,
                                 None if cu_seqlens is None else cu_seqlens.data_ptr(), S, coef,
                                 res["counts"].data_ptr(), res["loss"].data_ptr(), dscores, buf.data_ptr() + 64,
                                 _status_at(status, dev), _raw_stream(dev))
    if rc:
        _check(rc, "lmoe_balance_loss")
    return res


def layer_from_weights(shape, weights_cpu: dict, max_tokens=None, device="cuda", stream=None,
                       experts=EXPERTS_BF16) -> Layer:
    """Creates a Layer from the CPU weight dict of the seeded generator (copied to the device)."""
    w = {n: t.to(device) for n, t in weights_cpu.items()}
    return Layer(shape.d, shape.l, shape.E, shape.k, shape.h, shape.hs,
                 F32 if shape.dtype == "f32" else BF16, max_tokens or shape.T, w,
                 rms_eps=shape.rms_eps, stream=stream, experts=experts)
