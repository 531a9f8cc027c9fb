"""Thin Python binding of liblq.so (include/lq_state.h), same names as the C ABI.

Argument marshalling only: torch tensors are checked for device, dtype, shape
and contiguity and passed as raw device pointers together with torch's current
CUDA stream.  Every computation happens in the CUDA library; if liblq.so is
missing this module raises on import of the library instead of falling back.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblq.so")

LQ_OK = 0
LQ_ERR_INVALID_ARG = -1
LQ_ERR_SHAPE = -2
LQ_ERR_WORKSPACE = -3
LQ_ERR_WINDOW_FULL = -4
LQ_ERR_CUDA = -5
LQ_ERR_NONFINITE = -6
LQ_ERR_UNSUPPORTED = -7
LQ_ERR_TIMEOUT = -8

LQ_GATE_SCALAR, LQ_GATE_CHANNEL = 0, 1
LQ_MODE_FP32, LQ_MODE_INT8_STEP, LQ_MODE_INT8_WINDOW = 0, 1, 2

EXPORTED = ["lq_workspace_bytes", "lq_config_check", "lq_state_init", "lq_decode_step",
            "lq_window_flush", "lq_state_buffered", "lq_state_export_fp32",
            "lq_state_export_view", "lq_state_import_view", "lq_quantize_state",
            "lq_dequantize_state", "lq_quantize_state_static", "lq_damp_select", "lq_get_status",
            "lq_state_destroy", "lq_strerror", "lq_selftest_division", "lq_prefill",
            "lq_state_init_static", "lq_fit_static_scales", "lq_selftest_wait", "lq_state_set_phases",
            "lq_conv_prefill", "lq_conv_step", "lq_ssm_workspace_bytes", "lq_ssm_prefill", "lq_ssm_step",
            "lq_norm_in", "lq_norm_out"]


class LqError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} ({code})")


class lq_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("B", "H", "Hk", "dk", "dv", "gate", "mode", "W", "r",
                                          "power_iters", "n_hp_rows", "smoothing", "fused_flush",
                                          "buffer_bf16", "state_bits")]


class lq_conv_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("dtype", "B", "C", "K", "act")]


class lq_ssm_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("dtype", "B", "H", "G", "dk", "dv", "softplus")]


class lq_norm_config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("dtype", "x_dtype", "rows", "G", "D", "w_groups", "act",
                                          "gate_first")] + [("eps", C.c_float), ("scale", C.c_float)]


class lq_qstate_view(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("bf16_rows", C.c_void_p), ("m", C.c_void_p),
                ("s", C.c_void_p), ("comp_k", C.c_void_p), ("comp_v", C.c_void_p)]


_lib = None


def lib():
    """Load liblq.so (building it in-tree first if it is missing or stale)."""
    global _lib
    if _lib is None:
        from . import build as _build
        if not os.path.exists(LIB_PATH) or _build._stale():
            _build.build()
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        cfgp = C.POINTER(lq_config)
        viewp = C.POINTER(lq_qstate_view)
        sig = {
            "lq_workspace_bytes": (sz, [cfgp]),
            "lq_config_check": (C.c_int, [cfgp]),
            "lq_state_init": (C.c_int, [C.POINTER(vp), cfgp, vp, sz, vp, vp, vp]),
            "lq_decode_step": (C.c_int, [vp, vp, vp, vp, vp, vp, vp, vp]),
            "lq_window_flush": (C.c_int, [vp, vp]),
            "lq_state_buffered": (C.c_int, [vp]),
            "lq_state_export_fp32": (C.c_int, [vp, vp, vp]),
            "lq_state_export_view": (C.c_int, [vp, viewp, vp]),
            "lq_state_import_view": (C.c_int, [vp, viewp, vp]),
            "lq_quantize_state": (C.c_int, [cfgp, vp, vp, viewp, vp]),
            "lq_dequantize_state": (C.c_int, [cfgp, viewp, vp, vp, vp]),
            "lq_quantize_state_static": (C.c_int, [cfgp, vp, vp, viewp, vp]),
            "lq_damp_select": (C.c_int, [cfgp, i32, vp, i32, vp, vp, vp, vp]),
            "lq_get_status": (C.c_int, [vp, vp]),
            "lq_state_destroy": (None, [vp]),
            "lq_strerror": (C.c_char_p, [C.c_int]),
            "lq_selftest_division": (C.c_int, [vp, vp, vp, vp, vp, i32, vp]),
            "lq_prefill": (C.c_int, [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "lq_state_init_static": (C.c_int, [C.POINTER(vp), cfgp, vp, sz, vp, vp, vp, vp]),
            "lq_fit_static_scales": (C.c_int, [cfgp, i32, vp, i32, vp, vp, vp, vp]),
            "lq_selftest_wait": (C.c_int, [vp, C.c_int64, vp]),
            "lq_state_set_phases": (C.c_int, [vp, vp, vp]),
            "lq_conv_prefill": (C.c_int, [vp, i32, vp, vp, i64, vp, vp, vp, vp, vp, i64, vp]),
            "lq_conv_step": (C.c_int, [vp, vp, vp, i64, vp, vp, vp, i64, vp]),
            "lq_ssm_workspace_bytes": (sz, [vp, i32]),
            "lq_ssm_prefill": (C.c_int, [vp, i32, vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64,
                                         vp, sz, vp]),
            "lq_ssm_step": (C.c_int, [vp, vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp, i64, vp]),
            "lq_norm_in": (C.c_int, [vp, vp, i64, vp, vp, i64, vp, vp, i64, vp, i64, vp]),
            "lq_norm_out": (C.c_int, [vp, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().lq_strerror(code).decode()


def _chk(rc: int, what: str):
    if rc != LQ_OK:
        raise LqError(rc, what)


@dataclass
class Config:
    B: int
    H: int
    Hk: int
    dk: int
    dv: int
    gate: str = "gdn"            # "gdn" | "kda"
    mode: str = "window"         # "fp32" | "step" | "window"
    W: int = 32
    r: int = 4
    power_iters: int = 8
    n_hp_rows: int = 0
    smoothing: int = 1
    fused_flush: int = 1
    buffer_bf16: int = 0         # 1: buffered token updates kept in BF16 (window mode)
    state_bits: int = 8          # code width of the quantized state: 8, 6 or 4 (bit-packed)

    def c(self) -> lq_config:
        gate = {"gdn": LQ_GATE_SCALAR, "kda": LQ_GATE_CHANNEL}[self.gate]
        mode = {"fp32": LQ_MODE_FP32, "step": LQ_MODE_INT8_STEP, "window": LQ_MODE_INT8_WINDOW}[self.mode]
        return lq_config(self.B, self.H, self.Hk, self.dk, self.dv, gate, mode, self.W, self.r,
                         self.power_iters, self.n_hp_rows, self.smoothing, self.fused_flush,
                         self.buffer_bf16, self.state_bits)

    @property
    def heads(self) -> int:
        return self.B * self.H

    @property
    def ga(self) -> int:
        return self.dk if self.gate == "kda" else 1

    @staticmethod
    def from_workload(wl, mode: str = "window", **kw) -> "Config":
        base = dict(B=wl.B, H=wl.H, Hk=wl.Hk, dk=wl.dk, dv=wl.dv, gate=wl.gate, mode=mode,
                    W=(1 if mode == "step" else wl.W), r=wl.r, power_iters=wl.K,
                    n_hp_rows=(wl.P if mode != "fp32" else 0), smoothing=wl.smoothing,
                    buffer_bf16=(wl.buffer_bf16 if mode == "window" else 0),
                    state_bits=(wl.bits if mode != "fp32" else 8))
        base.update(kw)
        return Config(**base)


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t: torch.Tensor, name: str, shape=None, dtype=torch.float32) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _host_rows(cfg: Config, hp_rows):
    if cfg.n_hp_rows == 0:
        return None, None
    arr = torch.as_tensor(hp_rows, dtype=torch.int32).cpu().contiguous()
    if tuple(arr.shape) != (cfg.H, cfg.n_hp_rows):
        raise ValueError(f"hp_rows must be [H, P] = {(cfg.H, cfg.n_hp_rows)}")
    return arr, C.c_void_p(arr.data_ptr())


def view_shapes(cfg: Config) -> dict:
    B, H, dk, dv, P, r = cfg.B, cfg.H, cfg.dk, cfg.dv, cfg.n_hp_rows, cfg.r
    return {"codes": ((B, H, dk - P, dv), torch.int8), "bf16_rows": ((B, H, P, dv), torch.int16),
            "m": ((B, H, dk), torch.float32), "s": ((B, H, dv), torch.float32),
            "comp_k": ((B, H, r, dk), torch.float32), "comp_v": ((B, H, r, dv), torch.float32)}


def alloc_view(cfg: Config, device="cuda") -> dict:
    return {k: torch.zeros(shape, dtype=dt, device=device) for k, (shape, dt) in view_shapes(cfg).items()}


def _view_struct(cfg: Config, view: dict) -> lq_qstate_view:
    ptr = {}
    for k, (shape, dt) in view_shapes(cfg).items():
        t = view[k]
        ptr[k] = _dev(t, k, shape, dt) if t.numel() else None
    return lq_qstate_view(ptr["codes"], ptr["bf16_rows"], ptr["m"], ptr["s"], ptr["comp_k"], ptr["comp_v"])


def lq_config_check(cfg: Config) -> int:
    return lib().lq_config_check(C.byref(cfg.c()))


def lq_workspace_bytes(cfg: Config) -> int:
    return lib().lq_workspace_bytes(C.byref(cfg.c()))


class LqState:
    """Owns the opaque handle and keeps the workspace tensor alive."""

    def __init__(self, cfg: Config, handle: int, workspace: torch.Tensor, rows):
        self.cfg = cfg
        self.handle = C.c_void_p(handle)
        self.workspace = workspace
        self._rows = rows

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.lq_state_destroy(h)
            self.handle = C.c_void_p(0)


def lq_state_init(cfg: Config, S0: torch.Tensor, hp_rows=None, workspace: torch.Tensor | None = None,
                  stream=None, static_m: torch.Tensor | None = None,
                  static_s: torch.Tensor | None = None) -> LqState:
    """lq_state_init, or lq_state_init_static when the scales are given
    (cfg.smoothing = 2: static_m [H, dk], static_s [H, dv])."""
    nbytes = lq_workspace_bytes(cfg)
    if nbytes == 0:
        _chk(lq_config_check(cfg), "lq_config_check")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=S0.device)
    p_s0 = _dev(S0, "S0", (cfg.B, cfg.H, cfg.dk, cfg.dv))
    h = C.c_void_p()
    ws = (C.c_void_p(workspace.data_ptr()), workspace.numel() * workspace.element_size())
    if static_m is not None or static_s is not None:
        pm = _dev(static_m, "static_m", (cfg.H, cfg.dk))
        ps = _dev(static_s, "static_s", (cfg.H, cfg.dv))
        _chk(lib().lq_state_init_static(C.byref(h), C.byref(cfg.c()), *ws, C.c_void_p(p_s0), C.c_void_p(pm),
                                        C.c_void_p(ps), C.c_void_p(_stream(stream))), "lq_state_init_static")
        return LqState(cfg, h.value, workspace, None)
    rows, p_rows = _host_rows(cfg, hp_rows)
    _chk(lib().lq_state_init(C.byref(h), C.byref(cfg.c()), *ws, C.c_void_p(p_s0), p_rows,
                             C.c_void_p(_stream(stream))), "lq_state_init")
    return LqState(cfg, h.value, workspace, rows)


def lq_fit_static_scales(cfg: Config, states: torch.Tensor, gates: torch.Tensor | None = None,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Static scales (smoothing 2) of every head from calibration states
    [n, H, dk, dv]; gates [n_samples, H, 1 | dk] (the calibration decays that
    weight the rows by their persistence) or None (unweighted).  Returns
    (m [H, dk], s [H, dv])."""
    n = states.shape[0]
    p_st = _dev(states, "states", (n, cfg.H, cfg.dk, cfg.dv))
    ng, p_g = 0, None
    if gates is not None:
        ng = gates.shape[0]
        p_g = _dev(gates, "gates", (ng, cfg.H, cfg.dk if cfg.gate == "kda" else 1))
    m = torch.empty((cfg.H, cfg.dk), device=states.device)
    s = torch.empty((cfg.H, cfg.dv), device=states.device)
    _chk(lib().lq_fit_static_scales(C.byref(cfg.c()), C.c_int32(n), C.c_void_p(p_st), C.c_int32(ng),
                                    C.c_void_p(p_g), C.c_void_p(m.data_ptr()), C.c_void_p(s.data_ptr()),
                                    C.c_void_p(_stream(stream))), "lq_fit_static_scales")
    return m, s


def lq_decode_step(st: LqState, q, k, v, beta, alpha, o, stream=None):
    c = st.cfg
    args = [_dev(q, "q", (c.B, c.Hk, c.dk)), _dev(k, "k", (c.B, c.Hk, c.dk)),
            _dev(v, "v", (c.B, c.H, c.dv)), _dev(beta, "beta", (c.B, c.H)),
            _dev(alpha, "alpha", (c.B, c.H) if c.gate == "gdn" else (c.B, c.H, c.dk)),
            _dev(o, "o", (c.B, c.H, c.dv))]
    _chk(lib().lq_decode_step(st.handle, *[C.c_void_p(a) for a in args], C.c_void_p(_stream(stream))),
         "lq_decode_step")


def lq_state_set_phases(st: LqState, phases, stream=None):
    """Staggered windows: phases [B] (ints in [0, W)), or None to remove them."""
    if phases is None:
        _chk(lib().lq_state_set_phases(st.handle, None, C.c_void_p(_stream(stream))), "lq_state_set_phases")
        return
    vals = [int(x) for x in phases]
    if len(vals) != st.cfg.B:
        raise ValueError(f"phases: {len(vals)} values for B = {st.cfg.B}")
    arr = (C.c_int32 * len(vals))(*vals)
    _chk(lib().lq_state_set_phases(st.handle, C.cast(arr, C.c_void_p), C.c_void_p(_stream(stream))),
         "lq_state_set_phases")


def lq_window_flush(st: LqState, stream=None):
    _chk(lib().lq_window_flush(st.handle, C.c_void_p(_stream(stream))), "lq_window_flush")


def lq_state_buffered(st: LqState) -> int:
    return lib().lq_state_buffered(st.handle)


def lq_state_export_fp32(st: LqState, S: torch.Tensor, stream=None):
    c = st.cfg
    _chk(lib().lq_state_export_fp32(st.handle, C.c_void_p(_dev(S, "S", (c.B, c.H, c.dk, c.dv))),
                                    C.c_void_p(_stream(stream))), "lq_state_export_fp32")


def lq_state_export_view(st: LqState, view: dict, stream=None):
    v = _view_struct(st.cfg, view)
    _chk(lib().lq_state_export_view(st.handle, C.byref(v), C.c_void_p(_stream(stream))), "lq_state_export_view")


def lq_state_import_view(st: LqState, view: dict, stream=None):
    v = _view_struct(st.cfg, view)
    _chk(lib().lq_state_import_view(st.handle, C.byref(v), C.c_void_p(_stream(stream))), "lq_state_import_view")


def lq_quantize_state(cfg: Config, S: torch.Tensor, view: dict, hp_rows=None, stream=None):
    p = _dev(S, "S", (cfg.B, cfg.H, cfg.dk, cfg.dv))
    rows, p_rows = _host_rows(cfg, hp_rows)
    v = _view_struct(cfg, view)
    _chk(lib().lq_quantize_state(C.byref(cfg.c()), C.c_void_p(p), p_rows, C.byref(v),
                                 C.c_void_p(_stream(stream))), "lq_quantize_state")


LQ_STATIC_ROWS_MAX = 8192
LQ_MAX_WINDOW = 4096


def lq_quantize_state_static(cfg: Config, S: torch.Tensor, view: dict, hp_rows=None, stream=None):
    """lq_quantize_state for callers that must not let the library allocate
    device memory: the BF16 row list goes to a fixed array inside liblq.so
    (at most LQ_STATIC_ROWS_MAX = H * n_hp_rows entries) instead of a per-call
    temporary.  Calls that overlap on the GPU share that array and race."""
    p = _dev(S, "S", (cfg.B, cfg.H, cfg.dk, cfg.dv))
    rows, p_rows = _host_rows(cfg, hp_rows)
    v = _view_struct(cfg, view)
    _chk(lib().lq_quantize_state_static(C.byref(cfg.c()), C.c_void_p(p), p_rows, C.byref(v),
                                        C.c_void_p(_stream(stream))), "lq_quantize_state_static")


LQ_PREFILL_CHUNK = 16


def lq_prefill(cfg: Config, q, k, v, beta, alpha, S0=None, S_out=None, o=None, stream=None) -> torch.Tensor:
    """Chunked prefill of T tokens (inputs [T, ...] stacks of decode-step
    inputs) from S0 (None: zero state) into S_out (allocated when None; may be
    S0); o [T,B,H,dv] receives the outputs when given.  Returns S_out."""
    T = q.shape[0]
    B, H, Hk, dk, dv = cfg.B, cfg.H, cfg.Hk, cfg.dk, cfg.dv
    shapes = {"q": (T, B, Hk, dk), "k": (T, B, Hk, dk), "v": (T, B, H, dv), "beta": (T, B, H),
              "alpha": (T, B, H, dk) if cfg.gate == "kda" else (T, B, H)}
    ptr = {n: _dev(t, n, shapes[n]) for n, t in (("q", q), ("k", k), ("v", v), ("beta", beta), ("alpha", alpha))}
    if S_out is None:
        S_out = torch.empty((B, H, dk, dv), device=q.device)
    p_out = _dev(S_out, "S_out", (B, H, dk, dv))
    p_s0 = _dev(S0, "S0", (B, H, dk, dv)) if S0 is not None else None
    p_o = _dev(o, "o", (T, B, H, dv)) if o is not None else None
    _chk(lib().lq_prefill(C.byref(cfg.c()), C.c_int32(T), C.c_void_p(ptr["q"]), C.c_void_p(ptr["k"]),
                          C.c_void_p(ptr["v"]), C.c_void_p(ptr["beta"]), C.c_void_p(ptr["alpha"]),
                          C.c_void_p(p_s0), C.c_void_p(p_out), C.c_void_p(p_o), C.c_void_p(_stream(stream))),
         "lq_prefill")
    return S_out


def lq_selftest_division(a: torch.Tensor, b: torch.Tensor, stream=None):
    """Run the codec's division routine and IEEE division on the same device
    operands (float32, same even length; pairs b[2j] == b[2j+1] for the
    two-lane variant).  Returns (fast, pair, ieee)."""
    n = a.numel()
    pa = _dev(a, "a", (n,))
    pb = _dev(b, "b", (n,))
    fast, pair, ieee = (torch.empty_like(a) for _ in range(3))
    _chk(lib().lq_selftest_division(C.c_void_p(pa), C.c_void_p(pb), C.c_void_p(fast.data_ptr()),
                                    C.c_void_p(pair.data_ptr()), C.c_void_p(ieee.data_ptr()), n,
                                    C.c_void_p(_stream(stream))), "lq_selftest_division")
    return fast, pair, ieee


def lq_dequantize_state(cfg: Config, view: dict, S: torch.Tensor, hp_rows=None, stream=None):
    p = _dev(S, "S", (cfg.B, cfg.H, cfg.dk, cfg.dv))
    rows, p_rows = _host_rows(cfg, hp_rows)
    v = _view_struct(cfg, view)
    _chk(lib().lq_dequantize_state(C.byref(cfg.c()), C.byref(v), p_rows, C.c_void_p(p),
                                   C.c_void_p(_stream(stream))), "lq_dequantize_state")


def lq_damp_select(cfg: Config, states: torch.Tensor, gates: torch.Tensor, energy: torch.Tensor,
                   rows: torch.Tensor, stream=None):
    n = states.shape[0]
    ps = _dev(states, "states", (n, cfg.H, cfg.dk, cfg.dv))
    ng = gates.shape[0]
    pg = _dev(gates, "gates", (ng, cfg.H, cfg.ga))
    pe = _dev(energy, "energy", (cfg.H, cfg.dk), torch.float64)
    pr = _dev(rows, "rows", (cfg.H, cfg.n_hp_rows), torch.int32)
    _chk(lib().lq_damp_select(C.byref(cfg.c()), n, C.c_void_p(ps), ng, C.c_void_p(pg), C.c_void_p(pe),
                              C.c_void_p(pr), C.c_void_p(_stream(stream))), "lq_damp_select")


def lq_selftest_wait(st: LqState, limit_ns: int = 1_000_000, stream=None):
    """Make one bounded device wait run out on purpose (failure-detection self-test)."""
    _chk(lib().lq_selftest_wait(st.handle, C.c_int64(limit_ns), C.c_void_p(_stream(stream))),
         "lq_selftest_wait")


def lq_get_status(st: LqState, stream=None) -> int:
    return lib().lq_get_status(st.handle, C.c_void_p(_stream(stream)))


def lq_state_destroy(st: LqState):
    if st.handle.value:
        lib().lq_state_destroy(st.handle)
        st.handle = C.c_void_p(0)


# ---------------------------------------------------------------------------
# The recurrent layer around the state: short causal convolution, selective
# state-space scan, norms.  Activations float32, bfloat16 or float16; prompts
# are packed ([rows, ...] with cu, the B+1 int32 row offsets on the device) or
# time-major ([T, B, ...]); rows may be columns of a wider tensor.
# ---------------------------------------------------------------------------
LQ_F32, LQ_BF16, LQ_F16 = 0, 1, 2
LQ_ACT_NONE, LQ_ACT_SILU, LQ_ACT_SIGMOID = 0, 1, 2
LQ_CONV_MAX_TAPS = 4
LQ_NORM_MAX_D = 16384

_DTYPES = {torch.float32: LQ_F32, torch.bfloat16: LQ_BF16, torch.float16: LQ_F16}
_ACTS = {None: LQ_ACT_NONE, "silu": LQ_ACT_SILU, "sigmoid": LQ_ACT_SIGMOID}


_raw_stream = torch._C._cuda_getCurrentRawStream    # the current stream's handle, without a Stream object


def _layer_call(fn):
    """A call on the device of its first argument and on torch's current stream
    of it, or on the given stream: both are made current for the call, so that
    what it allocates belongs to the stream it is used on, and the arguments'
    memory is not reused before that stream is done with it."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        t = args[0] if args else next(iter(kw.values()), None)
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{fn.__name__} takes CUDA tensors")
        if stream is None:
            if t.get_device() == torch._C._cuda_getDevice():
                return fn(*args, **kw)
            with torch.cuda.device(t.device):
                return fn(*args, **kw)
        if stream.device != t.device:
            raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
            for v in (*args, *kw.values()):
                if isinstance(v, torch.Tensor) and v.is_cuda:
                    v.record_stream(stream)
            return out

    return call


def _refuse(t, name: str, shape, dtype, dev: int):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t, name: str, shape, n_tail: int, width: int, dtype, dev: int):
    """Pointer and row stride of a tensor of token rows: its last n_tail
    dimensions are one contiguous row of `width` elements, the others evenly
    spaced rows."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), width
    st = t.stride()
    n = len(st)
    w = 1
    for i in range(n - 1, n - 1 - n_tail, -1):
        if shape[i] != 1:
            if st[i] != w:
                raise ValueError(f"{name}: the elements of a row must be contiguous")
            w *= shape[i]
    ld, rows = width, 1
    for i in range(n - n_tail - 1, -1, -1):
        if shape[i] != 1:
            if rows == 1:
                ld = st[i]
            elif st[i] != rows * ld:
                raise ValueError(f"{name}: rows must be evenly spaced")
            rows *= shape[i]
    return t.data_ptr(), ld


def _flat(t, name: str, shape, dev: int, dtype=torch.float32):
    """Pointer of an optional contiguous tensor."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _refuse(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype_of(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"activations must be float32, bfloat16 or float16, got {t.dtype}")
    return _DTYPES[t.dtype]


def _act_of(act) -> int:
    if act not in _ACTS:
        raise ValueError(f"unknown activation {act!r}")
    return _ACTS[act]


def _prompt(x: torch.Tensor, cu, n_tail: int, dev: int):
    """(B, rows, pointer of cu or None) of a packed or time-major prompt batch."""
    lead = x.shape[:x.dim() - n_tail]
    if cu is None:
        if len(lead) != 2:
            raise ValueError(f"a time-major prompt is [T, B, ...], got {tuple(x.shape)}; a packed one needs cu")
        return lead[1], lead[0] * lead[1], None
    if len(lead) != 1:
        raise ValueError(f"a packed prompt is [rows, ...], got {tuple(x.shape)}")
    if cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu must hold B+1 offsets")
    return cu.shape[0] - 1, lead[0], _flat(cu, "cu", cu.shape, dev, torch.int32)


def _scale(scale, shape, dev: int):
    """(factor, pointer of the per-channel scale) of a number or a tensor."""
    if isinstance(scale, torch.Tensor):
        return 1.0, _flat(scale, "scale", shape, dev)
    return float(scale), None


@_layer_call
def lq_conv_prefill(x, w, bias=None, act="silu", state0=None, state_out=None, y=None, cu=None):
    """Short causal depthwise convolution over prompts x ([rows, C] with cu, or
    [T, B, C]) with taps w [C, K], from the windows state0 [B, K-1, C] (None:
    zeros).  Returns (y, state_out), allocated when None; state_out may be
    state0.  Takes stream=."""
    dt, dev, code = x.dtype, x.get_device(), _dtype_of(x)
    B, rows, p_cu = _prompt(x, cu, 1, dev)
    ch, K = w.shape
    shape = (*x.shape[:-1], ch)
    px, ldx = _rows(x, "x", shape, 1, ch, dt, dev)
    y = x.new_empty(shape) if y is None else y
    py, ldy = _rows(y, "y", shape, 1, ch, dt, dev)
    win = (B, K - 1, ch)
    state_out = x.new_empty(win) if state_out is None else state_out
    cfg = lq_conv_config(code, B, ch, K, _act_of(act))
    rc = lib().lq_conv_prefill(C.addressof(cfg), rows, p_cu, px, ldx, _flat(w, "w", (ch, K), dev),
                               _flat(bias, "bias", (ch,), dev), _flat(state0, "state0", win, dev, dt),
                               _flat(state_out, "state_out", win, dev, dt), py, ldy, _raw_stream(dev))
    _chk(rc, "lq_conv_prefill")
    return y, state_out


@_layer_call
def lq_conv_step(state, x, w, bias=None, act="silu", y=None):
    """One token of every sequence, x [B, C]; the windows state [B, K-1, C] move
    on in place.  Returns y [B, C] (allocated when None; may be x).  Takes
    stream=."""
    dt, dev, code = x.dtype, x.get_device(), _dtype_of(x)
    ch, K = w.shape
    B = x.shape[0]
    px, ldx = _rows(x, "x", (B, ch), 1, ch, dt, dev)
    y = x.new_empty((B, ch)) if y is None else y
    py, ldy = _rows(y, "y", (B, ch), 1, ch, dt, dev)
    cfg = lq_conv_config(code, B, ch, K, _act_of(act))
    rc = lib().lq_conv_step(C.addressof(cfg), _flat(state, "state", (B, K - 1, ch), dev, dt), px, ldx,
                            _flat(w, "w", (ch, K), dev), _flat(bias, "bias", (ch,), dev), py, ldy, _raw_stream(dev))
    _chk(rc, "lq_conv_step")
    return y


def lq_ssm_workspace_bytes(dtype, B: int, H: int, G: int, dk: int, dv: int, rows: int) -> int:
    """Bytes of the workspace lq_ssm_prefill takes for these sizes."""
    cfg = lq_ssm_config(_DTYPES[dtype], B, H, G, dk, dv, 1)
    return lib().lq_ssm_workspace_bytes(C.addressof(cfg), rows)


@_layer_call
def lq_ssm_prefill(x, dt, A, Bm, Cm, D=None, dt_bias=None, softplus=True, S0=None, S_out=None, y=None, cu=None,
                   workspace=None):
    """Selective state-space scan over prompts: x [..., H, dv], dt [..., H],
    Bm, Cm [..., G, dk] with [...] = [rows] (and cu) or [T, B]; A, D, dt_bias
    [H].  From the states S0 [B, H, dk, dv] (None: zeros).  Returns
    (y [..., H, dv], S_out), allocated when None; S_out may be S0.  The
    workspace (uint8, at least lq_ssm_workspace_bytes) is allocated when None.
    Takes stream=."""
    t, dev, code = x.dtype, x.get_device(), _dtype_of(x)
    B, rows, p_cu = _prompt(x, cu, 2, dev)
    lead, (H, dv), (G, dk) = x.shape[:-2], x.shape[-2:], Bm.shape[-2:]
    sx, sb = (*lead, H, dv), (*lead, G, dk)
    px, ldx = _rows(x, "x", sx, 2, H * dv, t, dev)
    pd, ldd = _rows(dt, "dt", (*lead, H), 1, H, t, dev)
    pb, ldb = _rows(Bm, "Bm", sb, 2, G * dk, t, dev)
    pc, ldc = _rows(Cm, "Cm", sb, 2, G * dk, t, dev)
    y = x.new_empty(sx) if y is None else y
    py, ldy = _rows(y, "y", sx, 2, H * dv, t, dev)
    st, hs = (B, H, dk, dv), (H,)
    S_out = x.new_empty(st, dtype=torch.float32) if S_out is None else S_out
    cfg = lq_ssm_config(code, B, H, G, dk, dv, 1 if softplus else 0)
    L, p_cfg = lib(), C.addressof(cfg)
    n_ws = L.lq_ssm_workspace_bytes(p_cfg, rows)
    if workspace is None and n_ws:
        workspace = x.new_empty(n_ws, dtype=torch.uint8)
    p_ws = None
    if workspace is not None:
        n_ws = workspace.numel()
        p_ws = _flat(workspace, "workspace", (n_ws,), dev, torch.uint8)
    rc = L.lq_ssm_prefill(p_cfg, rows, p_cu, px, ldx, pd, ldd, _flat(A, "A", hs, dev), pb, ldb, pc, ldc,
                          _flat(D, "D", hs, dev), _flat(dt_bias, "dt_bias", hs, dev), _flat(S0, "S0", st, dev),
                          _flat(S_out, "S_out", st, dev), py, ldy, p_ws, n_ws, _raw_stream(dev))
    _chk(rc, "lq_ssm_prefill")
    return y, S_out


@_layer_call
def lq_ssm_step(S, x, dt, A, Bm, Cm, D=None, dt_bias=None, softplus=True, y=None):
    """One token of every sequence: x [B, H, dv], dt [B, H], Bm, Cm [B, G, dk];
    the states S [B, H, dk, dv] are updated in place.  Returns y [B, H, dv]
    (allocated when None).  Takes stream=."""
    t, dev, code = x.dtype, x.get_device(), _dtype_of(x)
    (B, H, dv), (G, dk) = x.shape, Bm.shape[-2:]
    px, ldx = _rows(x, "x", (B, H, dv), 2, H * dv, t, dev)
    pd, ldd = _rows(dt, "dt", (B, H), 1, H, t, dev)
    pb, ldb = _rows(Bm, "Bm", (B, G, dk), 2, G * dk, t, dev)
    pc, ldc = _rows(Cm, "Cm", (B, G, dk), 2, G * dk, t, dev)
    y = x.new_empty((B, H, dv)) if y is None else y
    py, ldy = _rows(y, "y", (B, H, dv), 2, H * dv, t, dev)
    hs = (H,)
    cfg = lq_ssm_config(code, B, H, G, dk, dv, 1 if softplus else 0)
    rc = lib().lq_ssm_step(C.addressof(cfg), _flat(S, "S", (B, H, dk, dv), dev), px, ldx, pd, ldd,
                           _flat(A, "A", hs, dev), pb, ldb, pc, ldc, _flat(D, "D", hs, dev),
                           _flat(dt_bias, "dt_bias", hs, dev), py, ldy, _raw_stream(dev))
    _chk(rc, "lq_ssm_step")
    return y


@_layer_call
def lq_norm_in(x, w, res=None, scale=1.0, eps=1e-5, h=None, y=None):
    """Norm before a block, with the residual: h = res + scale x, y = rms(h) w
    over the last dimension of x [..., D]; scale is a number or a float32 tensor
    [D].  Returns (y, h), allocated when None; h and y may be x or res.  Takes
    stream=."""
    t, dev, code = x.dtype, x.get_device(), _dtype_of(x)
    shape = x.shape
    D = shape[-1]
    px, ldx = _rows(x, "x", shape, 1, D, t, dev)
    pr, ldr = _rows(res, "res", shape, 1, D, t, dev) if res is not None else (None, 0)
    h = x.new_empty(shape) if h is None else h
    y = x.new_empty(shape) if y is None else y
    ph, ldh = _rows(h, "h", shape, 1, D, t, dev)
    py, ldy = _rows(y, "y", shape, 1, D, t, dev)
    s, ps = _scale(scale, (D,), dev)
    cfg = lq_norm_config(code, code, x.numel() // max(D, 1), 1, D, 0, 0, 0, eps, s)
    rc = lib().lq_norm_in(C.addressof(cfg), px, ldx, _flat(w, "w", (D,), dev), pr, ldr, ps, ph, ldh, py, ldy,
                          _raw_stream(dev))
    _chk(rc, "lq_norm_in")
    return y, h


@_layer_call
def lq_norm_out(x, w, z=None, act="silu", gate_first=False, res=None, scale=1.0, eps=1e-5, y=None):
    """Norm after a block, with its gate and the residual, over the last
    dimension of x [..., G, D] (x may be float32 beside 16-bit z, res and y):
    y = res + scale (rms(x) w act(z)), gate_first: res + scale (rms(x act(z)) w).
    w is [D] or [G, D]; scale a number or a float32 tensor [G, D].  The type of
    y is that of a given y, z or res, else x's.  Returns y.  Takes stream=."""
    t = y.dtype if y is not None else z.dtype if z is not None else res.dtype if res is not None else x.dtype
    dev, shape = x.get_device(), x.shape
    if len(shape) < 2:
        raise ValueError(f"x is [..., G, D], got {tuple(shape)}")
    G, D = shape[-2:]
    xcode, n = _dtype_of(x), G * D
    px, ldx = _rows(x, "x", shape, 2, n, x.dtype, dev)
    pz, ldz = _rows(z, "z", shape, 2, n, t, dev) if z is not None else (None, 0)
    pr, ldr = _rows(res, "res", shape, 2, n, t, dev) if res is not None else (None, 0)
    y = x.new_empty(shape, dtype=t) if y is None else y
    py, ldy = _rows(y, "y", shape, 2, n, t, dev)
    wg = w.dim() == 2
    s, ps = _scale(scale, (G, D), dev)
    cfg = lq_norm_config(_dtype_of(y), xcode, x.numel() // max(n, 1), G, D, 1 if wg else 0, _act_of(act),
                         1 if gate_first else 0, eps, s)
    rc = lib().lq_norm_out(C.addressof(cfg), px, ldx, _flat(w, "w", (G, D) if wg else (D,), dev), pz, ldz, pr, ldr, ps,
                           py, ldy, _raw_stream(dev))
    _chk(rc, "lq_norm_out")
    return y
