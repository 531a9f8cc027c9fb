"""Workload driver on one GPU: builds the initial states, optionally calibrates
the DAMP rows, and runs windowed decode steps through the C ABI.

Every numerical step runs in liblq.so kernels: the prefill that produces the
initial state uses the chunked prefill (lq_prefill; or, on request, the
FP32-state decode kernel token by token), the initial quantization uses
lq_state_init, the DAMP choice uses lq_damp_select.  torch provides device
memory, the seeded input draws (inputs.py), streams and CUDA graphs.
"""
from __future__ import annotations

import math

import torch

from . import inputs as gen
from . import lq
from .configs import ScanLayer, Workload


def gpu_prefill(wl: Workload, *, tokens: int | None = None, batch: int | None = None, stream: str = "prefill",
                chunk: int = 64, device="cuda", capture_heads=None, keep_inputs: bool = False,
                method: str = "chunked"):
    """FP32 recurrence from zero over `tokens` generator tokens on the GPU:
    `method` "chunked" runs lq_prefill on each generator chunk, "recurrent"
    the FP32-state decode kernel one token at a time.

    Returns the state [batch, H, dk, dv] (float32, no outliers yet) and, if
    capture_heads lists (b, h) pairs, those heads' inputs on the host in the
    generator's [T, B', Hk|H, ...] layout restricted to the listed batch rows.
    """
    T = wl.prefill if tokens is None else tokens
    B = wl.B if batch is None else batch
    cfg = lq.Config(B=B, H=wl.H, Hk=wl.Hk, dk=wl.dk, dv=wl.dv, gate=wl.gate, mode="fp32", r=0, n_hp_rows=0)
    S0 = torch.zeros((B, wl.H, wl.dk, wl.dv), device=device)
    st = lq.lq_state_init(cfg, S0) if method != "chunked" else None
    o = torch.empty((B, wl.H, wl.dv), device=device)
    captured = []
    bsel = None
    if capture_heads:
        bsel = torch.tensor(sorted({b for b, _ in capture_heads}), device=device)
    S = torch.zeros_like(S0)
    for c in range((T + chunk - 1) // chunk):
        n = min(chunk, T - c * chunk)
        tok = gen.token_inputs(wl, n, stream=stream, chunk=c, batch=B, device=device)
        if method == "chunked":
            lq.lq_prefill(cfg, tok["q"], tok["k"], tok["v"], tok["beta"], tok["alpha"], S0=S, S_out=S)
        else:
            for t in range(n):
                lq.lq_decode_step(st, tok["q"][t], tok["k"][t], tok["v"][t], tok["beta"][t], tok["alpha"][t], o)
        if bsel is not None:
            captured.append({k: v.index_select(1, bsel).cpu() for k, v in tok.items()})
    if st is not None:
        lq.lq_state_export_fp32(st, S)
        rc = lq.lq_get_status(st)
        if rc != lq.LQ_OK:
            raise lq.LqError(rc, "prefill")
        lq.lq_state_destroy(st)
    elif not bool(torch.isfinite(S).all()):
        raise lq.LqError(lq.LQ_ERR_NONFINITE, "prefill")
    if bsel is None:
        return S, None
    cap = {k: torch.cat([c[k] for c in captured], dim=0) for k in captured[0]}
    return S, cap


def initial_state(wl: Workload, **kw):
    S, cap = gpu_prefill(wl, **kw)
    return gen.apply_outliers(S, wl), cap


def damp_rows(wl: Workload, device="cuda") -> torch.Tensor:
    """Offline DAMP calibration on the GPU: calibration prefills (lq_prefill),
    the workload's outliers, then lq_damp_select.  Returns rows [H, P] (host)."""
    n, T = wl.calib_prefills, wl.calib_tokens
    states, _ = gpu_prefill(wl, tokens=T, batch=n, stream="calib", device=device)
    states = gen.apply_outliers(states, wl)
    gates = []
    for c in range((T + 63) // 64):
        tok = gen.token_inputs(wl, min(64, T - c * 64), stream="calib", chunk=c, batch=n, device=device)
        gates.append(tok["alpha"].reshape(-1, wl.H, wl.dk if wl.gate == "kda" else 1))
    gates = torch.cat(gates).contiguous()
    cfg = lq.Config(B=1, H=wl.H, Hk=wl.H, dk=wl.dk, dv=wl.dv, gate=wl.gate, r=wl.r,
                    power_iters=wl.K, n_hp_rows=wl.P, smoothing=wl.smoothing)
    energy = torch.zeros((wl.H, wl.dk), dtype=torch.float64, device=device)
    rows = torch.zeros((wl.H, wl.P), dtype=torch.int32, device=device)
    lq.lq_damp_select(cfg, states.contiguous(), gates, energy, rows)
    return rows.cpu()


def static_scales(wl: Workload, n: int = 8, tokens: int | None = None, device="cuda"):
    """Offline fit of fixed key-row / value-column scales (smoothing 2) on the
    GPU: n calibration prefills of the workload's prefill length (calibration
    draws, the workload's outliers), rows weighted by their decay persistence
    (lq_fit_static_scales forms it from the calibration decays: per key channel
    for KDA, one value per head for GDN).  Returns (m [H, dk], s [H, dv]) on
    the device."""
    T = wl.prefill if tokens is None else tokens
    states, _ = gpu_prefill(wl, tokens=T, batch=n, stream="calib", device=device)
    states = gen.apply_outliers(states, wl).contiguous()
    tok = gen.token_inputs(wl, min(T, 256), stream="calib", batch=n, device=device)
    gates = tok["alpha"].reshape(-1, wl.H, wl.dk if wl.gate == "kda" else 1).contiguous()
    cfg = lq.Config(B=1, H=wl.H, Hk=wl.H, dk=wl.dk, dv=wl.dv, gate=wl.gate, r=wl.r, power_iters=wl.K,
                    state_bits=wl.bits, smoothing=2)
    return lq.lq_fit_static_scales(cfg, states, gates=gates)


class WindowRunner:
    """Holds a decode state, the decode inputs of T tokens and one CUDA graph
    per window of W tokens (the W-th call also flushes)."""

    def __init__(self, wl: Workload, S0: torch.Tensor, *, mode: str = "window", hp_rows=None,
                 tokens: int | None = None, device="cuda", static=None, phases=None):
        self.wl = wl
        self.cfg = lq.Config.from_workload(wl, mode=mode)
        self.W = wl.W          # tokens per graph; in step mode every call also requantizes
        self.T = wl.T if tokens is None else tokens
        self.hp_rows = hp_rows
        if static is not None:   # fixed scales (smoothing 2): (m [H, dk], s [H, dv])
            self.st = lq.lq_state_init(self.cfg, S0.contiguous(), static_m=static[0], static_s=static[1])
        else:
            self.st = lq.lq_state_init(self.cfg, S0.contiguous(), hp_rows=hp_rows)
        # staggered windows: batch entry b ends its windows at the steps where
        # (step + phases[b]) mod W = W - 1 (lq_state_set_phases)
        self.phases = phases
        if phases is not None:
            lq.lq_state_set_phases(self.st, phases)
        self.tok = gen.token_inputs(wl, self.T, device=device)
        self.out = torch.empty((self.T, wl.B, wl.H, wl.dv), device=device)
        self.graphs = {}

    @property
    def n_windows(self) -> int:
        return self.T // self.W

    def step_call(self, t: int):
        tk = self.tok
        lq.lq_decode_step(self.st, tk["q"][t], tk["k"][t], tk["v"][t], tk["beta"][t], tk["alpha"][t], self.out[t])

    def run_window_eager(self, w: int):
        for t in range(w * self.W, (w + 1) * self.W):
            self.step_call(t)

    def capture(self):
        """One graph per window slot; replays must start at a window boundary.
        The warm-up runs window 0 eagerly: with phases it holds every entry's
        shorter first window, and the graphs then hold full windows only."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.run_window_eager(0)          # warm the launch path before capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for w in range(self.n_windows):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.run_window_eager(w)
            self.graphs[w] = g
        torch.cuda.synchronize()

    def replay(self, w: int):
        self.graphs[w % self.n_windows].replay()


def scan_weights(sl: ScanLayer, dtype=torch.bfloat16, device="cuda") -> dict:
    """Seeded weights of a scan layer: the two projections in the activations'
    type, everything else float32.  The steps' bias is the inverse softplus of
    steps log-uniform in [dt_lo, dt_hi], the decays' rates A uniform in -[1, 16]."""
    g = torch.Generator(device=device).manual_seed(sl.seed)
    randn = lambda *s: torch.randn(s, generator=g, device=device)   # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=device)     # noqa: E731
    step = torch.exp(math.log(sl.dt_lo) + rand(sl.H) * math.log(sl.dt_hi / sl.dt_lo))
    return {"w_norm": 1 + 0.1 * randn(sl.d),
            "w_in": (randn(sl.d, sl.proj) * sl.d ** -0.5).to(dtype),
            "w_conv": randn(sl.conv, sl.K) * sl.K ** -0.5, "b_conv": 0.1 * randn(sl.conv),
            "A": -(1 + 15 * rand(sl.H)), "D": torch.ones(sl.H, device=device),
            "dt_bias": step + torch.log(-torch.expm1(-step)),
            "w_gate": 1 + 0.1 * randn(sl.dv),
            "w_out": (randn(sl.inner, sl.d) * sl.inner ** -0.5).to(dtype)}


class ScanRunner:
    """One selective-scan layer for a batch of B sequences, prompts and single
    tokens: norm with the residual (lq_norm_in), input projection, short
    convolution (lq_conv_*), scan (lq_ssm_*), norm of each head's outputs and then
    the gate (lq_norm_out), output projection.  The projections are plain library products; all else
    runs in liblq.so.  Holds the sequences' convolution windows and states."""

    def __init__(self, sl: ScanLayer, B: int, dtype=torch.bfloat16, device="cuda", weights=None):
        self.sl, self.B, self.dtype = sl, B, dtype
        self.w = scan_weights(sl, dtype, device) if weights is None else weights
        self.window = torch.zeros((B, sl.K - 1, sl.conv), dtype=dtype, device=device)
        self.state = torch.zeros((B, sl.H, sl.dk, sl.dv), device=device)
        self.graph = None

    def _split(self, p: torch.Tensor):
        """z, convolution inputs and steps: columns of the projection."""
        n, c = self.sl.inner, self.sl.conv
        return p[..., :n].unflatten(-1, (self.sl.H, self.sl.dv)), p[..., n:n + c], p[..., n + c:]

    def _heads(self, xbc: torch.Tensor):
        n, gk = self.sl.inner, self.sl.G * self.sl.dk
        return (xbc[..., :n].unflatten(-1, (self.sl.H, self.sl.dv)),
                xbc[..., n:n + gk].unflatten(-1, (self.sl.G, self.sl.dk)),
                xbc[..., n + gk:].unflatten(-1, (self.sl.G, self.sl.dk)))

    def prompt(self, x: torch.Tensor, res=None, cu=None):
        """Tokens of all sequences, x [rows, d] with cu or [T, B, d], from the
        windows and states held, which move on.  Returns (block output,
        residual): the next block's norm adds them.  Output rows of no sequence
        (before cu[0], from cu[B] on) hold nothing in particular."""
        sl, w = self.sl, self.w
        u, h = lq.lq_norm_in(x, w["w_norm"], res=res, scale=sl.scale, eps=sl.eps)
        z, xbc, dt = self._split(u @ w["w_in"])
        xbc, _ = lq.lq_conv_prefill(xbc, w["w_conv"], w["b_conv"], state0=self.window, state_out=self.window, cu=cu)
        xs, Bm, Cm = self._heads(xbc)
        y, _ = lq.lq_ssm_prefill(xs, dt, w["A"], Bm, Cm, D=w["D"], dt_bias=w["dt_bias"], S0=self.state,
                                 S_out=self.state, cu=cu)
        y = lq.lq_norm_out(y, w["w_gate"], z=z, eps=sl.eps, y=y)
        return y.flatten(-2) @ w["w_out"], h

    def step(self, x: torch.Tensor, res=None):
        """One token of every sequence, x [B, d]."""
        sl, w = self.sl, self.w
        u, h = lq.lq_norm_in(x, w["w_norm"], res=res, scale=sl.scale, eps=sl.eps)
        z, xbc, dt = self._split(u @ w["w_in"])
        xs, Bm, Cm = self._heads(lq.lq_conv_step(self.window, xbc, w["w_conv"], w["b_conv"]))
        y = lq.lq_ssm_step(self.state, xs, dt, w["A"], Bm, Cm, D=w["D"], dt_bias=w["dt_bias"])
        y = lq.lq_norm_out(y, w["w_gate"], z=z, eps=sl.eps, y=y)
        return y.flatten(-2) @ w["w_out"], h

    def capture(self):
        """A CUDA graph of one step on fixed buffers: fill x_in (and res_in), call
        replay(), read the returned (out, residual)."""
        with torch.cuda.device(self.window.device):   # its streams are the current device's otherwise
            keep = self.window.clone(), self.state.clone()
            self.x_in = torch.zeros((self.B, self.sl.d), dtype=self.dtype, device=self.window.device)
            self.res_in = torch.zeros_like(self.x_in)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.step(self.x_in, self.res_in)      # warm the launch path before capture
            torch.cuda.current_stream().wait_stream(s)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self.step(self.x_in, self.res_in)
            self.window.copy_(keep[0])
            self.state.copy_(keep[1])

    def replay(self):
        self.graph.replay()
        return self.out
