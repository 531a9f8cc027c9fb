"""What the recurrent layer's operators cost: the short causal convolution, the selective
state-space scan, and the norms before and after a block -- for prompts and single tokens.

A prompt batch is either packed (sequences of their own lengths in consecutive rows, `cu`
the B+1 row offsets) or time-major with equal lengths (row t*B + b).  `run` computes one
pass in elementary torch operations (own = False) or through the package (own = True);
`exact` walks the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_CHUNK = 128      # tokens per chunk of the plain scan


def listed():
    return [
        # the layer's convolution over a batch of prompts of mixed lengths (x, B and C of 16 heads of 128)
        {"name": "conv_prompts_packed", "op": "conv", "dtype": "bf16", "B": 48, "rows": 32768, "packed": True,
         "C": 2304, "K": 4},
        # one token of 1024 sequences: q, k and v of 16 heads of 128
        {"name": "conv_step_b1024", "op": "conv_step", "dtype": "bf16", "B": 1024, "C": 6144, "K": 4},
        # one long prompt: few heads, the work is along the sequence
        {"name": "ssm_one_long_prompt", "op": "ssm", "dtype": "bf16", "B": 1, "rows": 16384, "packed": True,
         "H": 32, "G": 1, "dk": 128, "dv": 64},
        # a batch of prompts of mixed lengths, wide heads, two groups of B and C
        {"name": "ssm_prompts_packed", "op": "ssm", "dtype": "bf16", "B": 40, "rows": 16384, "packed": True,
         "H": 32, "G": 2, "dk": 128, "dv": 128},
        # a short time-major prompt of two sequences, the tiny workload's heads, in the framework's own type
        {"name": "ssm_short_f32", "op": "ssm", "dtype": "f32", "B": 2, "rows": 100, "packed": False,
         "H": 2, "G": 2, "dk": 64, "dv": 64},
        # odd row counts and heads
        {"name": "ssm_odd_f16", "op": "ssm", "dtype": "f16", "B": 7, "rows": 3001, "packed": True,
         "H": 6, "G": 3, "dk": 64, "dv": 128},
        # a decode step of a large batch: the states stream through
        {"name": "ssm_step_b256", "op": "ssm_step", "dtype": "bf16", "B": 256, "H": 32, "G": 1, "dk": 128, "dv": 128},
        # a decode step of one sequence: latency
        {"name": "ssm_step_b1", "op": "ssm_step", "dtype": "bf16", "B": 1, "H": 16, "G": 1, "dk": 128, "dv": 64},
        # the norm before a block over a prompt batch, residual carried along
        {"name": "norm_in_prompts", "op": "norm_in", "dtype": "bf16", "rows": 16384, "D": 4096, "vec": False},
        # the same for one token
        {"name": "norm_in_one_row", "op": "norm_in", "dtype": "f32", "rows": 1, "D": 2048, "vec": True},
        # the gated norm of the heads' f32 outputs in a decode step
        {"name": "norm_out_decode", "op": "norm_out", "dtype": "bf16", "x_f32": True, "rows": 1024, "G": 16, "D": 128,
         "first": False, "res": False},
        # gate first, one statistic over the whole width, scaled onto the residual
        {"name": "norm_out_prompts", "op": "norm_out", "dtype": "f16", "x_f32": False, "rows": 16384, "G": 1,
         "D": 2048, "first": True, "res": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm_step", "norm_in", "norm_out"])
    c = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16", "bf16"])}
    if op in ("conv", "ssm"):
        c["packed"] = rng.random() < 0.6
        c["B"] = _log_int(rng, 1, 64)
        rows = max(c["B"], _log_int(rng, 1, 16384))
        c["rows"] = rows if c["packed"] else rows // c["B"] * c["B"]
    if op == "conv":
        c["C"] = _log_int(rng, 1, 2304) if c["dtype"] == "f32" else _log_int(rng, 1, 4096)
        c["K"] = rng.choice([2, 3, 4, 4])
    elif op == "conv_step":
        c["B"], c["C"], c["K"] = _log_int(rng, 1, 512), _log_int(rng, 1, 6144), rng.choice([2, 3, 4, 4])
    elif op in ("ssm", "ssm_step"):
        if op == "ssm_step":
            c["B"] = _log_int(rng, 1, 256)
        elif c["dtype"] != "bf16":
            c["rows"] = max(c["B"], c["rows"] // 4 // c["B"] * c["B"])
        c["G"] = rng.choice([1, 1, 2, 3, 4])
        c["H"] = c["G"] * _log_int(rng, 1, 32 // c["G"])
        c["dk"], c["dv"] = rng.choice([64, 128]), rng.choice([64, 128])
    elif op == "norm_in":
        c["rows"], c["D"], c["vec"] = _log_int(rng, 1, 8192), _log_int(rng, 16, 4096), rng.random() < 0.5
    else:
        c["x_f32"] = rng.random() < 0.5
        c["rows"], c["G"], c["D"] = _log_int(rng, 1, 8192), rng.choice([1, 1, 2, 8, 16]), 0
        c["D"] = _log_int(rng, 16, 4096 // c["G"])
        c["first"], c["res"] = rng.random() < 0.5, rng.random() < 0.5
    return c


# -- inputs ----------------------------------------------------------------------------

def _offsets(case, seed):
    """B+1 row offsets of a packed batch: mixed lengths of at least one token, about three times apart."""
    r = random.Random(seed * 7919 + case["rows"])
    w = [math.exp(r.uniform(-0.6, 0.6)) for _ in range(case["B"])]
    spare, total = case["rows"] - case["B"], sum(w)
    at, acc = [0], 0.0
    for b, x in enumerate(w):
        acc += x
        at.append(b + 1 + int(round(spare * acc / total)))
    return at


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _rows_shape(case, *tail):
    return (case["rows"], *tail) if case["packed"] else (case["rows"] // case["B"], case["B"], *tail)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    s = {"case": case}
    if case.get("packed"):
        s["at"] = _offsets(case, seed)
        s["cu"] = torch.tensor(s["at"], dtype=torch.int32, device="cuda")
    if op in ("conv", "conv_step"):
        C, K = case["C"], case["K"]
        lead = _rows_shape(case) if op == "conv" else (case["B"],)
        s["proj"] = _normal(g, (*lead, C + 64), dt)      # the input projection: the convolution reads its first C columns
        s["x"] = s["proj"][..., :C]
        s["w"] = _normal(g, (C, K), scale=K ** -0.5)
        s["bias"] = _normal(g, (C,), scale=0.1)
        s["state"] = _normal(g, (case["B"], K - 1, C), dt)
    elif op in ("ssm", "ssm_step"):
        H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
        lead = _rows_shape(case) if op == "ssm" else (case["B"],)
        # x, B and C are the columns of the convolution's output, dt those of the projection
        s["xbc"] = torch.nn.functional.silu(_normal(g, (*lead, H * dv + 2 * G * dk))).to(dt)
        s["x"] = s["xbc"][..., : H * dv].unflatten(-1, (H, dv))
        s["Bm"] = s["xbc"][..., H * dv: H * dv + G * dk].unflatten(-1, (G, dk))
        s["Cm"] = s["xbc"][..., H * dv + G * dk:].unflatten(-1, (G, dk))
        s["dt"] = _normal(g, (*lead, H), dt)
        s["A"] = -(1 + 15 * torch.rand((H,), generator=g, device="cuda"))
        step = torch.exp(torch.rand((H,), generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1 + _normal(g, (H,), scale=0.1)
        s["S"] = _normal(g, (case["B"], H, dk, dv), scale=0.3)
    elif op == "norm_in":
        R, D = case["rows"], case["D"]
        s["x"], s["res"] = _normal(g, (R, D), dt), _normal(g, (R, D), dt, 3.0)
        s["w"] = 1 + _normal(g, (D,), scale=0.2)
        s["scale"] = 0.2 + 0.1 * torch.rand((D,), generator=g, device="cuda") if case["vec"] else 0.22
    else:
        R, G, D = case["rows"], case["G"], case["D"]
        s["x"] = _normal(g, (R, G, D), torch.float32 if case["x_f32"] else dt, 0.5)
        s["z"] = _normal(g, (R, G, D), dt)
        s["w"] = 1 + _normal(g, (D,) if G > 1 else (1, D), scale=0.2)
        s["res"] = _normal(g, (R, G, D), dt, 3.0) if case["res"] else None
        s["scale"] = 0.22 if case["res"] else 1.0
    return s


def prepare(case, seed):
    return _inputs(case, seed)


def _lq():
    from quantized_recurrent_state_lq_b200 import lq
    return lq


# -- plain forms ------------------------------------------------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _windows(s):
    """Each row's last K inputs [.., C, K] and each sequence's next window [B, K-1, C]."""
    x, state, K = s["x"], s["state"], s["case"]["K"]
    if not s["case"]["packed"]:
        ext = torch.cat([state.transpose(0, 1), x])
        return ext.unfold(0, K, 1), ext[ext.shape[0] - (K - 1):].transpose(0, 1)
    cu, R = s["cu"].long(), x.shape[0]
    B = state.shape[0]
    seq = torch.repeat_interleave(torch.arange(B, device=x.device), cu[1:] - cu[:-1], output_size=R)
    pos = torch.arange(R, device=x.device) + (seq + 1) * (K - 1)
    back = torch.arange(K - 1, device=x.device)
    head = (cu[:-1] + torch.arange(B, device=x.device) * (K - 1))[:, None] + back
    ext = torch.empty((R + B * (K - 1), x.shape[1]), dtype=x.dtype, device=x.device)
    ext[pos] = x
    ext[head] = state
    return ext.unfold(0, K, 1)[pos - (K - 1)], ext[head + (cu[1:] - cu[:-1])[:, None]]


def _conv(s):
    win, last = _windows(s)
    y = (win.float() * s["w"]).sum(-1) + s["bias"]
    return [_silu(y).to(s["x"].dtype), last.contiguous()]


def _conv_step(s):
    win = torch.cat([s["state"], s["x"][:, None]], 1)
    y = (win.float() * s["w"].t()).sum(1) + s["bias"]
    s["state"].copy_(win[:, 1:])
    return [_silu(y).to(s["x"].dtype), s["state"]]


def _segments(g):
    """e^{g_i - g_j} for j <= i along the last axis of g (64 bits), else 0."""
    n = g.shape[-1]
    low = torch.ones((n, n), dtype=torch.bool, device=g.device).tril()
    return torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~low, -math.inf)).float()


def _chunked(x, d, A, Bm, Cm, S0):
    """The scan of [B, T, H, ..] inputs chunk by chunk as products; tokens with d = 0 change nothing."""
    B, T, H, P = x.shape
    Q = min(_CHUNK, T)
    pad = -T % Q
    x, d, Bm, Cm = (torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, pad)) for v in (x, d, Bm, Cm))
    x, d, Bm, Cm = (v.unflatten(1, (-1, Q)) for v in (x, d, Bm, Cm))
    r = H // Bm.shape[3]
    g = torch.cumsum((d.double() * A.double()).permute(0, 3, 1, 2), -1)                  # [B, H, c, Q]
    xd = x * d[..., None]
    pair = torch.einsum("bcqgn,bcsgn->bgcqs", Cm, Bm).repeat_interleave(r, 1)
    y = torch.einsum("bhcqs,bcshp->bcqhp", pair * _segments(g), xd)
    end = torch.exp(g[..., -1:] - g).float()                                             # [B, H, c, Q]
    heads = lambda v: v.repeat_interleave(r, 3)                                          # noqa: E731
    new = torch.einsum("bcshn,bcshp->bchnp", heads(Bm), xd * end.permute(0, 2, 3, 1)[..., None])
    new = torch.cat([S0[:, None], new], 1)                                               # [B, c + 1, H, N, P]
    total = torch.nn.functional.pad(torch.cumsum(g[..., -1], -1), (1, 0))
    S = torch.einsum("bhij,bjhnp->bihnp", _segments(total), new)
    y = y + torch.einsum("bcqhn,bchnp->bcqhp", heads(Cm) * torch.exp(g).float().permute(0, 2, 3, 1)[..., None], S[:, :-1])
    return y.flatten(1, 2)[:, :T], S[:, -1]


def _ssm(s):
    case = s["case"]
    x, Bm, Cm = (s[k].float() for k in ("x", "Bm", "Cm"))
    d = _softplus(s["dt"].float() + s["dt_bias"])
    if case["packed"]:
        cu, R, B = s["cu"].long(), case["rows"], case["B"]
        n = cu[1:] - cu[:-1]
        seq = torch.repeat_interleave(torch.arange(B, device=x.device), n, output_size=R)
        at = torch.arange(R, device=x.device) - cu[seq]
        T = max(b - a for a, b in zip(s["at"], s["at"][1:]))

        def spread(v):
            out = torch.zeros((B, T, *v.shape[1:]), device=v.device)
            out[seq, at] = v
            return out
        y, S = _chunked(spread(x), spread(d), s["A"], spread(Bm), spread(Cm), s["S"])
        y = y[seq, at]
    else:
        y, S = _chunked(*(v.transpose(0, 1) for v in (x, d)), s["A"], *(v.transpose(0, 1) for v in (Bm, Cm)), s["S"])
        y = y.transpose(0, 1)
    y = y + s["D"][:, None] * x
    return [y.to(s["x"].dtype).contiguous(), S]


def _ssm_step(s):
    x = s["x"].float()
    d = _softplus(s["dt"].float() + s["dt_bias"])
    r = x.shape[1] // s["Bm"].shape[1]
    Bm, Cm = (s[k].float().repeat_interleave(r, 1) for k in ("Bm", "Cm"))
    S = s["S"]
    S.mul_(torch.exp(d * s["A"])[..., None, None]).add_(Bm[..., :, None] * (d[..., None] * x)[..., None, :])
    y = (S * Cm[..., :, None]).sum(2) + s["D"][:, None] * x
    return [y.to(s["x"].dtype), S]


_EPS = 1e-5


def _rms(u, w):
    return u * torch.rsqrt(u.square().mean(-1, keepdim=True) + _EPS) * w


def _norm_in(s):
    h = s["res"].float() + s["scale"] * s["x"].float()
    return [_rms(h, s["w"]).to(s["x"].dtype), h.to(s["x"].dtype)]


def _norm_out(s):
    x, gate = s["x"].float(), _silu(s["z"].float())
    y = _rms(x * gate, s["w"]) if s["case"]["first"] else _rms(x, s["w"]) * gate
    if s["res"] is not None:
        y = s["res"].float() + s["scale"] * y
    return y.to(s["z"].dtype)


_PLAIN = {"conv": _conv, "conv_step": _conv_step, "ssm": _ssm, "ssm_step": _ssm_step, "norm_in": _norm_in,
          "norm_out": _norm_out}


def run(s):
    op = s["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    lq = _lq()
    if op == "conv":
        return list(lq.lq_conv_prefill(s["x"], s["w"], s["bias"], act="silu", state0=s["state"], cu=s.get("cu")))
    if op == "conv_step":
        return [lq.lq_conv_step(s["state"], s["x"], s["w"], s["bias"], act="silu"), s["state"]]
    if op == "ssm":
        return list(lq.lq_ssm_prefill(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["dt_bias"],
                                      S0=s["S"], cu=s.get("cu")))
    if op == "ssm_step":
        return [lq.lq_ssm_step(s["S"], s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["D"], dt_bias=s["dt_bias"]),
                s["S"]]
    if op == "norm_in":
        return list(lq.lq_norm_in(s["x"], s["w"], res=s["res"], scale=s["scale"], eps=_EPS))
    return lq.lq_norm_out(s["x"], s["w"], z=s["z"], act="silu", gate_first=s["case"]["first"], res=s["res"],
                          scale=s["scale"], eps=_EPS)


# -- cost and definition ------------------------------------------------------------------

def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op in ("conv", "conv_step"):
        R = case["rows"] if op == "conv" else case["B"]
        C, K = case["C"], case["K"]
        return {"bytes": 2 * R * C * e + 2 * case["B"] * (K - 1) * C * e + 4 * C * (K + 1), "flops": 2 * R * C * K}
    if op in ("ssm", "ssm_step"):
        R = case["rows"] if op == "ssm" else case["B"]
        H, G, dk, dv = case["H"], case["G"], case["dk"], case["dv"]
        row = 2 * H * dv + 2 * G * dk + H
        return {"bytes": R * row * e + 2 * case["B"] * H * dk * dv * 4, "flops": 5 * R * H * dk * dv}
    if op == "norm_in":
        n = case["rows"] * case["D"]
        return {"bytes": 4 * n * e + 4 * case["D"], "flops": 6 * n}
    n = case["rows"] * case["G"] * case["D"]
    return {"bytes": n * ((4 if case["x_f32"] else e) + (3 if case["res"] else 2) * e), "flops": 8 * n}


def _d64(s, *names):
    return (s[k].double() for k in names)


def _exact_rows(case, s):
    """Per step t: the rows it touches and the sequences they belong to."""
    if not case["packed"]:
        T, B = case["rows"] // case["B"], case["B"]
        every = torch.arange(B, device="cuda")
        for t in range(T):
            yield t * B + every, every
        return
    at = np.array(s["at"])
    n = np.diff(at)
    order = np.argsort(-n, kind="stable")          # the longest first: the live ones are a prefix
    live = np.searchsorted(-n[order], -np.arange(1, n.max() + 1), side="right")
    starts = torch.from_numpy(at[:-1][order].copy()).cuda()
    order = torch.from_numpy(order.copy()).cuda()
    for t, m in enumerate(live.tolist()):
        yield starts[:m] + t, order[:m]


def _exact_scan(case, s, rows):
    H, G = case["H"], case["G"]
    x, Bm, Cm, dt, S, A, D = _d64(s, "x", "Bm", "Cm", "dt", "S", "A", "D")
    R = case["rows"] if case["op"] == "ssm" else case["B"]
    x, dt = x.reshape(R, H, -1), dt.reshape(R, H)
    of = torch.arange(H, device="cuda") * G // H
    Bm, Cm = Bm.reshape(R, G, -1), Cm.reshape(R, G, -1)
    d = torch.logaddexp(dt + s["dt_bias"].double(), torch.zeros_like(dt))
    keep = torch.exp(d * A)
    y = torch.empty_like(x)
    for r, b in rows:
        cur = S[b] * keep[r][..., None, None]
        cur = torch.addcmul(cur, Bm[r][:, of][..., :, None], (d[r][..., None] * x[r])[..., None, :])
        y[r] = torch.matmul(Cm[r][:, of][..., None, :], cur)[..., 0, :] + D[:, None] * x[r]
        S[b] = cur
    return [y.reshape(s["x"].shape), S]


def exact(case, seed):
    op = case["op"]
    s = _inputs(case, seed)
    if op == "ssm":
        return _exact_scan(case, s, _exact_rows(case, s))
    if op == "ssm_step":
        every = torch.arange(case["B"], device="cuda")
        return _exact_scan(case, s, [(every, every)])
    if op in ("conv", "conv_step"):
        x, w, bias, past = _d64(s, "x", "w", "bias", "state")
        B, C, K = case["B"], case["C"], case["K"]
        if op == "conv_step":
            parts = [x[b:b + 1] for b in range(B)]
        elif case["packed"]:
            parts = [x[a:b] for a, b in zip(s["at"], s["at"][1:])]
        else:
            parts = [x[:, b] for b in range(B)]
        outs, last = [], []
        for b, part in enumerate(parts):
            line = torch.cat([past[b], part])
            out = bias.expand(part.shape[0], C).clone()
            for j in range(K):
                out += line[j:j + part.shape[0]] * w[:, j]
            outs.append(out * torch.sigmoid(out))
            last.append(line[line.shape[0] - (K - 1):])
        y = torch.stack(outs, 1) if op == "conv" and not case["packed"] else torch.cat(outs)
        return [y, torch.stack(last)]
    if op == "norm_in":
        x, res, w = _d64(s, "x", "res", "w")
        h = res + (s["scale"].double() if case["vec"] else float(np.float32(s["scale"]))) * x
        return [h / torch.sqrt((h * h).mean(-1, keepdim=True) + _EPS) * w, h]
    x, z, w = _d64(s, "x", "z", "w")
    gate = z * torch.sigmoid(z)
    u = x * gate if case["first"] else x
    y = u / torch.sqrt((u * u).mean(-1, keepdim=True) + _EPS) * w
    y = y if case["first"] else y * gate
    if case["res"]:
        y = s["res"].double() + float(np.float32(s["scale"])) * y
    return y
