"""The recurrent layer's operators from their definitions in 64 bits, one
sequence and one token at a time, with the magnitude sums their rounding
bounds are proportional to.  Plain torch on whatever device the inputs are."""
import torch

U = 2.0 ** -24            # unit roundoff of float32


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half a step of dtype's smallest values (below its normal range)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def parts(x, cu):
    """Index tuples of each sequence's rows: packed by cu, else time-major."""
    if cu is None:
        return [(slice(None), b) for b in range(x.shape[1])]
    c = cu.tolist()
    return [(slice(a, b),) for a, b in zip(c, c[1:])]


def silu(v):
    return v * torch.sigmoid(v)


def conv(x, w, bias, act, state, cu):
    """(y, new windows, magnitude of the sums)."""
    K, ch = w.shape[1], w.shape[0]
    B = x.shape[1] if cu is None else cu.numel() - 1
    x64, w64 = x.double(), w.double()
    past = torch.zeros((B, K - 1, ch), dtype=torch.float64, device=x.device) if state is None else state.double()
    y = torch.full(x.shape, float("nan"), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    last = []
    for b, p in enumerate(parts(x, cu)):
        line = torch.cat([past[b], x64[p]])
        n = line.shape[0] - (K - 1)
        out = torch.zeros((n, ch), dtype=torch.float64, device=x.device)
        if bias is not None:
            out += bias.double()
        m = out.abs()
        for j in range(K):
            out += line[j:j + n] * w64[:, j]
            m += (line[j:j + n] * w64[:, j]).abs()
        y[p] = silu(out) if act == "silu" else out
        mag[p] = m
        last.append(line[n:])
    return y, torch.stack(last), mag


def ssm(x, dt, A, Bm, Cm, D, dt_bias, softplus, S0, cu):
    """(y, S, magnitude of y's sums, magnitude of S's sums, longest sequence)."""
    H, dv = x.shape[-2:]
    G, dk = Bm.shape[-2:]
    dev = x.device
    B = x.shape[1] if cu is None else cu.numel() - 1
    of = torch.arange(H, device=dev) * G // H
    f64 = torch.float64
    x, dt, Bm, Cm, A = x.to(f64), dt.to(f64), Bm.to(f64), Cm.to(f64), A.to(f64)
    D = torch.zeros(H, dtype=f64, device=dev) if D is None else D.to(f64)
    if dt_bias is not None:
        dt = dt + dt_bias.to(f64)
    if softplus:
        dt = torch.logaddexp(dt, torch.zeros_like(dt))
    S = torch.zeros((B, H, dk, dv), dtype=f64, device=dev) if S0 is None else S0.to(f64).clone()
    M = S.abs()
    y, my = torch.full(x.shape, float("nan"), dtype=f64, device=dev), torch.zeros(x.shape, dtype=f64, device=dev)
    longest = 0
    for b, p in enumerate(parts(x, cu)):
        xs, ds, bs, cs = x[p], dt[p], Bm[p][:, of], Cm[p][:, of]
        longest = max(longest, xs.shape[0])
        ys, ms = torch.empty_like(xs), torch.empty_like(xs)
        for t in range(xs.shape[0]):
            a = torch.exp(ds[t] * A)[:, None, None]
            add = bs[t][:, :, None] * (ds[t][:, None] * xs[t])[:, None, :]
            S[b] = a * S[b] + add
            M[b] = a * M[b] + add.abs()
            ys[t] = (S[b] * cs[t][:, :, None]).sum(1) + D[:, None] * xs[t]
            ms[t] = (M[b] * cs[t][:, :, None].abs()).sum(1) + (D[:, None] * xs[t]).abs()
        y[p], my[p] = ys, ms
    return y, S, my, M, longest


def norm_in(x, w, res, scale, eps):
    h = scale * x.double() + (0 if res is None else res.double())
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double(), h


def norm_out(x, w, z, act, first, res, scale, eps):
    x = x.double()
    gate = 1.0 if z is None else (silu(z.double()) if act == "silu" else torch.sigmoid(z.double()))
    u = x * gate if first else x
    y = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * w.double()
    y = y if first else y * gate
    return scale * y + (0 if res is None else res.double())
