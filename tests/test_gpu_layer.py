"""GPU parity of the recurrent layer's operators (convolution, selective scan,
norms) against their definitions in 64 bits.

Tolerances, per element: one rounding to the output's type (half a step of its
value) plus the FP32 error of the sum behind it, a multiple of 2^-24 times the
sum of the magnitudes of its terms:
  conv   K + 1 roundings of the products and sums;
  scan   every term passes at most n = T decays, each rounded twice and with an
         exponential good to a few ulps: Higham and Mary's probabilistic bound
         lambda sqrt(n) u per path (lambda = 8) with 3 roundings a step, plus
         the split products of the chunk form (2^-21 of a term) and dk-term sums;
  norm   sqrt(D) of the statistic (probabilistic) and a few roundings.
SiLU and sigmoid take the hardware exponential for 16-bit outputs: 2^-18
relative for the arguments drawn here (|v| < 30: the argument's rounding moves
the exponential by |v| 2^-23), and at f32 the library's (2^-21)."""
import math

import pytest
import torch

from quantized_recurrent_state_lq_b200 import configs, inputs as gen, lq, runner
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
ids = lambda v: str(v).replace("torch.", "")   # noqa: E731


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _cu(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _close(got, want, tol, what):
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got.double() - want).abs() / tol
    worst = off.max().item() if off.numel() else 0.0
    print(f"{what}: {worst:.3f} of the tolerance")
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance at {int(off.argmax())}"


def _act_rel(dtype, act):
    return 0.0 if act is None else (2.0 ** -21 if dtype == F32 else 2.0 ** -18)


# -- convolution ------------------------------------------------------------------

def _conv_tol(y, mag, dtype, K, act):
    # |silu'| <= 1.1: the sum's error passes through
    return (R.half_step(dtype) * (1 + 1e-3) + _act_rel(dtype, act)) * y.abs() + 1.1 * (K + 2) * R.U * mag + R.tiny(dtype)


def _check_conv(x, w, bias, act, state, cu, what):
    y, win = lq.lq_conv_prefill(x, w, bias, act=act, state0=state, cu=cu)
    ry, rw, mag = R.conv(x, w, bias, act, state, cu)
    _close(y, ry, _conv_tol(ry, mag, x.dtype, w.shape[1], act), what)
    assert torch.equal(win.double(), rw), f"{what}: window"


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("C", [1, 37, 64, 1030, 2304])
def test_conv_packed(dtype, K, C):
    """Sequences of 0, 1, 2, 3 tokens and around the pieces' ends, windows given."""
    _gpu()
    g = _gen(C * 10 + K)
    cu = _cu([0, 1, 2, 3, 64, 0, 65, 63, 130, 1])
    n = int(cu[-1])
    x = _randn(g, (n, C + 24), dtype)[:, 8:8 + C]          # columns of a wider tensor
    w, bias = _randn(g, (C, K)), _randn(g, (C,))
    state = _randn(g, (10, K - 1, C), dtype)
    _check_conv(x, w, bias, "silu", state, cu, f"conv {ids(dtype)} K{K} C{C}")
    _check_conv(x, w, None, None, None, cu, f"conv plain {ids(dtype)} K{K} C{C}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [0, 1, 2, 3, 64, 100])
def test_conv_time_major(dtype, T):
    _gpu()
    g = _gen(T)
    x, w, bias = _randn(g, (T, 3, 80), dtype), _randn(g, (80, 4)), _randn(g, (80,))
    state = _randn(g, (3, 3, 80), dtype)
    _check_conv(x, w, bias, "silu", state, None, f"conv time-major {ids(dtype)} T{T}")


def test_conv_in_place_window_and_pieces_match_one_call():
    """Two calls with the window carried in place equal one call, bit for bit."""
    _gpu()
    g = _gen(5)
    x, w, bias = _randn(g, (150, 2, 96), BF16), _randn(g, (96, 4)), _randn(g, (96,))
    state = _randn(g, (2, 3, 96), BF16)
    one, last = lq.lq_conv_prefill(x, w, bias, state0=state)
    s = state.clone()
    got = []
    for a, b in ((0, 1), (1, 3), (3, 70), (70, 150)):
        y, _ = lq.lq_conv_prefill(x[a:b], w, bias, state0=s, state_out=s)
        got.append(y)
    assert torch.equal(torch.cat(got), one) and torch.equal(s, last)
    s = state.clone()
    for t in range(150):
        assert torch.equal(lq.lq_conv_step(s, x[t], w, bias), one[t]), t
    assert torch.equal(s, last)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("B,C,K", [(1, 2304, 4), (3, 37, 2), (130, 200, 3)])
def test_conv_step(dtype, B, C, K):
    _gpu()
    g = _gen(B)
    x = _randn(g, (B, C + 8), dtype)[:, :C]
    w, bias, state = _randn(g, (C, K)), _randn(g, (C,)), _randn(g, (B, K - 1, C), dtype)
    ry, rw, mag = R.conv(x[None], w, bias, "silu", state, None)
    y = lq.lq_conv_step(state, x, w, bias)
    _close(y, ry[0], _conv_tol(ry[0], mag[0], dtype, K, "silu"), f"conv step {ids(dtype)}")
    assert torch.equal(state.double(), rw)


def test_conv_rows_outside_the_sequences_stay():
    """Rows before cu[0] and from cu[B] on are not written."""
    _gpu()
    g = _gen(1)
    x, w = _randn(g, (40, 64), BF16), _randn(g, (64, 4))
    cu = torch.tensor([5, 9, 9, 30], dtype=torch.int32, device="cuda")
    y = torch.full((40, 64), 7.0, dtype=BF16, device="cuda")
    lq.lq_conv_prefill(x, w, y=y, cu=cu)
    assert (y[:5] == 7).all() and (y[30:] == 7).all()
    ry, _, mag = R.conv(x, w, None, "silu", None, cu)
    _close(y[5:30], ry[5:30], _conv_tol(ry, mag, BF16, 4, "silu")[5:30], "conv inner rows")


# -- selective scan ---------------------------------------------------------------

def _ssm_inputs(seed, lead, B, H, G, dk, dv, dtype, pad=8):
    g = _gen(seed)
    wide = _randn(g, (*lead, pad + H * dv + 2 * G * dk), scale=0.7).to(dtype)
    x = wide[..., pad:pad + H * dv].unflatten(-1, (H, dv))
    Bm = wide[..., pad + H * dv:pad + H * dv + G * dk].unflatten(-1, (G, dk))
    Cm = wide[..., pad + H * dv + G * dk:].unflatten(-1, (G, dk))
    dt = _randn(g, (*lead, H), dtype)
    A = -(1 + 15 * torch.rand((H,), generator=g, device="cuda"))
    step = torch.exp(torch.rand((H,), generator=g, device="cuda") * math.log(100) + math.log(1e-3))
    return {"x": x, "dt": dt, "A": A, "Bm": Bm, "Cm": Cm, "D": 1 + _randn(g, (H,), scale=0.1),
            "dt_bias": step + torch.log(-torch.expm1(-step)), "S0": _randn(g, (B, H, dk, dv), scale=0.3)}


def _ssm_tol(y, S, my, mS, n, dtype, dk):
    k = (24 * math.sqrt(max(n, 1)) + 8 * math.sqrt(dk) + 64) * R.U
    return R.half_step(dtype) * (1 + 1e-3) * y.abs() + k * my + R.tiny(dtype), k * mS + 1e-30


def _check_ssm(v, cu, what, softplus=True, **kw):
    a = {**v, **kw}
    dtype, dk = v["x"].dtype, v["Bm"].shape[-1]
    y, S = lq.lq_ssm_prefill(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], D=a["D"], dt_bias=a["dt_bias"],
                             softplus=softplus, S0=a["S0"], cu=cu)
    ry, rS, my, mS, n = R.ssm(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], a["D"], a["dt_bias"], softplus, a["S0"], cu)
    ty, tS = _ssm_tol(ry, rS, my, mS, n, dtype, dk)
    _close(y, ry, ty, f"{what} y")
    _close(S, rS, tS, f"{what} S")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("H,G,dk,dv", [(2, 1, 64, 64), (3, 3, 128, 64), (4, 2, 64, 128), (5, 1, 128, 128), (6, 2, 128, 64)])
def test_ssm_packed(dtype, H, G, dk, dv):
    """Sequences of no token, one token and lengths around the chunks' ends."""
    _gpu()
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 200]
    cu = _cu(lens)
    v = _ssm_inputs(H * dk + dv, (int(cu[-1]),), len(lens), H, G, dk, dv, dtype)
    _check_ssm(v, cu, f"ssm {ids(dtype)} H{H} G{G} {dk}x{dv}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("T", [0, 1, 3, 100, 130])
def test_ssm_time_major(dtype, T):
    _gpu()
    v = _ssm_inputs(T, (T, 3), 3, 4, 2, 64, 64, dtype)
    _check_ssm(v, None, f"ssm time-major {ids(dtype)} T{T}")
    _check_ssm(v, None, f"ssm bare {ids(dtype)} T{T}", D=None, dt_bias=None, S0=None)


def test_ssm_rows_not_16_byte_aligned():
    _gpu()
    for dtype in TYPES:
        v = _ssm_inputs(3, (300,), 1, 2, 1, 128, 64, dtype, pad=1)
        assert v["x"].data_ptr() % 16 != 0
        _check_ssm(v, _cu([300]), f"ssm odd base {ids(dtype)}")


def test_ssm_without_softplus():
    """d_t used as given: zero steps leave the state, negative log decays as usual."""
    _gpu()
    for dtype in TYPES:
        v = _ssm_inputs(4, (140,), 2, 2, 1, 64, 128, dtype)
        v["dt"] = (v["dt"].abs() * 0.05).to(dtype)
        v["dt"][3:9] = 0
        v["dt_bias"] = None
        _check_ssm(v, _cu([100, 40]), f"ssm no softplus {ids(dtype)}", softplus=False)


def test_ssm_long_sequence():
    """One sequence of 3001 tokens beside short ones: split along the sequence."""
    _gpu()
    for dtype in TYPES:
        cu = _cu([5, 3001, 0, 40])
        v = _ssm_inputs(6, (int(cu[-1]),), 4, 2, 1, 64, 64, dtype)
        _check_ssm(v, cu, f"ssm long {ids(dtype)}")


def test_ssm_few_long_among_many_sequences():
    """Three of 70 sequences are split along their length, behind and between
    short and empty ones (heads enough that one pass looks over 32 or 64)."""
    _gpu()
    for dtype in (F32, BF16):
        lens = [7 * i % 23 for i in range(70)]
        lens[1], lens[66], lens[69] = 700, 1100, 300
        cu = _cu(lens)
        v = _ssm_inputs(8, (int(cu[-1]),), 70, 16, 1, 128, 128, dtype)
        _check_ssm(v, cu, f"ssm few long {ids(dtype)}")


def test_ssm_extreme_steps():
    """Steps of 0, of 1e-30 and so large that a token wipes the state: no
    inf - inf inside a chunk, and what follows depends on the wiping token on."""
    _gpu()
    for dtype in (F32, BF16):
        v = _ssm_inputs(7, (200,), 1, 2, 1, 128, 64, dtype)
        v["dt"] = (v["dt"].abs() * 0.02).to(dtype)
        v["dt"][10] = 0.0
        v["dt"][20] = 1e-30
        v["dt"][50] = 100.0
        v["dt"][127] = 100.0
        v["dt"][128] = 100.0
        v["dt_bias"] = None
        _check_ssm(v, _cu([200]), f"ssm extreme {ids(dtype)}", softplus=False)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_ssm_non_finite_inputs_reach_only_what_follows(dtype):
    """An inf or NaN in one token's x, B, C or step leaves every earlier output
    and the other sequences as they are, and shows in what it touches."""
    _gpu()
    for name in ("x", "Bm", "Cm", "dt"):
        for bad in (float("inf"), float("nan")):
            lens = [90, 150, 20]
            cu = _cu(lens)
            v = _ssm_inputs(8, (260,), 3, 2, 1, 64, 64, dtype)
            args = lambda u: (u["x"], u["dt"], u["A"], u["Bm"], u["Cm"])   # noqa: E731
            y0, S0 = lq.lq_ssm_prefill(*args(v), D=v["D"], dt_bias=v["dt_bias"], cu=cu)
            t = 90 + 70
            u = {k: (w.clone() if k == name else w) for k, w in v.items()}
            if name == "dt":
                u[name][t, 1] = bad
            else:
                u[name][t, 0, 5] = bad
            y1, S1 = lq.lq_ssm_prefill(*args(u), D=v["D"], dt_bias=v["dt_bias"], cu=cu)
            assert torch.equal(y1[:t], y0[:t]) and torch.equal(y1[240:], y0[240:]), (name, bad)
            assert torch.equal(S1[0], S0[0]) and torch.equal(S1[2], S0[2])
            h = 1 if name == "dt" else 0
            assert not torch.isfinite(y1[t, h]).all(), (name, bad)
            if name == "Cm":
                assert torch.equal(S1, S0) and torch.equal(y1[t + 1:], y0[t + 1:])
            else:
                assert not torch.isfinite(S1[1, h]).all()
            if name == "x":       # one value column of one head
                ok = [c for c in range(64) if c != 5]
                assert torch.equal(y1[:, 1], y0[:, 1]) and torch.equal(y1[:, 0, ok], y0[:, 0, ok])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("B,H,G,dk,dv", [(1, 16, 1, 128, 64), (2, 3, 3, 64, 64), (40, 8, 2, 128, 128), (300, 2, 1, 64, 128)])
def test_ssm_step(dtype, B, H, G, dk, dv):
    _gpu()
    v = _ssm_inputs(B + dk, (B,), B, H, G, dk, dv, dtype, pad=3)
    S = v["S0"].clone()
    y = lq.lq_ssm_step(S, v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], dt_bias=v["dt_bias"])
    one = lambda t: t[None]   # noqa: E731
    ry, rS, my, mS, n = R.ssm(one(v["x"]), one(v["dt"]), v["A"], one(v["Bm"]), one(v["Cm"]), v["D"], v["dt_bias"], True,
                              v["S0"], None)
    ty, tS = _ssm_tol(ry[0], rS, my[0], mS, 1, dtype, dk)
    _close(y, ry[0], ty, f"ssm step {ids(dtype)} y")
    _close(S, rS, tS, f"ssm step {ids(dtype)} S")


def test_ssm_prompt_in_parts_and_steps():
    """A prompt in two calls with the state in place, then single tokens."""
    _gpu()
    v = _ssm_inputs(9, (260, 2), 2, 4, 1, 128, 64, F32)
    S = v["S0"].clone()
    kw = {"D": v["D"], "dt_bias": v["dt_bias"]}
    ys = []
    for a, b in ((0, 150), (150, 250)):
        y, _ = lq.lq_ssm_prefill(*(v[k][a:b] if k != "A" else v[k] for k in ("x", "dt", "A", "Bm", "Cm")), S0=S, S_out=S, **kw)
        ys.append(y)
    for t in range(250, 260):
        ys.append(lq.lq_ssm_step(S, *(v[k][t] if k != "A" else v[k] for k in ("x", "dt", "A", "Bm", "Cm")), **kw)[None])
    ry, rS, my, mS, n = R.ssm(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["dt_bias"], True, v["S0"], None)
    ty, tS = _ssm_tol(ry, rS, my, mS, n, F32, 128)
    _close(torch.cat(ys), ry, ty, "ssm parts y")
    _close(S, rS, tS, "ssm parts S")


def test_ssm_rows_outside_the_sequences_stay():
    _gpu()
    for dtype in TYPES:
        v = _ssm_inputs(2, (300,), 2, 2, 1, 64, 64, dtype)
        cu = torch.tensor([7, 60, 280], dtype=torch.int32, device="cuda")
        y = torch.full((300, 2, 64), 7.0, dtype=dtype, device="cuda")
        lq.lq_ssm_prefill(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], y=y, cu=cu)
        assert (y[:7] == 7).all() and (y[280:] == 7).all() and not (y[7:280] == 7).all(-1).any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_ssm_many_short_sequences(dtype):
    """More sequences than a warp looks at in one step, of 0 to 40 tokens."""
    _gpu()
    lens = [(i * 37) % 41 if i % 5 else 0 for i in range(700)]
    cu = _cu(lens)
    v = _ssm_inputs(17, (int(cu[-1]),), len(lens), 2, 1, 64, 64, dtype)
    y, S = lq.lq_ssm_prefill(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], dt_bias=v["dt_bias"], S0=v["S0"], cu=cu)
    at = cu.tolist()
    for b in (0, 1, 31, 32, 255, 256, 257, 511, 512, 698, 699):
        one = slice(at[b], at[b + 1])
        part = {k: (w[one] if k in ("x", "dt", "Bm", "Cm") else w[b:b + 1] if k == "S0" else w) for k, w in v.items()}
        n = at[b + 1] - at[b]
        ry, rS, my, mS, _ = R.ssm(part["x"], part["dt"], v["A"], part["Bm"], part["Cm"], v["D"], v["dt_bias"], True,
                                  part["S0"], _cu([n]))
        ty, tS = _ssm_tol(ry, rS, my, mS, n, dtype, 64)
        if n:
            _close(y[one], ry, ty, f"sequence {b} y")
        _close(S[b:b + 1], rS, tS, f"sequence {b} S")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("lens", [[1] * 9, [2, 0, 1, 3], [16], [1, 0, 30, 0, 0, 0] * 3])
def test_ssm_token_by_token_prompts(dtype, lens):
    """Prompts short enough to run token by token, and just longer ones."""
    _gpu()
    cu = _cu(lens)
    v = _ssm_inputs(19, (int(cu[-1]),), len(lens), 3, 1, 128, 64, dtype)
    _check_ssm(v, cu, f"ssm short {ids(dtype)} {lens[:4]}")


def test_ssm_growing_states():
    """A rate above 0 makes the state grow: factors above 1 in every path."""
    _gpu()
    for dtype in (F32, BF16):
        v = _ssm_inputs(23, (150,), 1, 2, 1, 64, 64, dtype)
        v["A"] = torch.tensor([0.5, -2.0], device="cuda")
        _check_ssm(v, _cu([150]), f"ssm growing {ids(dtype)}")


def test_rows_beyond_32_bit_offsets():
    """Rows of a projection so wide that element offsets pass 2^31 (4.3 GB)."""
    _gpu()
    g = _gen(41)
    rows, ld = 70000, 32768
    wide = torch.zeros((rows, ld), dtype=BF16, device="cuda")
    at = rows - 200
    C = 2 * 64 + 2 * 64
    cols = _randn(g, (200, C + 2), BF16)
    wide[at:, :C + 2] = cols
    cu = torch.tensor([at, rows - 50, rows], dtype=torch.int32, device="cuda")
    w = _randn(g, (C, 4))
    y = lq.lq_conv_prefill(wide[:, :C], w, y=wide[:, 512:512 + C], cu=cu)[0]
    local = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    want = lq.lq_conv_prefill(cols[:, :C].contiguous(), w, cu=local)[0]
    assert torch.equal(y[at:], want) and (y[:at] == 0).all()
    heads = lambda t: (t[:, :128].unflatten(-1, (2, 64)), t[:, 128:192].unflatten(-1, (1, 64)),   # noqa: E731
                       t[:, 192:256].unflatten(-1, (1, 64)))
    A = torch.tensor([-1.0, -4.0], device="cuda")
    x, Bm, Cm = heads(y)
    out = wide[:, 1024:1152].unflatten(-1, (2, 64))
    _, S = lq.lq_ssm_prefill(x, wide[:, C:C + 2], A, Bm, Cm, y=out, cu=cu)
    x, Bm, Cm = heads(want)
    yl, Sl = lq.lq_ssm_prefill(x, cols[:, C:].contiguous(), A, Bm, Cm, cu=local)
    for got, ref in ((out[at:], yl), (S, Sl)):
        assert (got.double() - ref.double()).norm() <= 1e-2 * ref.double().norm()
    wn = torch.ones(128, device="cuda")
    n = lq.lq_norm_out(out.flatten(1)[:, None], wn, y=wide[:, 2048:2176].unflatten(-1, (1, 128)))
    assert torch.equal(n[at:], lq.lq_norm_out(out[at:].reshape(200, 1, 128), wn))


# -- norms --------------------------------------------------------------------------

def _norm_tol(y, terms, dtype, D, act):
    # statistic: D squares summed (probabilistic), its root halves the error
    k = (4 * math.sqrt(D) + 12) * R.U + _act_rel(dtype, act)
    return R.half_step(dtype) * (1 + 1e-3) * y.abs() + 2 * k * terms + R.tiny(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 7), (5, 64), (9, 129), (4, 512), (2, 1000), (3, 2048), (2, 4096), (2, 4097),
                                    (2, 8192), (1, 16384), (1, 16383)])
def test_norm_in(dtype, rows, D):
    _gpu()
    g = _gen(D)
    x, res = _randn(g, (rows, D), dtype), _randn(g, (rows, D), dtype, 3.0)
    w, vec = 1 + _randn(g, (D,), scale=0.2), torch.rand((D,), generator=g, device="cuda")
    for r, sc in ((res, vec), (res, 0.25), (None, 1.0)):
        y, h = lq.lq_norm_in(x, w, res=r, scale=sc, eps=1e-5)
        s64 = sc.double() if isinstance(sc, torch.Tensor) else sc
        ry, rh = R.norm_in(x, w, r, s64, 1e-5)
        terms = ((s64 * x.double()).abs() + (0 if r is None else r.double().abs()))
        inv = 1 / torch.sqrt((rh * rh).mean(-1, keepdim=True) + 1e-5)
        _close(h, rh, R.half_step(dtype) * (1 + 1e-3) * rh.abs() + 2 * R.U * terms + R.tiny(dtype), f"h {ids(dtype)} {D}")
        _close(y, ry, _norm_tol(ry, ry.abs() + terms * inv * w.double().abs(), dtype, D, None), f"norm_in {ids(dtype)} {D}")


@pytest.mark.parametrize("dtype,xt", [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)], ids=ids)
@pytest.mark.parametrize("rows,G,D", [(1, 1, 1), (5, 3, 47), (7, 16, 128), (3, 2, 64), (33, 1, 2048), (2, 2, 4104), (1, 1, 16384)])
def test_norm_out(dtype, xt, rows, G, D):
    _gpu()
    g = _gen(D + rows)
    x = _randn(g, (rows, G, D), xt, 0.5)
    z = _randn(g, (rows, G * D + 16), dtype, 2.0)[:, 16:].unflatten(-1, (G, D))    # columns of a projection
    res = _randn(g, (rows, G, D), dtype, 3.0)
    w1, w2 = 1 + _randn(g, (D,), scale=0.2), 1 + _randn(g, (G, D), scale=0.2)
    vec = torch.rand((G, D), generator=g, device="cuda")
    for w, zz, act, first, r, sc in ((w1, z, "silu", False, None, 1.0), (w2, z, "sigmoid", True, res, vec),
                                     (w2, z, "silu", True, res, 0.5), (w1, None, "silu", False, None, 2.0)):
        y = lq.lq_norm_out(x, w, z=zz, act=act, gate_first=first, res=r, scale=sc, eps=1e-6, y=torch.empty_like(res))
        s64 = sc.double() if isinstance(sc, torch.Tensor) else sc
        ry = R.norm_out(x, w, zz, act, first, r, s64, 1e-6)
        inner = R.norm_out(x, w, zz, act, first, None, s64, 1e-6).abs()
        _close(y, ry, _norm_tol(ry, inner + ry.abs(), dtype, D, act if zz is not None else None),
               f"norm_out {ids(dtype)} {G}x{D} {act} first={first}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_norms_of_every_size_class(dtype):
    """Groups on both sides of every bound at which the team or the elements per
    thread change, aligned ones and ones whose rows start anywhere."""
    _gpu()
    bounds = (4, 8, 16, 32, 48, 64, 96, 128, 192, 256, 384, 512, 1024, 1536, 2048, 4096)
    for D in sorted({d + k for d in bounds for k in (0, 1)}):
        for off in (0, 1):
            g = _gen(2 * D + off)
            x, res = (_randn(g, (7, D + off), dtype)[:, off:] for _ in range(2))
            w = 1 + _randn(g, (D,), scale=0.2)
            y, h = lq.lq_norm_in(x, w, res=res, scale=0.5, eps=1e-5)
            ry, rh = R.norm_in(x, w, res, 0.5, 1e-5)
            terms = 0.5 * x.double().abs() + res.double().abs()
            inv = 1 / torch.sqrt((rh * rh).mean(-1, keepdim=True) + 1e-5)
            _close(h, rh, R.half_step(dtype) * (1 + 1e-3) * rh.abs() + 2 * R.U * terms + R.tiny(dtype), f"h {D}")
            _close(y, ry, _norm_tol(ry, ry.abs() + terms * inv * w.double().abs(), dtype, D, None), f"in {D} {off}")
            a, b = x.unflatten(-1, (1, D)), res.unflatten(-1, (1, D))
            y = lq.lq_norm_out(a, w, z=b, eps=1e-6)
            ry = R.norm_out(a, w, b, "silu", False, None, 1.0, 1e-6)
            _close(y, ry, _norm_tol(ry, 2 * ry.abs(), dtype, D, "silu"), f"out {D} {off}")


def test_norms_in_place_and_zero_rows():
    _gpu()
    g = _gen(3)
    x, res, w = _randn(g, (6, 256), BF16), _randn(g, (6, 256), BF16), _randn(g, (256,))
    y0, h0 = lq.lq_norm_in(x, w, res=res, scale=0.5)
    a, b = x.clone(), res.clone()
    y1, h1 = lq.lq_norm_in(a, w, res=b, scale=0.5, y=a, h=b)
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and y1 is a and h1 is b
    x3, z3, r3 = (t.view(6, 2, 128) for t in (x, res, h0))
    want = lq.lq_norm_out(x3, w[:128], z=z3, res=r3)
    for alias in range(3):
        t = [v.clone() for v in (x3, z3, r3)]
        got = lq.lq_norm_out(t[0], w[:128], z=t[1], res=t[2], y=t[alias])
        assert torch.equal(got, want), alias
    assert (lq.lq_norm_in(torch.zeros_like(x), w)[0] == 0).all()
    assert lq.lq_norm_in(x[:0], w)[0].shape == (0, 256)
    # all-zero rows and a row with an infinity stay apart
    x[2] = 0
    x[3, 5] = float("inf")
    y, _ = lq.lq_norm_in(x, w)
    assert (y[2] == 0).all() and torch.isfinite(y[[0, 1, 2, 4, 5]]).all() and not torch.isfinite(y[3]).all()


# -- streams, graphs, chains ----------------------------------------------------------

def test_binding_refuses_what_it_cannot_pass_on():
    """Tensors of another type, shape, spacing or device, unknown names and sizes
    beyond 32 bits are refused before anything is allocated or launched."""
    _gpu()
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")   # noqa: E731
    x, w, h = z(6, 2, 64), z(64, 4, t=F32), z(6, 2, 2, 64)
    dt, A, S, B1 = z(6, 2, 2), z(2, t=F32), z(2, 2, 64, 64, t=F32), z(6, 2, 1, 64)
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    wrong_type = [
        lambda: lq.lq_conv_prefill(x.double(), w), lambda: lq.lq_conv_prefill(x, w.half()),
        lambda: lq.lq_conv_prefill(x, w.cpu()), lambda: lq.lq_conv_prefill(x, w, bias=3.0),
        lambda: lq.lq_conv_prefill(x[:, 0], w, cu=cu.long()), lambda: lq.lq_conv_prefill(x[:, 0], w, cu=[0, 6]),
        lambda: lq.lq_conv_step(z(2, 3, 64, t=F32), x[0], w), lambda: lq.lq_ssm_prefill(h, dt.float(), A, B1, B1),
        lambda: lq.lq_ssm_prefill(h, dt, A, B1, B1, S0=S.bfloat16()), lambda: lq.lq_ssm_step(S, h[0], dt[0], A, B1[0], 1),
        lambda: lq.lq_norm_in(x, w[:, 0].contiguous(), res=x.float()), lambda: lq.lq_norm_in(x, None),
        lambda: lq.lq_norm_in(x, w[:, 0].contiguous(), scale="1"), lambda: lq.lq_norm_out(x, w[:, 0].contiguous(), z=3),
        lambda: lq.lq_norm_out(x, w[:, 0].contiguous(), z=x.half(), res=x),
    ]
    wrong_value = [
        lambda: lq.lq_conv_prefill(x, w[:32]), lambda: lq.lq_conv_prefill(x, w, act="relu"),
        lambda: lq.lq_conv_prefill(x, w[0]), lambda: lq.lq_conv_prefill(x[:, 0], w), lambda: lq.lq_conv_prefill(x, w, cu=cu),
        lambda: lq.lq_conv_prefill(x[:, 0], w, cu=cu[:1]), lambda: lq.lq_conv_prefill(x, w[:, ::2]),
        lambda: lq.lq_conv_prefill(z(6, 2, 128)[..., ::2], w), lambda: lq.lq_conv_prefill(z(12, 4, 64)[::2, ::2][:, :2], w, y=x[:5]),
        lambda: lq.lq_conv_prefill(z(6, 3, 64)[:, :2], w), lambda: lq.lq_conv_step(z(2, 3, 32), x[0], w),
        lambda: lq.lq_ssm_prefill(h, dt[:5], A, B1, B1), lambda: lq.lq_ssm_prefill(h, dt, A, B1, B1[..., :32]),
        lambda: lq.lq_ssm_prefill(h, dt, A[:1], B1, B1), lambda: lq.lq_ssm_step(S[:1], h[0], dt[0], A, B1[0], B1[0]),
        lambda: lq.lq_ssm_step(S.transpose(2, 3), h[0], dt[0], A, B1[0], B1[0]),
        lambda: lq.lq_norm_in(x, w[:32, 0].contiguous()), lambda: lq.lq_norm_in(x, w[:, 0]),
        lambda: lq.lq_norm_out(x, w[:, 0].contiguous(), scale=w[:, 0].contiguous()),
        lambda: lq.lq_norm_out(x[0, 0], w[:, 0].contiguous()),
    ]
    for n, call in enumerate(wrong_type):
        with pytest.raises(TypeError):
            call()
            pytest.fail(f"type {n}")
    for n, call in enumerate(wrong_value):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"value {n}")
    with pytest.raises(lq.LqError) as e:
        lq.lq_ssm_prefill(z(6, 2, 2, 32), dt, A, B1, B1)
    assert e.value.code == lq.LQ_ERR_UNSUPPORTED
    with pytest.raises(lq.LqError) as e:
        lq.lq_conv_prefill(x, w, y=x)
    assert e.value.code == lq.LQ_ERR_INVALID_ARG


def test_side_stream_and_graph_replay():
    """Calls on a stream of the caller's, and captured and replayed, give the
    eager call's bits."""
    _gpu()
    v = _ssm_inputs(11, (600,), 3, 4, 1, 128, 64, BF16)
    cu = _cu([400, 1, 199])
    g = _gen(12)
    w, wn = _randn(g, (256, 4)), _randn(g, (64,))
    xc = v["x"].reshape(600, 256)

    def chain(stream=None):
        xs, _ = lq.lq_conv_prefill(xc, w, cu=cu, stream=stream)
        y, S = lq.lq_ssm_prefill(xs.view(600, 4, 64), v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"],
                                 dt_bias=v["dt_bias"], S0=v["S0"], cu=cu, stream=stream)
        return lq.lq_norm_out(y, wn, z=v["x"], res=y, scale=0.5, stream=stream), S
    want = chain()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = chain(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(2):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_cut_prompts_queued_one_after_the_other(dtype):
    """Prompts cut along their length, queued without a wait: one workspace for
    all, states in place from call to call, inputs overwritten behind each call;
    eager and from a graph replayed with other values and other lengths.  The
    same bits as with a wait after every call."""
    _gpu()
    v = _ssm_inputs(17, (1600,), 2, 4, 2, 64, 64, dtype)
    x = [v["x"] * f for f in (1.0, -0.5, 0.25)]
    offsets = [_cu([1300, 300]), _cu([20, 1580]), _cu([800, 800])]
    need = lq.lq_ssm_workspace_bytes(dtype, 2, 4, 2, 64, 64, 1600)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    xin, cu, S = torch.empty_like(x[0]), offsets[0].clone(), v["S0"].clone()
    y = [torch.empty_like(x[0]) for _ in range(3)]

    def calls(wait):
        for k in range(3):
            xin.copy_(x[k])
            cu.copy_(offsets[k])
            lq.lq_ssm_prefill(xin, v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], dt_bias=v["dt_bias"], S0=S, S_out=S,
                              y=y[k], cu=cu, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        xin.fill_(float("nan"))
        ws.fill_(255)

    calls(True)
    want = [t.clone() for t in (*y, S)]
    for run in range(3):
        S.copy_(v["S0"])
        if run < 2:
            calls(False)
        else:
            S0 = S.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                calls(False)
            for _ in range(2):
                S.copy_(S0)
                for t in y:
                    t.fill_(float("nan"))
                graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, (*y, S))), run


def test_two_streams_at_once():
    """Cut prompts, convolutions, norms and steps queued on two streams at a time,
    each call with its own workspace: the bits of one after the other."""
    _gpu()
    for dtype in (BF16, F32):
        sets = []
        for seed in (31, 32):
            v = _ssm_inputs(seed, (900,), 2, 4, 2, 128, 64, dtype)
            g = _gen(seed)
            sets.append((v, _randn(g, (256, 4)), _randn(g, (64,)), _cu([640, 260])))

        def chain(v, w, wn, cu, stream):
            xs, win = lq.lq_conv_prefill(v["x"].reshape(900, 256), w, cu=cu, stream=stream)
            y, S = lq.lq_ssm_prefill(xs.view(900, 4, 64), v["dt"], v["A"], v["Bm"], v["Cm"], S0=v["S0"], cu=cu, stream=stream)
            z = lq.lq_norm_out(y, wn, z=v["x"], stream=stream)
            s = lq.lq_ssm_step(S, z[:2], v["dt"][:2], v["A"], v["Bm"][:2], v["Cm"][:2], stream=stream)
            return y, S, z, s, win
        want = [chain(*a, torch.cuda.current_stream()) for a in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in sets]
        for _ in range(5):
            got = [chain(*a, s) for a, s in zip(sets, streams)]
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for u, o in zip(want, got) for p, q in zip(u, o))


def test_same_inputs_same_bits():
    _gpu()
    for dtype in TYPES:
        v = _ssm_inputs(13, (1500,), 2, 4, 2, 64, 64, dtype)
        cu = _cu([1300, 200])
        a = [lq.lq_ssm_prefill(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], S0=v["S0"], cu=cu) for _ in range(3)]
        assert all(torch.equal(a[0][i], b[i]) for b in a[1:] for i in range(2))


def _scan_layer_ref(sl, w, x, res, lens):
    """The layer of ScanRunner in 64 bits over packed sequences."""
    f = {k: v.double() for k, v in w.items()}
    u, h = R.norm_in(x, f["w_norm"], res, sl.scale, sl.eps)
    p = u @ f["w_in"]
    cu = _cu(lens)
    n, gk = sl.inner, sl.G * sl.dk
    xbc, win, _ = R.conv(p[:, n:n + sl.conv], f["w_conv"], f["b_conv"], "silu", None, cu)
    y, S, _, _, _ = R.ssm(xbc[:, :n].unflatten(-1, (sl.H, sl.dv)), p[:, n + sl.conv:], f["A"],
                          xbc[:, n:n + gk].unflatten(-1, (sl.G, sl.dk)), xbc[:, n + gk:].unflatten(-1, (sl.G, sl.dk)),
                          f["D"], f["dt_bias"], True, None, cu)
    y = R.norm_out(y, f["w_gate"], p[:, :n].unflatten(-1, (sl.H, sl.dv)), "silu", False, None, 1.0, sl.eps)
    return y.flatten(-2) @ f["w_out"], h, win, S


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_scan_layer_prompts_then_tokens(dtype):
    """ScanRunner: ragged prompts, then single tokens, eager and from a captured
    graph, against the whole sequences in 64 bits.  Every stage rounds its
    output once and the stages after it carry that on: 12 half steps of the type
    relative to the largest value of each output (two projections, two norms,
    convolution, scan, gate; sums of random-sign errors), plus 1e-5."""
    _gpu()
    sl = configs.TINY_SCAN
    lens, more = [70, 1, 133], 4
    g = _gen(21)
    x = _randn(g, (sum(lens) + 3 * more, sl.d), dtype)
    res = _randn(g, x.shape, dtype)
    # rows of each sequence: its prompt, then its single tokens
    prompt, steps, at = [], [[] for _ in range(more)], 0
    for n in lens:
        prompt += range(at, at + n)
        for i in range(more):
            steps[i].append(at + n + i)
        at += n + more
    run = runner.ScanRunner(sl, 3, dtype)
    out, h = torch.empty_like(x), torch.empty_like(x)
    out[prompt], h[prompt] = run.prompt(x[prompt], res[prompt], cu=_cu(lens))
    for i in range(more):
        if i == 2:
            run.capture()
        if i < 2:
            out[steps[i]], h[steps[i]] = run.step(x[steps[i]], res[steps[i]])
        else:
            run.x_in.copy_(x[steps[i]])
            run.res_in.copy_(res[steps[i]])
            out[steps[i]], h[steps[i]] = run.replay()
    ro, rh, rw, rS = _scan_layer_ref(sl, run.w, x, res, [n + more for n in lens])
    for name, got, want in (("out", out, ro), ("residual", h, rh), ("window", run.window, rw), ("state", run.state, rS)):
        off = (got.double() - want).abs().max().item() / want.abs().max().item()
        print(f"scan layer {ids(dtype)} {name}: {off:.2e}")
        assert off <= 12 * R.half_step(dtype) + 1e-5, (name, off)


def test_delta_rule_layer_around_the_windowed_state():
    """The operators around the library's own recurrence, as a delta-rule layer
    uses them: convolution, L2 norm of q and k, prefill, the quantized windowed
    state, decode steps, gated norm of their float32 outputs -- the convolution
    and norms against 64 bits at every token, and the decode against the FP32
    state's decode on the same inputs (the quantized state's own error is the
    windowed decode's subject)."""
    _gpu()
    wl = configs.TINY_GDN.with_(B=2, W=4, T=8)
    B, H, d, T = wl.B, wl.H, wl.dk, 20
    g = _gen(31)
    C = 3 * H * d
    raw = _randn(g, (T + 8, B, C + H * d), F32)           # q | k | v and the gate's columns
    w, bias = _randn(g, (C, 4), scale=0.5), _randn(g, (C,), scale=0.1)
    wn, wl2 = 1 + _randn(g, (d,), scale=0.1), torch.full((d,), d ** -0.5, device="cuda")
    tok = gen.token_inputs(wl, T + 8, device="cuda")
    xs, window = lq.lq_conv_prefill(raw[:T, :, :C], w, bias)
    tail = torch.stack([lq.lq_conv_step(window, raw[t, :, :C], w, bias) for t in range(T, T + 8)])
    xs = torch.cat([xs, tail])
    ry, _, mag = R.conv(raw[..., :C], w, bias, "silu", None, None)
    _close(xs, ry, _conv_tol(ry, mag, F32, 4, "silu"), "delta layer convolution")
    q, k, v = (t.unflatten(-1, (H, d)) for t in xs.split(H * d, -1))
    unit = [lq.lq_norm_out(t.contiguous(), wl2, eps=1e-12) for t in (q, k)]
    for t, n in zip((q, k), unit):
        want = t.double() / torch.linalg.vector_norm(t.double(), dim=-1, keepdim=True)
        _close(n, want, 1e-6 * want.abs() + 1e-9, "L2 norm")
    q, k, v = unit[0], unit[1], v.contiguous()
    outs = {}
    for mode in ("fp32", "window"):
        cfg = lq.Config.from_workload(wl, mode=mode)
        S = lq.lq_prefill(cfg, q[:T], k[:T], v[:T], tok["beta"][:T], tok["alpha"][:T])
        st = lq.lq_state_init(cfg, S)
        o = torch.empty((8, B, H, d), device="cuda")
        for i in range(8):
            t = T + i
            lq.lq_decode_step(st, q[t], k[t], v[t], tok["beta"][t].contiguous(), tok["alpha"][t].contiguous(), o[i])
        assert lq.lq_get_status(st) == lq.LQ_OK
        z = raw[T:, :, C:].unflatten(-1, (H, d)).to(BF16)
        y = lq.lq_norm_out(o, wn, z=z, eps=1e-6)
        assert y.dtype == BF16
        ref = R.norm_out(o, wn, z, "silu", False, None, 1.0, 1e-6)
        _close(y, ref, _norm_tol(ref, ref.abs(), BF16, d, "silu"), f"delta layer gate {mode}")
        outs[mode] = y.double()
    # an 8-bit state: a step of the codes is amax / 127 of a column
    off = (outs["window"] - outs["fp32"]).norm() / outs["fp32"].norm()
    print(f"delta layer, windowed against FP32 state: {off:.2e}")
    assert off < 0.05
