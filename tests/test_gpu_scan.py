"""GPU parity of the selective scan on the paths and values where it can go
wrong, against its definition in 64 bits; tolerances as in test_gpu_layer."""
import pytest
import torch

from quantized_recurrent_state_lq_b200 import lq
from tests import layer_ref as R
from tests.test_gpu_layer import BF16, F16, F32, TYPES, _check_ssm, _close, _cu, _gpu, _ssm_inputs, _ssm_tol, ids

pytestmark = pytest.mark.gpu


def slow_tokens_after_wiping_ones(dtype, device):
    """Sequences of 32 tokens, 28 of which wipe the state (steps of 16 at rate
    -16: log2 decays of -150 each, as far as FP32 goes); the last four have
    steps of 1e-4 to 4e-4 and terms +1, -1, +1, -1 that cancel to about 1%."""
    B, H, dk, dv, T = 8, 8, 64, 64, 32
    g = torch.Generator().manual_seed(43)
    rand = lambda *s: torch.rand(s, generator=g)   # noqa: E731
    dt = torch.full((B, T, H), 16.0)
    dt[:, 28:] = 1e-4 * 4 ** rand(B, 4, H)
    dt = dt.to(dtype)
    sign = torch.tensor([1.0, -1.0, 1.0, -1.0])[None, :, None, None]
    x = torch.zeros(B, T, H, dv)
    x[:, 28:] = sign * (0.5 + rand(B, 1, H, dv)) / dt[:, 28:, :, None].float()
    b = torch.full((B * T, 1, dk), 0.125, dtype=dtype)
    return {"x": x.to(dtype).reshape(B * T, H, dv).to(device), "dt": dt.reshape(B * T, H).to(device),
            "A": torch.full((H,), -16.0, device=device), "Bm": b.to(device), "Cm": b.to(device), "D": None,
            "dt_bias": None, "S0": None}, [T] * B


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_slow_tokens_after_wiping_ones(dtype):
    """Running sums of log decays of 4200 whose differences are 0.002 to 0.01."""
    _gpu()
    v, lens = slow_tokens_after_wiping_ones(dtype, "cuda")
    _check_ssm(v, _cu(lens), f"ssm slow after wiping {ids(dtype)}", softplus=False)


def _is_cut(v, B, rows):
    H, dv = v["x"].shape[-2:]
    G, dk = v["Bm"].shape[-2:]
    return lq.lq_ssm_workspace_bytes(v["x"].dtype, B, H, G, dk, dv, rows) > 0


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("H,G,dk,dv", [(3, 1, 64, 64), (6, 2, 128, 64), (2, 1, 64, 128), (3, 3, 128, 128)])
@pytest.mark.parametrize("pad", [8, 1], ids=["aligned", "odd_base"])
def test_one_packed_prompt_cut(dtype, H, G, dk, dv, pad):
    """One prompt of 1500 tokens, cut along its length; odd_base: rows that no
    tensor copy takes.  Odd numbers of 64-column heads a group among them."""
    _gpu()
    v = _ssm_inputs(50 + H + pad, (1500,), 1, H, G, dk, dv, dtype, pad=pad)
    assert (v["x"].data_ptr() % 16 == 0) == (pad == 8)
    assert _is_cut(v, 1, 1500)
    _check_ssm(v, _cu([1500]), f"ssm cut {ids(dtype)} H{H} G{G} {dk}x{dv} pad {pad}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("H,G,dk,dv,pad", [(3, 1, 64, 64, 8), (2, 2, 128, 64, 8), (2, 1, 128, 128, 8), (1, 1, 64, 128, 1)])
def test_time_major_prompts_cut(dtype, H, G, dk, dv, pad):
    """Two sequences of 1100 tokens, row t * 2 + b, cut along their length."""
    _gpu()
    v = _ssm_inputs(60 + H + dv, (1100, 2), 2, H, G, dk, dv, dtype, pad=pad)
    assert _is_cut(v, 2, 2200)
    _check_ssm(v, None, f"ssm time-major cut {ids(dtype)} H{H} G{G} {dk}x{dv} pad {pad}")


@pytest.mark.parametrize("dtype", [BF16, F16], ids=ids)
@pytest.mark.parametrize("H,G,dk,dv,pad", [(8, 2, 64, 64, 8), (5, 1, 128, 128, 8), (9, 3, 64, 64, 1)])
def test_time_major_more_items_than_ctas(dtype, H, G, dk, dv, pad):
    """40 sequences of 200 tokens, uncut: each CTA walks its share of them."""
    _gpu()
    v = _ssm_inputs(70 + H, (200, 40), 40, H, G, dk, dv, dtype, pad=pad)
    _check_ssm(v, None, f"ssm time-major walk {ids(dtype)} H{H} G{G} {dk}x{dv} pad {pad}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_packed_prompts_cut_in_some_sequences_at_odd_bases(dtype):
    """Sequences of 1300, 0, 37 and 700 tokens behind rows that belong to none,
    no row on a 16-byte boundary, an odd number of 64-column heads."""
    _gpu()
    v = _ssm_inputs(81, (2050,), 4, 3, 1, 128, 64, dtype, pad=3)
    cu = torch.tensor([9, 1309, 1309, 1346, 2046], dtype=torch.int32, device="cuda")
    assert _is_cut(v, 4, 2050)
    inner = {k: (w[9:2046] if k in ("x", "dt", "Bm", "Cm") else w) for k, w in v.items()}
    y = torch.full((2050, 3, 64), 7.0, dtype=dtype, device="cuda")
    got, S = lq.lq_ssm_prefill(v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], D=v["D"], dt_bias=v["dt_bias"], S0=v["S0"],
                               cu=cu, y=y)
    want, rS, my, mS, n = R.ssm(inner["x"], v["dt"][9:2046], v["A"], inner["Bm"], inner["Cm"], v["D"], v["dt_bias"], True,
                                v["S0"], cu - 9)
    ty, tS = _ssm_tol(want, rS, my, mS, n, dtype, 128)
    assert (got[:9] == 7).all() and (got[2046:] == 7).all()
    _close(got[9:2046], want, ty, f"ssm cut at odd bases {ids(dtype)} y")
    _close(S, rS, tS, f"ssm cut at odd bases {ids(dtype)} S")


@pytest.mark.parametrize("H,G,dk,dv,lens,B,row,nan", [
    # 12 pieces of 128 tokens; the fourth one's start: also its own state, so all behind it
    (3, 1, 64, 64, [1500], 1, 384, [(384, 1500)]),
    (3, 1, 64, 64, [1500], 1, 511, [(384, 512)]),          # its end: the scan of that piece alone
    (2, 1, 128, 128, [1500], 1, 1499, [(1408, 1500)]),     # the last piece's end: the state too
    (2, 1, 128, 128, None, 2, 257, [(128, 1100)]),         # time-major, cut: token 128 of sequence 1
    # walked: and what the same CTAs take afterwards
    (9, 1, 128, 128, [200, 140, 0, 131] * 9, 36, 200, None),
    (9, 1, 128, 128, [200, 140, 0, 131] * 9, 36, 339, None),
    (9, 1, 128, 128, [200, 140, 0, 131] * 9, 36, 9 * 471 - 1, None),
    (8, 2, 64, 64, [300, 7] * 30, 60, 614, None),
], ids=["piece_start", "piece_end", "last_end", "time_major_cut", "start", "end", "very_last", "cut_and_walked"])
def test_a_wait_that_runs_out_leaves_nan(H, G, dk, dv, lens, B, row, nan):
    """A wait counted as run out (lq_selftest_ssm_wait; every real wait ends):
    the outputs and states behind it are NaN, every other value is that of the
    ordinary call, and nothing keeps what its memory held before."""
    _gpu()
    lead = (1100, B) if lens is None else (sum(lens),)
    cu = None if lens is None else _cu(lens)
    v = {k: t.contiguous() for k, t in _ssm_inputs(90 + H, lead, B, H, G, dk, dv, BF16).items()}
    args = [v[k] for k in ("x", "dt", "A", "Bm", "Cm")]
    want, wS = lq.lq_ssm_prefill(*args, S0=v["S0"], cu=cu)
    n_ws = lq.lq_ssm_workspace_bytes(BF16, B, H, G, dk, dv, want[..., 0, 0].numel())
    ws = torch.full((n_ws,), 1, dtype=torch.uint8, device="cuda") if n_ws else None
    y, S = torch.full_like(want, 7.0), torch.full_like(wS, 7.0)
    lq.lq_selftest_ssm_wait(row, *args, v["S0"], S, y, cu=cu, workspace=ws)
    for got, ref in ((y, want), (S, wS)):
        off = torch.isnan(got)
        assert (off | (got == ref)).all()
        # whole heads of a row, whole states
        assert torch.equal(off.any(-1), off.all(-1))
    assert torch.equal(torch.isnan(S).flatten(2).any(-1), torch.isnan(S).flatten(2).all(-1))
    b = row % B if lens is None else int((cu > row).nonzero()[0]) - 1
    mine = y[:, b] if lens is None else y[int(cu[b]):int(cu[b + 1])]
    bad = torch.isnan(mine).all(-1).all(-1)
    if nan is None:
        at = row if lens is None else row - int(cu[b])
        assert bad[at:].all() and torch.isnan(S[b]).all()
    else:
        assert [(int(i.min()), int(i.max()) + 1) for i in [bad.nonzero()]] == nan and bad.sum() == nan[0][1] - nan[0][0]
        assert torch.isnan(S[b]).all() if nan[0][1] == mine.shape[0] else not torch.isnan(S).any()
        assert torch.isnan(y).sum() == bad.sum() * H * dv
    # an ordinary call afterwards is as before
    again, aS = lq.lq_ssm_prefill(*args, S0=v["S0"], cu=cu)
    assert torch.equal(again, want) and torch.equal(aS, wS)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
def test_states_at_the_end_of_the_fp32_range(dtype):
    """States within 2^-13 of the FP32 maximum that C reads at 2^-70: every
    output is far inside the range, though rounding the state itself to fewer
    bits would pass the end of it."""
    _gpu()
    v = _ssm_inputs(97, (70,), 1, 4, 1, 64, 64, dtype)
    big = torch.finfo(F32).max * (1 - 2.0 ** -14)
    v["S0"] = torch.where(v["S0"] < 0, -big, big)
    v["Cm"] = (v["Cm"].float() * 2.0 ** -70).to(dtype)
    v["A"] = torch.tensor([-2.0 ** -20, -0.01, -1.0, -16.0], device="cuda")
    v["dt"] = (v["dt"].abs() * 0.01).to(dtype)
    v["D"] = v["dt_bias"] = None
    _check_ssm(v, _cu([70]), f"ssm end of the range {ids(dtype)}", softplus=False)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
def test_values_at_the_end_of_the_fp32_range(dtype):
    """x at the type's largest values beside steps of 1 (bf16: 1.003, within the
    FP32 range but past the end of bf16's) and B and C at 2^-40."""
    _gpu()
    v = _ssm_inputs(98, (70,), 1, 2, 1, 64, 64, dtype)
    big = torch.finfo(dtype).max if dtype == BF16 else torch.finfo(F32).max * (1 - 2.0 ** -14)
    v["x"] = torch.where(v["x"] < 0, -big, big).to(dtype)
    v["Bm"], v["Cm"] = ((v[k].float() * 2.0 ** -40).to(dtype) for k in ("Bm", "Cm"))
    v["dt"] = torch.full_like(v["dt"], 1.0)
    v["dt_bias"] = torch.full((2,), 0.003 if dtype == BF16 else 0.0, device="cuda")
    v["A"] = torch.tensor([-1e-6, -0.5], device="cuda")
    v["D"] = torch.tensor([0.5, 2.0 ** -30], device="cuda")
    v["S0"] = None
    _check_ssm(v, _cu([70]), f"ssm values at the end of the range {ids(dtype)}", softplus=False)
