"""GPU parity of the selective scan on the paths and values where it can go
wrong, against its definition in 64 bits; tolerances as in test_gpu_layer."""
import pytest
import torch

from tests.test_gpu_layer import TYPES, _check_ssm, _cu, _gpu, ids

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
