"""The residual norms at the largest number of rows, 2^31 - 1 (of one column): the number of blocks is
formed from T and the rows a block takes at once, beyond 32 bits."""
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"
B = torch.bfloat16
T, STEP = (1 << 31) - 1, 1 << 27


def values(n, period):
    """bf16 values that repeat with a period that divides no power of two."""
    v = (torch.arange(period, device=DEV) % 251 - 125).to(B) / 8
    return v.repeat(n // period + 1)[:n].view(n, 1)


def test_most_rows(bl):
    x, y = values(T, 999_983), values(T, 1_000_003)
    new = bl.bitlinear_residual_norm(x, y, post_norm=False, mode="none")["x"]
    assert bl.check_device_status() == 0
    for i in range(0, T, STEP):
        # both values are multiples of 1/8 below 16: the fp32 sum is exact, and rounded once
        assert torch.equal(new[i:i + STEP], (x[i:i + STEP].float() + y[i:i + STEP].float()).to(B)), i
    del new
    dx = torch.ones(T, 1, device=DEV)
    dx[-1], dx[0] = 3.0, 5.0
    got = bl.bitlinear_residual_norm_backward(dx, None, x, y, gate=torch.full((1,), 0.5, device=DEV), alpha=2.0,
                                              want_dgate=False)
    assert bl.check_device_status() == 0
    for i in range(0, T, STEP):
        assert torch.equal(got["dx"][i:i + STEP], 2.0 * dx[i:i + STEP]), i
        assert torch.equal(got["dy"][i:i + STEP], (0.5 * dx[i:i + STEP]).to(B)), i
