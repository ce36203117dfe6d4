"""Offsets beyond 2^31 elements and bytes: the last rows of large operands against the same rows alone."""
import pytest
import torch

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("K", [2048, 2047])
def test_residual_norm(bl, K):
    T, n = (1 << 31) // K + 300, 3
    x, y = torch.zeros(T, K, dtype=B, device=DEV), torch.zeros(T, K, dtype=B, device=DEV)
    for t in (x, y):
        t[-n:] = torch.randn(n, K, device=DEV).to(B)
    g = 1 + 0.1 * torch.randn(K, device=DEV)
    mode = "quant" if K % 32 == 0 else "norm"
    o = bl.bitlinear_residual_norm(x, y, g_post=g, g_pre=g, mode=mode)
    s = bl.bitlinear_residual_norm(x[-n:].clone(), y[-n:].clone(), g_post=g, g_pre=g, mode=mode)
    for k in o:
        assert torch.equal(o[k][-n:], s[k]), k
    for k in {"x", "h", "xdq"} & set(o):
        assert float(o[k][1 << 20].float().abs().max()) == 0.0, k
    dx = torch.zeros(T, K, device=DEV)
    dx[-n:] = torch.randn(n, K, device=DEV)
    b = bl.bitlinear_residual_norm_backward(dx, None, o["x"], y, r_post=o["r_post"], g_post=g)
    bs = bl.bitlinear_residual_norm_backward(dx[-n:].clone(), None, s["x"], y[-n:].clone(), r_post=s["r_post"],
                                             g_post=g)
    assert torch.equal(b["dx"][-n:], bs["dx"]) and torch.equal(b["dy"][-n:], bs["dy"])
    # the column sums add the same three rows, in another order: three roundings
    assert float((b["dpost_gain"] - bs["dpost_gain"]).abs().max()) <= 2.0 ** -22 * float(bs["dpost_gain"].abs().max()) * 3


def test_clip(bl):
    g = torch.zeros((1 << 31) + 4097, dtype=B, device=DEV)
    g[-5:] = 2.0
    g[0] = 4.0
    o = bl.bitlinear_clip_grads([g], 1.0)
    assert float(o["norm"]) == 6.0
    assert torch.equal(g[-5:], (2.0 * o["coef"]).to(B).expand(5)) and torch.equal(g[:1], (4.0 * o["coef"]).to(B))


@pytest.mark.parametrize("T", [1, 40])
def test_linear_int8_weight(bl, T):
    N, K = (1 << 31) // 2048 + 1024, 2048
    wq = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    tail = torch.randint(-127, 128, (40, K), dtype=torch.int8, device=DEV)
    wq[-40:] = tail
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device=DEV)
    y, acc = bl.bitlinear_linear_int8(xq, torch.ones(T, device=DEV), wq, torch.ones(N, device=DEV), want_acc=True)
    assert torch.equal(acc[:, -40:].double(), xq.double() @ tail.double().t())
    assert int(acc[:, :-40].abs().max()) == 0 and bl.check_device_status() == 0


def test_linear_int8_output(bl):
    """More than 2^31 outputs, through the large tiles."""
    T, N, K = 70000, 32768, 32
    xq = torch.randint(-127, 128, (T, K), dtype=torch.int8, device=DEV)
    wq = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV)
    y, _ = bl.bitlinear_linear_int8(xq, torch.ones(T, device=DEV), wq, torch.ones(N, device=DEV), out_dtype=F)
    for rows in (slice(0, 3), slice(T - 3, T)):
        assert torch.equal(y[rows].double(), xq[rows].double() @ wq.double().t())
    assert bl.check_device_status() == 0
