"""Launches of the gradient norm and the clip: one table of up to 960 non-empty gradients each."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("full,empty", [(0, 3), (1, 0), (64, 0), (64, 5), (65, 0), (960, 0), (960, 7), (961, 0), (961, 2),
                                        (1920, 1), (1921, 1)])
def test_launches(bl, full, empty):
    flat = torch.ones(max(full, 1) * 3, device=DEV)
    g = [flat[3 * i:3 * i + 3] for i in range(full)] + [flat[:0]] * empty
    if empty > 1:
        g.insert(full // 2, flat[:0])
    tables = max(1, -(-full // 960))
    n0 = bl.launch_count()
    o = bl.bitlinear_grad_norm(g, 1.0)
    n1 = bl.launch_count()
    c = bl.bitlinear_clip_grads(g, 1.0)
    n2 = bl.launch_count()
    assert (n1 - n0, n2 - n1) == (tables + 1, 2 * tables)
    assert torch.equal(o["norm"], c["norm"]) and abs(float(o["norm"]) ** 2 - 3 * full) <= 1e-6 * 3 * full
    assert full == 0 or torch.equal(flat, c["coef"].expand_as(flat))
