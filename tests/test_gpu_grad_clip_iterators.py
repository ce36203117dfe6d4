"""Gradients and outputs given as iterators, as `(p.grad for p in parameters)` is."""
import pytest
import torch

DEV = "cuda:0"


def test_iterator_reaches_the_checks():
    """On the CPU: what is refused is the tensors' device, not a second, used-up list."""
    import bit_ternary_qat_b200 as pkg
    from bit_ternary_qat_b200 import build
    build.build()
    for call in (pkg.bitlinear_grad_norm, pkg.bitlinear_clip_grads):
        with pytest.raises(ValueError, match="CUDA"):
            call(torch.ones(3) for _ in range(2))


@pytest.mark.gpu
def test_iterators(bl):
    src = [torch.randn(100 + i, device=DEV) for i in range(5)]
    want = bl.bitlinear_clip_grads(src, 0.5, out=[torch.zeros_like(t) for t in src])
    n = bl.bitlinear_grad_norm((t for t in src), 0.5)
    assert torch.equal(n["norm"], want["norm"]) and torch.equal(n["coef"], want["coef"])
    out = [torch.zeros_like(t) for t in src]
    got = bl.bitlinear_clip_grads((t for t in src), 0.5, out=(t for t in out))
    place = [t.clone() for t in src]
    same = bl.bitlinear_clip_grads((t for t in place), 0.5)
    for a, b, c, d, e, w in zip(got["grads"], out, same["grads"], place, src, want["grads"], strict=True):
        assert a is b and c is d and torch.equal(a, w) and torch.equal(c, w) and not torch.equal(e, w)
    listed = bl.bitlinear_clip_grads(place, 0.5)
    assert listed["grads"] is place
