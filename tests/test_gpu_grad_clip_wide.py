"""Clipping of lists long enough for chunks of 32768 and 65536 elements: every element of a tensor's
last, partial chunk is scaled exactly once, however the 32-byte loop, the 16-byte loop and the single
elements share it.

The scaled gradients are one fp32 product with the coefficient, rounded once: compared exactly, in
place and into outputs that hold NaN beforehand.  Norm and coefficient as in test_gpu_grad_clip.py:
within two half steps of the fp64 sum's.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16
ROUND = 2048          # pairs of 16-byte vectors that a block takes in one round of the 32-byte loop


def tails(per, chunk):
    """Lengths (elements, `per` in a 16-byte vector) whose last chunk holds so many pairs of vectors
    and so many vectors and elements besides."""
    most = chunk // per // 2
    pairs = [p for r in range(0, most, ROUND) for p in (r, r + 1, r + 1536, r + 1537, r + 1792, r + 2047) if p < most]
    return [chunk * (i % 2) + (2 * p + i % 2) * per + (i * 5) % per for i, p in enumerate(pairs) if p + i % 2]


@pytest.mark.parametrize("offset", [0, 1, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("chunk,filler", [(32768, 39_000_000), (65536, 78_000_000)])
def test_last_chunks(bl, chunk, filler, offset):
    gen = torch.Generator(device=DEV).manual_seed(chunk + offset)
    small = [(n, t) for t in (F, B) for n in tails(4 if t is F else 8, chunk)]
    total = filler + sum(n for n, _ in small)
    # the rule that chooses the chunk: the smallest of 4096 x 2^k that leaves at most 4 chunks a block
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    assert total // (chunk // 2) > 4 * blocks and (chunk == 65536 or total // chunk <= 4 * blocks)
    g = [torch.randn(n + offset, generator=gen, device=DEV).to(t)[offset:] for n, t in small]
    g.insert(len(g) // 2, torch.randn(filler, generator=gen, device=DEV))
    norm = float(torch.stack([(t.double() ** 2).sum() for t in g]).sum().sqrt())
    src = [t.clone() for t in g]
    out = [torch.full((t.numel() + offset,), float("nan"), dtype=t.dtype, device=DEV)[offset:] for t in g]
    o = bl.bitlinear_clip_grads(g, 1.0, out=out)
    assert abs(float(o["norm"]) - norm) <= 2 * 2.0 ** -24 * norm
    assert abs(float(o["coef"]) * norm - 1) <= 1e-6
    for t, s, r in zip(g, src, out):
        assert torch.equal(t, s)
        assert torch.equal(r, (s.float() * o["coef"]).to(s.dtype)), (t.numel(), t.dtype)
    p = bl.bitlinear_clip_grads(g, 1.0)
    assert torch.equal(p["coef"], o["coef"])
    for t, r in zip(g, out):
        assert torch.equal(t, r), (t.numel(), t.dtype)
