"""The global gradient norm, clipping to it, and the optimizer step with its coefficient.

The norm's squares and sums are fp64, so norm and coefficient may differ from a long fp64 sum by
the final fp32 rounding alone (one half step, and a second where fp64's own error tips a tie);
the scaled gradients are one fp32 product with the coefficient, rounded once: compared exactly.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_ternary_qat_b200 import _lib, synth
from parity_util import np_
from test_gpu_optimizer import HP, HP_LOUD, _bounds, _state

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def tensors(sizes, types, seed=0, std=1e-2, offset=0):
    """Gradients as views `offset` elements into their own buffers."""
    gen = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(n + offset, generator=gen)).to(types[i % len(types)]).to(DEV)[offset:]
            for i, n in enumerate(sizes)]


def want_norm(grads):
    return float(np.sqrt(np.sum([float((g.cpu().double() ** 2).sum()) for g in grads])))


def check(bl, grads, max_norm):
    norm = want_norm(grads)
    o = bl.bitlinear_grad_norm(grads, max_norm)
    out = [torch.full_like(g, 3.0) for g in grads]
    c = bl.bitlinear_clip_grads(grads, max_norm, out=out)
    before = [g.clone() for g in grads]
    torch.cuda.synchronize()
    assert torch.equal(o["norm"], c["norm"]) and torch.equal(o["coef"], c["coef"])
    assert abs(float(o["norm"]) - norm) <= 2 * 2.0 ** -24 * norm
    coef = min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
    assert abs(float(o["coef"]) - coef) <= 2 * 2.0 ** -24 * coef
    for g, b, r in zip(grads, before, c["grads"]):
        assert torch.equal(g, b)
        assert torch.equal(r, (g.float() * c["coef"]).to(g.dtype))
    place = [g.clone() for g in grads]
    bl.bitlinear_clip_grads(place, max_norm)
    for p, r in zip(place, c["grads"]):
        assert torch.equal(p, r)
    return o


@pytest.mark.parametrize("sizes", [[1], [3, 1, 2], [4096], [4097, 5, 0, 8191], [0, 0], [100003, 7, 65536, 1 << 20],
                                   [1 + 37 * i for i in range(64)], [1 + 11 * i for i in range(65)],
                                   [5] * 3000])
@pytest.mark.parametrize("types", [[F], [B], [F, B]])
def test_norm_and_clip(bl, sizes, types):
    check(bl, tensors(sizes, types, seed=len(sizes)), 0.01)


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
def test_unaligned_views(bl, offset):
    check(bl, tensors([1, 9, 4099, 70001], [F, B], seed=offset, offset=offset), 0.1)
    # source and destination of different alignment
    g = tensors([5001, 333], [F, B], seed=9, offset=offset)
    out = [torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)[1:] for t in g]
    c = bl.bitlinear_clip_grads(g, 0.1, out=out)
    for t, r in zip(g, out):
        assert torch.equal(r, (t.float() * c["coef"]).to(t.dtype))


def test_large(bl):
    g = [torch.randn(11008, 4096, device=DEV), torch.randn(30_000_001, device=DEV).to(B)]
    norm = float(torch.sqrt(sum((t.double() ** 2).sum() for t in g)))
    o = bl.bitlinear_clip_grads(g, 1.0, out=[torch.empty_like(t) for t in g])
    assert abs(float(o["norm"]) - norm) <= 2 * 2.0 ** -24 * norm
    for t, r in zip(g, o["grads"]):
        assert torch.equal(r, (t.float() * o["coef"]).to(t.dtype))


def test_no_clip(bl):
    g = tensors([1000, 17], [F, B], std=1e-5)
    o = check(bl, g, 1.0)
    assert float(o["coef"]) == 1.0
    for mn in (0.0, -1.0):
        assert float(bl.bitlinear_grad_norm(g, mn)["coef"]) == 1.0


def test_extremes(bl):
    """Squares beyond fp32's range both ways, and gradients that are not finite."""
    big = [torch.full((5000,), 1e30, device=DEV), torch.full((7,), -1e30, device=DEV)]
    o = bl.bitlinear_grad_norm(big, 1.0)
    assert abs(float(o["norm"]) / (1e30 * np.sqrt(5007)) - 1) < 1e-6 and 0 < float(o["coef"]) < 1e-30
    small = [torch.full((5000,), 1e-30, device=DEV)]
    o = bl.bitlinear_grad_norm(small, 1.0)
    assert abs(float(o["norm"]) / (1e-30 * np.sqrt(5000)) - 1) < 1e-6 and float(o["coef"]) == 1.0
    zero = [torch.zeros(100, device=DEV)]
    o = bl.bitlinear_clip_grads(zero, 1.0)
    assert float(o["norm"]) == 0.0 and float(o["coef"]) == 1.0 and float(zero[0].abs().max()) == 0.0
    for bad, coef in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        g = [torch.ones(100, device=DEV), torch.ones(9000, device=DEV)]
        g[1][8999] = bad
        o = bl.bitlinear_clip_grads(g, 1.0)
        torch.cuda.synchronize()
        assert not np.isfinite(float(o["norm"]))
        assert np.array_equal(np.float32(float(o["coef"])), np.float32(coef), equal_nan=True)
        assert np.array_equal(g[0].cpu().numpy(), np.full(100, coef, np.float32), equal_nan=True)


def test_repeatable_and_ordered(bl):
    g = tensors([70001, 3, 4096, 999], [F, B], seed=4)
    first = bl.bitlinear_grad_norm(g, 0.5)
    for _ in range(20):
        o = bl.bitlinear_grad_norm(g, 0.5)
        assert torch.equal(o["norm"], first["norm"]) and torch.equal(o["coef"], first["coef"])


def test_graph(bl):
    g = tensors([5000, 33], [F, B], seed=5)
    src = [t.clone() for t in g]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = bl.bitlinear_clip_grads(g, 0.1)
    for scale in (1.0, 2.0, 0.5):
        for t, u in zip(g, src):
            t.copy_(u * scale)
        want = bl.bitlinear_clip_grads([t.clone() for t in g], 0.1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["norm"], want["norm"])
        for t, r in zip(g, want["grads"]):
            assert torch.equal(t, r)
    del graph


@pytest.mark.parametrize("N,K", [(16, 32), (48, 160), (512, 256), (272, 4096)])
@pytest.mark.parametrize("hp", [HP, HP_LOUD])
def test_optimizer_step_with_coef(bl, N, K, hp):
    """Two matrices under one global clip, three steps, against the oracle's step with the
    coefficient of the joint norm (the oracle takes it as a per-matrix threshold that gives the
    same coefficient: a gradient scaled by it beforehand, and no clip)."""
    states = [_state(N, K, seed=N + K + i) for i in range(2)]
    on = [[t.to(DEV) for t in s] for s in states]
    step = [torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2)]
    for t in range(1, 4):
        dW = [synth.normal((N, K), 0.3 * t, synth.generator(N * K + i)).to(DEV) for i in range(2)]
        o = bl.bitlinear_grad_norm(dW, 1.0)
        coef = float(o["coef"])
        assert 0 < coef < 1
        for i in range(2):
            W, m, v = on[i]
            W0, m0, v0 = np_(W).copy(), np_(m).copy(), np_(v).copy()
            bl.bitlinear_optimizer_step(W, dW[i], m, v, step[i], coef=o["coef"], **hp)
            torch.cuda.synchronize()
            assert int(step[i]) == t
            g = (dW[i] * o["coef"]).cpu()               # the kernel's own first product, rounded once
            Wo, mo, vo, c = oracle.optimizer_step(W0, g, m0, v0, t, max_norm=0.0, **hp)
            assert c == 1.0
            bm, bv, bw = _bounds(W0, g.numpy(), m0, v0, 1.0, mo, vo, t, hp)
            assert np.all(np.abs(np_(m).astype(np.float64) - mo) <= bm)
            assert np.all(np.abs(np_(v).astype(np.float64) - vo) <= bv)
            assert np.all(np.abs(np_(W).astype(np.float64) - Wo) <= bw)


def test_optimizer_step_coef_matches_own_clip(bl):
    """With one matrix the global clip is the per-matrix clip: the same bits, codes included."""
    N, K = 272, 512
    W, m, v = _state(N, K, seed=3)
    dW = synth.normal((N, K), 0.05, synth.generator(4)).to(DEV)
    got = []
    for use in (False, True):
        on = [t.to(DEV) for t in (W, m, v)]
        step = torch.zeros(1, dtype=torch.int32, device=DEV)
        coef = bl.bitlinear_grad_norm([dW], 1.0)["coef"] if use else None
        for _ in range(2):
            q = bl.bitlinear_optimizer_step(on[0], dW, on[1], on[2], step, requantize=True, coef=coef, **HP)
        got.append(on + [q[k] for k in sorted(q)] + [step])
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_binding_refusals(bl):
    g = tensors([100, 64], [F])
    call = bl.bitlinear_clip_grads
    for bad in ([], [g[0].cpu()], [g[0].double()], [g[0].view(10, 10).t()], [g[0], g[1].cpu()]):
        with pytest.raises(ValueError):
            call(bad, 1.0)
    with pytest.raises(ValueError):
        call(g, 1.0, out=[g[0]])
    with pytest.raises(ValueError):
        call(g, 1.0, out=[g[0], g[1].to(B)])
    with pytest.raises(ValueError):                      # clipped twice
        call([g[0], g[0]], 1.0)
    with pytest.raises(_lib.BitLinearError):
        call(g, float("nan"))
    with pytest.raises(_lib.BitLinearError):
        call(g, 1.0, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    W = torch.zeros(16, 32, device=DEV)
    step = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        bl.bitlinear_optimizer_step(W, W[:8], W.clone(), W.clone(), step, coef=torch.ones(1, device=DEV))
    with pytest.raises(ValueError):
        bl.bitlinear_optimizer_step(W, W.clone(), W.clone(), W.clone(), step, coef=torch.ones(1))
    torch.cuda.synchronize()
