"""The new calls together, as a stack of blocks uses them: a training step of two blocks (ternary,
then 8-bit) with the residual norms between them, their gradients, the global clip and the optimizer
step, and a single decoded token through the same layers."""
import numpy as np
import pytest
import torch

import operator_ref as ref
from bit_ternary_qat_b200 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16
K = 512


def weights(seed):
    gen = synth.generator(seed)
    W = [synth.normal((K, K), 0.02, gen).to(DEV) for _ in range(2)]
    g = [(1 + synth.normal((K,), 0.1, gen)).to(DEV) for _ in range(4)]
    gate = (0.5 + synth.normal((K,), 0.1, gen)).to(DEV)
    return W, g, gate


def forward(bl, x, W, g, gate):
    """x -> norm, ternary linear -> x1, norm -> 8-bit linear -> x2 (residual stream fp32)."""
    q1, q2 = bl.bitlinear_quant_weight(W[0]), bl.bitlinear_quant_weight_int8(W[1])
    zero = torch.zeros(x.shape, dtype=B, device=DEV)
    n0 = bl.bitlinear_residual_norm(x, zero, post_norm=False, g_pre=g[0])          # the first block's norm
    y1, _ = bl.bitlinear_linear(n0["xq"], n0["sx"], q1["wq_i8"], q1["gamma"])
    n1 = bl.bitlinear_residual_norm(n0["x"], y1, g_post=g[1], gate=gate, beta=0.7, g_pre=g[2])
    y2, _ = bl.bitlinear_linear_int8(n1["xq"], n1["sx"], q2["wq_i8"], q2["gamma_rows"])
    n2 = bl.bitlinear_residual_norm(n1["x"], y2, g_post=g[3], alpha=0.9, mode="none")
    return q1, q2, n0, y1, n1, y2, n2


def backward(bl, dx2, parts, W, g, gate):
    q1, q2, n0, y1, n1, y2, n2 = parts
    one = torch.ones(1, device=DEV)
    b2 = bl.bitlinear_residual_norm_backward(dx2, None, n2["x"], y2, r_post=n2["r_post"], g_post=g[3], alpha=0.9)
    dh1 = bl.bitlinear_grad_input(b2["dy"], q2["wq_bf16"], one)
    dW2 = bl.bitlinear_backward_weight(b2["dy"], n1["xdq"])
    b1 = bl.bitlinear_residual_norm_backward(b2["dx"], dh1, n1["x"], y1, r_post=n1["r_post"], r_pre=n1["r_pre"],
                                             g_post=g[1], gate=gate, beta=0.7, g_pre=g[2], out={"dx": b2["dx"]})
    dh0 = bl.bitlinear_grad_input(b1["dy"], q1["wq_bf16"], q1["gamma"])
    dW1 = bl.bitlinear_backward_weight(b1["dy"], n0["xdq"])
    return b2, dh1, dW2, b1, dh0, dW1


def test_training_step(bl):
    T = 96
    W, g, gate = weights(1)
    x = synth.normal((T, K), 1.0, synth.generator(2)).to(DEV)
    dx2 = synth.normal((T, K), 1e-2, synth.generator(3)).to(DEV)
    parts = forward(bl, x, W, g, gate)
    q1, q2, n0, y1, n1, y2, n2 = parts
    assert torch.equal(n0["x"], x)                        # a zero block leaves the stream as it is
    keep = dx2.clone()
    b2, dh1, dW2, b1, dh0, dW1 = backward(bl, dx2, parts, W, g, gate)
    torch.cuda.synchronize()
    assert bl.check_device_status() == 0 and torch.equal(dx2, keep)
    # the residual stream and each layer's gradients against fp64 autograd, the quantisers passed
    # straight through and the forward's codes held: 2e-3 of the largest value, the framework's
    # tolerance for its bf16 paths, each of the four bf16 roundings on a path being 2^-8 of an element
    d = lambda t: t.detach().cpu().double()
    leaves = {k: d(v).requires_grad_() for k, v in dict(x=x, W1=q1["wq_i8"].float() * q1["gamma"],
                                                         W2=q2["wq_bf16"], g0=g[0], g1=g[1], g2=g[2], g3=g[3],
                                                         gate=gate).items()}

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)

    def held(v, value):                                   # value forward, identity backward
        return v + (d(value) - v).detach()
    h0 = held(rms(leaves["x"]) * leaves["g0"], n0["xdq"])
    s1 = held(h0 @ leaves["W1"].t(), y1)
    x1 = held(leaves["x"] + 0.7 * leaves["gate"] * rms(s1) * leaves["g1"], n1["x"])
    h1 = held(rms(x1) * leaves["g2"], n1["xdq"])
    s2 = held(h1 @ leaves["W2"].t(), y2)
    x2 = 0.9 * x1 + rms(s2) * leaves["g3"]
    assert float((d(x2) - d(n2["x"])).abs().max()) <= 2.0 ** -20 * float(d(x2).abs().max())
    (x2 * d(dx2)).sum().backward()
    back = bl.bitlinear_residual_norm_backward(b1["dx"], dh0, n0["x"], torch.zeros_like(y1), r_pre=n0["r_pre"],
                                               g_pre=g[0])
    for got, want in ((dW2, leaves["W2"]), (dW1, leaves["W1"]), (back["dx"], leaves["x"]),
                      (b2["dpost_gain"], leaves["g3"]), (b1["dpost_gain"], leaves["g1"]),
                      (b1["dpre_gain"], leaves["g2"]), (b1["dgate"], leaves["gate"]), (back["dpre_gain"], leaves["g0"])):
        w = want.grad
        assert float((d(got) - w).abs().max()) <= 4 * 2e-3 * float(w.abs().max())
    # clip over everything, then the step
    grads = [dW1, dW2, b2["dpost_gain"], b1["dpost_gain"], b1["dpre_gain"], b1["dgate"], back["dpre_gain"]]
    c = bl.bitlinear_grad_norm(grads, 0.05)
    norm = float(torch.sqrt(sum((t.double() ** 2).sum() for t in grads)))
    assert abs(float(c["norm"]) - norm) <= 2.0 ** -22 * norm and float(c["coef"]) < 1
    before = [w.clone() for w in W]
    for w, dw in zip(W, (dW1, dW2)):
        m, v = torch.zeros_like(w), torch.zeros_like(w)
        step = torch.zeros(1, dtype=torch.int32, device=DEV)
        bl.bitlinear_optimizer_step(w, dw, m, v, step, coef=c["coef"])
        assert torch.equal(m, ((dw * c["coef"]) * torch.tensor(1.0 - np.float64(np.float32(0.9)), dtype=F).item()))
    assert all(not torch.equal(a, b) for a, b in zip(W, before))


def test_training_step_captured(bl):
    """Forward, backward, clip and step in one graph, replayed: the same bits as eager calls, while
    an eager graph's buffers live."""
    T = 40
    x = synth.normal((T, K), 1.0, synth.generator(5)).to(DEV)
    dx2 = synth.normal((T, K), 1e-2, synth.generator(6)).to(DEV)

    def one_step(W, m, v, step, g, gate):
        parts = forward(bl, x, W, g, gate)
        _, _, dW2, b1, _, dW1 = backward(bl, dx2, parts, W, g, gate)
        c = bl.bitlinear_grad_norm([dW1, dW2, b1["dgate"]], 0.05)
        for i, dw in enumerate((dW1, dW2)):
            bl.bitlinear_optimizer_step(W[i], dw, m[i], v[i], step[i], coef=c["coef"])
        return parts[-1]["x"], c["norm"]

    def state():
        W, g, gate = weights(4)
        return (W, [torch.zeros_like(w) for w in W], [torch.zeros_like(w) for w in W],
                [torch.zeros(1, dtype=torch.int32, device=DEV) for _ in W], g, gate)
    eager = state()
    want = [one_step(*eager) for _ in range(3)]
    torch.cuda.synchronize()
    held = state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            out = one_step(*held)
    torch.cuda.current_stream().wait_stream(stream)
    for x2, norm in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], x2) and torch.equal(out[1], norm)
    for a, b in zip(eager[0] + eager[1] + eager[2] + eager[3], held[0] + held[1] + held[2] + held[3]):
        assert torch.equal(a, b)
    assert bl.check_device_status() == 0
    del graph


def test_decode_matches_the_batch(bl):
    """One token at a time gives the batch's rows, bit for bit (residual stream and 8-bit product)."""
    W, g, gate = weights(7)
    x = synth.normal((6, K), 1.0, synth.generator(8)).to(DEV)
    parts = forward(bl, x, W, g, gate)
    for t in range(6):
        one = forward(bl, x[t:t + 1].contiguous(), W, g, gate)
        for a, b in zip((parts[4], parts[6]), (one[4], one[6])):
            for k in a:
                assert torch.equal(a[k][t:t + 1], b[k]), k
        assert torch.equal(parts[5][t:t + 1], one[5])


def test_two_streams_at_once(bl):
    """Independent calls on two streams, each with its own workspace."""
    W, g, gate = weights(9)
    xs = [synth.normal((700, K), 1.0, synth.generator(i)).to(DEV) for i in (10, 11)]
    want = [forward(bl, x, W, g, gate)[-1]["x"] for x in xs]
    norms = [bl.bitlinear_grad_norm([x, W[i]], 1.0)["norm"] for i, x in enumerate(xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None, None]
    for rep in range(4):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = (forward(bl, xs[i], W, g, gate)[-1]["x"], bl.bitlinear_grad_norm([xs[i], W[i]], 1.0)["norm"])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i][0], want[i]) and torch.equal(got[i][1], norms[i])
    assert ref.CHAIN > 0 and bl.check_device_status() == 0
