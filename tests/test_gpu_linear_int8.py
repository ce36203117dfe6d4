"""The 8-bit weight quantiser and the 8-bit linear, all compared exactly: the codes and scales
against one fp32 rounding an operation, the accumulators as whole numbers, Y as
fl(fl(acc gamma_n) fl(1 / s_t)) rounded once to its type."""
import numpy as np
import pytest
import torch

from bit_ternary_qat_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def operands(T, N, K, seed):
    gen = torch.Generator().manual_seed(seed)
    xq = torch.randint(-128, 128, (T, K), generator=gen, dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int8)
    sx = torch.rand(T, generator=gen) * 190 + 10
    gm = torch.rand(N, generator=gen) * 1e-2 + 1e-4
    return [t.to(DEV) for t in (xq, sx, wq, gm)]


def check(bl, T, N, K, seed=0, out_dtype=F):
    xq, sx, wq, gm = operands(T, N, K, seed + 3 * T + 5 * N + K)
    y, acc = bl.bitlinear_linear_int8(xq, sx, wq, gm, out_dtype=out_dtype, want_acc=True)
    y2, none = bl.bitlinear_linear_int8(xq, sx, wq, gm, out_dtype=out_dtype)
    torch.cuda.synchronize()
    assert bl.check_device_status() == 0
    want = xq.double() @ wq.double().t()              # whole numbers below 2^53
    assert torch.equal(acc.double(), want)
    r = torch.from_numpy(np.float32(1) / sx.cpu().numpy()[:, None])
    yw = (acc.cpu().to(F) * gm.cpu()[None, :] * r).to(out_dtype)
    assert torch.equal(y.cpu(), yw)
    assert none is None and torch.equal(y2, y)


TOKENS = [1, 2, 3, 7, 8, 15, 16, 17, 31, 33, 48, 64, 65, 100, 127, 128, 129, 160, 200, 255, 256, 257, 300, 512, 513]


@pytest.mark.parametrize("T", TOKENS)
def test_tokens(bl, T):
    check(bl, T, 272, 160, out_dtype=F if T % 2 else B)
    check(bl, T, 4096, 1024, out_dtype=B if T % 2 else F)


@pytest.mark.parametrize("N,K", [(16, 32), (16, 16384), (48, 96), (112, 4096), (144, 2080), (2048, 2048),
                                 (4096, 11008), (11008, 4096), (20480, 512), (40000, 64), (32, 30016)])
def test_shapes(bl, N, K):
    for T in (1, 5, 37, 96, 250):
        check(bl, T, N, K, out_dtype=F if T % 2 else B)


@pytest.mark.parametrize("T,N,K", [(519, 720, 12480), (1131, 64, 7072), (2000, 512, 8192), (700, 256, 16384),
                                   (300, 48, 1024), (5000, 16, 4096), (4097, 32, 32), (1300, 1040, 160)])
def test_several_token_tiles(bl, T, N, K):
    """More tokens than one tile, with few weight rows: tiles of both kinds, split and whole."""
    check(bl, T, N, K, out_dtype=B)
    check(bl, T, N, K, out_dtype=F)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(bl, seed):
    rng = np.random.default_rng(seed)
    T = int(np.exp(rng.uniform(0, np.log(700))))
    N = 16 * int(np.exp(rng.uniform(0, np.log(600))))
    K = 32 * int(np.exp(rng.uniform(0, np.log(300))))
    check(bl, T, N, K, seed=seed, out_dtype=[F, B][seed % 2])


def test_sums_at_the_limit(bl):
    """K just below 2^17 of the extreme codes: 2^31 - 2^19 in the accumulator."""
    K = (1 << 17) - 32
    for T in (1, 40, 300):
        xq = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
        wq = torch.full((16, K), -128, dtype=torch.int8, device=DEV)
        y, acc = bl.bitlinear_linear_int8(xq, torch.ones(T, device=DEV), wq, torch.ones(16, device=DEV), out_dtype=F,
                                          want_acc=True)
        assert bool((acc == 128 * 128 * K).all())


def test_large_single_token(bl):
    check(bl, 1, 28672, 8192, out_dtype=B)
    check(bl, 16, 28672, 8192, out_dtype=F)


def test_repeatable_behind_itself(bl):
    """Back-to-back calls of different shapes on one stream: no state survives a call."""
    ops = [operands(T, N, K, T) for T, N, K in ((1, 4096, 4096), (64, 2048, 8192), (200, 4096, 2048), (5, 16, 32))]
    first = [bl.bitlinear_linear_int8(a[0], a[1], a[2], a[3], want_acc=True) for a in ops]
    for _ in range(16):
        for a, (y, acc) in zip(ops, first):
            y2, acc2 = bl.bitlinear_linear_int8(a[0], a[1], a[2], a[3], want_acc=True)
            assert torch.equal(acc2, acc) and torch.equal(y2, y)
    assert bl.check_device_status() == 0


def test_nothing_outside_is_written(bl):
    for T, N, K in ((1, 16, 64), (3, 48, 512), (37, 272, 1024), (130, 4112, 256)):
        xq, sx, wq, gm = operands(T, N, K, 1)
        for dt in (F, B):
            flat = torch.full((T * N + 256,), 7.0, dtype=dt, device=DEV)
            fa = torch.full((T * N + 256,), 7, dtype=torch.int32, device=DEV)
            bl.bitlinear_linear_int8(xq, sx, wq, gm, y=flat[:T * N].view(T, N), acc=fa[:T * N].view(T, N))
            torch.cuda.synchronize()
            assert bool((flat[T * N:] == 7.0).all()) and bool((fa[T * N:] == 7).all())


def test_graph_and_side_stream(bl):
    cases = [operands(T, 1024, 2048, T) for T in (1, 40, 300)]
    want = [bl.bitlinear_linear_int8(a[0], a[1], a[2], a[3])[0] for a in cases]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000)
        got = [bl.bitlinear_linear_int8(a[0], a[1], a[2], a[3])[0] for a in cases]
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [bl.bitlinear_linear_int8(a[0], a[1], a[2], a[3])[0] for a in cases]
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    del graph


@pytest.mark.parametrize("N,K", [(16, 32), (48, 160), (272, 4096), (1024, 2048), (32, 16416), (64, 65536)])
def test_quant_weight(bl, N, K):
    gen = torch.Generator().manual_seed(N + K)
    W = torch.randn(N, K, generator=gen) * torch.exp(torch.randn(N, 1, generator=gen))
    W[1] = 0                                             # a row of zeros, one below the floor, one of ties
    W[2] *= 1e-9
    W[3] = torch.arange(K).remainder(255).sub(127).float() * 0.5
    W[4, K - 1] = -1e30
    o = bl.bitlinear_quant_weight_int8(W.to(DEV))
    torch.cuda.synchronize()
    w = W.numpy()
    m = np.maximum(np.abs(w).max(1), np.float32(1e-5))
    gm, q = m / np.float32(127), np.rint(w * (np.float32(127) / m)[:, None])
    assert np.array_equal(o["gamma_rows"].cpu().numpy(), gm)
    assert np.array_equal(o["wq_i8"].cpu().numpy(), q.astype(np.int8)) and np.abs(q).max() == 127
    gb = torch.from_numpy(gm).to(B).float()
    assert torch.equal(o["wq_bf16"].cpu(), (torch.from_numpy(q) * gb[:, None]).to(B))
    only = bl.bitlinear_quant_weight_int8(W.to(DEV), want_bf16=False)
    assert "wq_bf16" not in only and torch.equal(only["wq_i8"], o["wq_i8"])


def test_straight_through_gradients(bl):
    """An 8-bit layer's training step: the framework's backward takes the bf16 operand with a
    gamma of 1.  Products of bf16 values summed in fp32: 2e-3 of the largest value, the
    framework's tolerance for its bf16 paths."""
    T, N, K = 96, 272, 256
    gen = torch.Generator().manual_seed(2)
    X, W = torch.randn(T, K, generator=gen).to(B).to(DEV), (0.05 * torch.randn(N, K, generator=gen)).to(DEV)
    dY = (1e-2 * torch.randn(T, N, generator=gen)).to(B).to(DEV)
    q = bl.bitlinear_quant_weight_int8(W)
    a = bl.bitlinear_act_quant(X)
    y, _ = bl.bitlinear_linear_int8(a["xq"], a["sx"], q["wq_i8"], q["gamma_rows"])
    one = torch.ones(1, device=DEV)
    dx = bl.bitlinear_grad_input(dY, q["wq_bf16"], one)
    dw = bl.bitlinear_backward_weight(dY, a["xdq"])
    torch.cuda.synchronize()
    wd, xd = q["wq_i8"].double() * q["gamma_rows"].double()[:, None], a["xq"].double() / a["sx"].double()[:, None]
    for got, want, tol in ((y, xd @ wd.t(), 2.0 ** -8 + 2.0 ** -20), (dx, dY.double() @ q["wq_bf16"].double(), 2e-3),
                           (dw, dY.double().t() @ a["xdq"].double(), 2e-3)):
        assert float((got.double() - want).abs().max()) <= tol * float(want.abs().max())
    # the bf16 operand: gamma rounded once, its product with the code once
    assert bool(((q["wq_bf16"].double() - wd).abs() <= (2.0 ** -7 + 2.0 ** -15) * wd.abs()).all())


def test_binding_refusals(bl):
    xq, sx, wq, gm = operands(4, 32, 64, 0)
    call = bl.bitlinear_linear_int8
    for a in ((xq.float(), sx, wq, gm), (xq, sx[:3], wq, gm), (xq, sx, wq[:, :32].contiguous(), gm),
              (xq, sx, wq, gm[:16]), (xq, sx, wq.t(), gm), (xq.cpu(), sx, wq, gm), (xq, sx.double(), wq, gm)):
        with pytest.raises(ValueError):
            call(*a)
    with pytest.raises(ValueError):
        call(xq, sx, wq, gm, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        call(xq, sx, wq, gm, y=torch.empty(4, 16, device=DEV))
    with pytest.raises(_lib.BitLinearError):
        call(xq, sx, wq[:24].contiguous(), gm[:24].contiguous())
    big = torch.zeros(16, 1 << 17, dtype=torch.int8, device=DEV)
    with pytest.raises(_lib.BitLinearError):
        call(big[:1], sx[:1], big, torch.ones(16, device=DEV))
    torch.cuda.synchronize()
