"""The residual norms and their gradient against fp64 forms, with bounds counted in roundings
(operator_ref.py); the quantised output against the framework's activation quantiser."""
import numpy as np
import pytest
import torch

import operator_ref as ref
from bit_ternary_qat_b200 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16
TYPES = [(F, F), (B, B), (F, B)]
GATES = ["none", "scalar", "channel", "token", "element"]
# rows enough for the forward's shared-memory ring, whole vectors and odd ones, in every group size
RING = [(6200, 256), (3100, 512), (1600, 1000), (800, 2048), (420, 4096), (200, 8192), (150, 11008), (100, 16384),
        (3400, 500), (3601, 499), (1601, 1001), (500, 4001), (200, 8191), (130, 12289), (100, 16381)]
# warp rows, block rows of every block size, and rows that are no whole vectors
SIZES = [(1, 1), (3, 7), (5, 8), (9, 33), (2, 96), (40, 250), (17, 256), (300, 512), (77, 1003), (6, 1024), (1, 2048),
         (13, 4096), (4, 5000), (3, 5001), (5, 11008), (2, 16384), (2, 16381)]


def close(got, want, bound, what):
    err = (ref.f64(got) - want).abs()
    bad = err > bound
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / bound).max()):.3g} bounds"


def check_forward(bl, T, K, xt, yt, gate, post, gains, mode, alpha=0.9, beta=0.7, seed=0):
    s = ref.inputs(T, K, xt, yt, gate, seed + 7 * T + K, DEV, post, gains)
    if mode == "none":
        s["g_pre"] = None
    o = bl.bitlinear_residual_norm(**s, post_norm=post, alpha=alpha, beta=beta, mode=mode)
    torch.cuda.synchronize()
    new, bound, r1 = ref.forward(s["x"], s["y"], s["g_post"], s["gate"], alpha, beta, post)
    close(o["x"], new, bound + ref.STORE[xt] * (new.abs() + bound), "x")
    if post:
        close(o["r_post"], r1, 2 * ref.HALF * r1, "r_post")
    else:
        assert "r_post" not in o
    if mode == "none":
        assert set(o) <= {"x", "r_post"}
        return
    h, r2 = ref.pre_norm(o["x"], s["g_pre"])
    close(o["r_pre"], r2, 2 * ref.HALF * r2, "r_pre")
    if mode == "norm":
        close(o["h"], h, (5 * ref.HALF + ref.STORE[yt]) * h.abs() + ref.TINY, "h")
        return
    # the codes from the stored residual and statistic, one fp32 rounding an operation
    held, r = o["x"].float().cpu().numpy(), o["r_pre"].cpu().numpy()
    xh = held * r[:, None]
    if s["g_pre"] is not None:
        xh = xh * s["g_pre"].cpu().numpy()
    sx = np.float32(127.0) / np.maximum(np.abs(xh).max(1), np.float32(1e-5))
    q = np.rint(xh * sx[:, None])
    assert np.array_equal(o["sx"].cpu().numpy(), sx)
    assert np.array_equal(o["xq"].cpu().numpy(), q.astype(np.int8))
    assert torch.equal(o["xdq"].cpu(), torch.from_numpy(q / sx[:, None]).to(yt))
    if xt == yt:
        a = bl.bitlinear_act_quant(o["x"], g=s["g_pre"])
        assert torch.equal(a["xq"], o["xq"]) and torch.equal(a["sx"], o["sx"]) and torch.equal(a["xdq"], o["xdq"])
        assert torch.equal(a["rinv"], o["r_pre"])


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("i", range(3))
def test_forward_sizes(bl, T, K, i):
    xt, yt = TYPES[i]
    mode = ["quant" if K % 32 == 0 else "norm", "norm", "none"][(T + i) % 3]
    check_forward(bl, T, K, xt, yt, GATES[(T + K + i) % 5], (T + i) % 4 != 0, (K + i) % 3 != 0, mode)


@pytest.mark.parametrize("T,K", RING)
@pytest.mark.parametrize("i", range(3))
def test_forward_ring(bl, T, K, i):
    xt, yt = TYPES[i]
    for n, mode in enumerate(["quant", "norm", "none"] if K % 32 == 0 else ["norm", "norm", "none"]):
        check_forward(bl, T, K, xt, yt, GATES[(T + i + n) % 5], (K // 8 + i + n) % 4 != 0, (T + i + n) % 3 != 0, mode)
    check_backward(bl, T, K, xt, yt, GATES[(T + i) % 5], (K // 8 + i) % 4 != 0, True, True, True)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("types", range(3))
@pytest.mark.parametrize("post", [True, False])
def test_forward_gates(bl, gate, types, post):
    for T, K in ((19, 160), (5, 4096)):
        for mode in ("quant", "norm", "none"):
            check_forward(bl, T, K, *TYPES[types], gate, post, True, mode)
    check_forward(bl, 21, 77, *TYPES[types], gate, post, True, "norm")


def run_backward(bl, s, o, dx, dh, alpha, beta, post, **kw):
    return bl.bitlinear_residual_norm_backward(dx, dh, o["x"], s["y"], r_post=o.get("r_post") if post else None,
                                               r_pre=o.get("r_pre") if dh is not None else None, g_post=s["g_post"],
                                               gate=s["gate"], alpha=alpha, beta=beta,
                                               g_pre=s["g_pre"] if dh is not None else None, **kw)


def check_backward(bl, T, K, xt, yt, gate, post, gains, with_dx, with_dh, alpha=0.9, beta=0.7):
    s = ref.inputs(T, K, xt, yt, gate, 3 * T + K, DEV, post, gains)
    o = bl.bitlinear_residual_norm(**s, post_norm=post, alpha=alpha, beta=beta, mode="norm")
    gen = torch.Generator().manual_seed(T + K)
    dx = (1e-2 * torch.randn(T, K, generator=gen)).to(DEV) if with_dx else None
    dh = (1e-2 * torch.randn(T, K, generator=gen)).to(DEV) if with_dh else None
    got = run_backward(bl, s, o, dx, dh, alpha, beta, post)
    torch.cuda.synchronize()
    want = ref.backward(dx, dh, o["x"], s["y"], o["r_post"] if post else None, o["r_pre"] if with_dh else None,
                        s["g_post"], s["g_pre"] if with_dh else None, s["gate"], alpha, beta, yt)
    assert set(got) == set(want)
    for k, (v, b) in want.items():
        assert got[k].shape == v.shape
        close(got[k], v, b, k)


@pytest.mark.parametrize("T,K", SIZES + [(700, 64), (1500, 8), (300, 4096), (160, 8192), (151, 11008)])
@pytest.mark.parametrize("i", range(3))
def test_backward_sizes(bl, T, K, i):
    xt, yt = TYPES[i]
    check_backward(bl, T, K, xt, yt, GATES[(T + K + i) % 5], (T + i) % 4 != 0, (K + i) % 3 != 0,
                   (T + i) % 5 != 0, (T + i) % 7 != 1 or (T + i) % 5 == 0)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("types", range(3))
@pytest.mark.parametrize("post", [True, False])
def test_backward_gates(bl, gate, types, post):
    for T, K in ((19, 160), (5, 4096), (3, 9216), (21, 77)):
        for with_dx, with_dh in ((True, True), (False, True), (True, False)):
            check_backward(bl, T, K, *TYPES[types], gate, post, True, with_dx, with_dh)


@pytest.mark.parametrize("gate", GATES)
def test_backward_against_differences(bl, gate):
    """<gradient, direction> against central differences of the fp64 forward."""
    T, K, alpha, beta = 11, 264, 0.8, 0.6
    s = ref.inputs(T, K, F, F, gate, 5, DEV)
    o = bl.bitlinear_residual_norm(**s, alpha=alpha, beta=beta, mode="norm")
    gen = torch.Generator().manual_seed(6)
    dx, dh = torch.randn(T, K, generator=gen).to(DEV), torch.randn(T, K, generator=gen).to(DEV)
    got = run_backward(bl, s, o, dx, dh, alpha, beta, True)
    torch.cuda.synchronize()
    wx, wh = ref.f64(dx), ref.f64(dh)

    def loss(x, y, g_post, g_pre, gt):
        r1 = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + 1e-6)
        new = alpha * x + beta * y * r1 * g_post * (1.0 if gt is None else gt)
        r2 = 1.0 / torch.sqrt((new * new).mean(1, keepdim=True) + 1e-6)
        return float((wx * new).sum() + (wh * new * r2 * g_pre).sum())

    at = [ref.f64(s[k]) for k in ("x", "y", "g_post", "g_pre", "gate")]
    for i, name in enumerate(["dx", "dy", "dpost_gain", "dpre_gain", "dgate"]):
        if at[i] is None:
            continue
        v = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
        step = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * v, at[i] - step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        along = ref.f64(got[name]) * v
        # the differences' own error is step^2; fp32 gradients are off by their bounds' size
        assert abs(float(along.sum()) - diff) <= 1e-4 * float(along.abs().sum()) + 1e-6, name


@pytest.mark.parametrize("T,K", [(6, 1024), (5, 1003), (3, 9216)])
def test_backward_of_large_and_small_rows(bl, T, K):
    """Rows far from 1: the statistic's cube leaves fp32 (1e-60, 1e9), the gradient does not."""
    s = ref.inputs(T, K, F, F, "channel", 15, DEV)
    for i, f in enumerate([1e20, 1e-4, 1.0][:T]):
        s["x"][i] *= f
        s["y"][i] *= f
    o = bl.bitlinear_residual_norm(**s, mode="norm")
    gen = torch.Generator().manual_seed(T)
    dh = torch.randn(T, K, generator=gen).to(DEV)
    for row in range(T):                                  # a row alone: column sums of one scale
        one = dict(s, x=s["x"][row:row + 1].clone(), y=s["y"][row:row + 1].clone())
        o1 = bl.bitlinear_residual_norm(**one, mode="norm")
        d1 = dh[row:row + 1].clone()
        got = run_backward(bl, one, o1, None, d1, 1.0, 1.0, True)
        torch.cuda.synchronize()
        want = ref.backward(None, d1, o1["x"], one["y"], o1["r_post"], o1["r_pre"], s["g_post"], s["g_pre"], s["gate"],
                            1.0, 1.0, F)
        for k, (v, b) in want.items():
            close(got[k], v, b, f"{k} of row {row}")
    assert torch.equal(o["x"][0:1], bl.bitlinear_residual_norm(**dict(s, x=s["x"][:1].clone(), y=s["y"][:1].clone()),
                                                              mode="norm")["x"])


def test_in_place(bl):
    """The new residual over the old one, and the gradient over either incoming one."""
    for (T, K), (xt, yt) in [((33, 1184), t) for t in TYPES] + [((1400, 1184), t) for t in TYPES]:
        s = ref.inputs(T, K, xt, yt, "channel", 8, DEV)
        o = bl.bitlinear_residual_norm(**s, mode="quant")
        x = s["x"].clone()
        o2 = bl.bitlinear_residual_norm(x, s["y"], g_post=s["g_post"], gate=s["gate"], g_pre=s["g_pre"], mode="quant",
                                        out={"x": x})
        assert o2["x"] is x and torch.equal(x, o["x"]) and torch.equal(o2["xq"], o["xq"])
        dx, dh = torch.randn(T, K, device=DEV), torch.randn(T, K, device=DEV)
        a = run_backward(bl, s, o, dx, dh, 1.0, 1.0, True)
        for which in range(2):
            d = [dx.clone(), dh.clone()]
            b = run_backward(bl, s, o, d[0], d[1], 1.0, 1.0, True, out={"dx": d[which]})
            assert b["dx"] is d[which]
            for k in a:
                assert torch.equal(a[k], b[k]), k


def test_rows_of_zeros_large_and_not_finite(bl):
    """Rows with nothing in them, squares beyond fp32, and a NaN that stays in its row."""
    K = 1024
    for K in (1024, 1003):
        s = ref.inputs(6, K, F, F, "none", 9, DEV, gains=False)
        s["x"][1] = 0
        s["y"][1] = 0
        s["y"][2] *= 1e25
        s["x"][3] *= 1e25
        s["y"][4, 5] = float("nan")
        s["x"][5] = 0
        o = bl.bitlinear_residual_norm(**s, mode="norm")
        torch.cuda.synchronize()
        assert float(o["x"][1].abs().max()) == 0 and float(o["h"][1].abs().max()) == 0
        assert float(o["r_pre"][1]) == float(np.float32(1.0 / np.sqrt(np.float64(np.float32(1e-6)))))
        ok = [0, 1, 2, 3, 5]
        new, bound, _ = ref.forward(s["x"], s["y"], None, None, 1.0, 1.0, True)
        close(o["x"][ok], new[ok], 2 * bound[ok], "x")
        h, _ = ref.pre_norm(o["x"], None)
        close(o["h"][ok], h[ok], 6 * ref.HALF * h[ok].abs() + ref.TINY, "h")
        assert bool(torch.isnan(o["h"][4]).all())


def test_quantised_row_of_zeros(bl):
    s = ref.inputs(3, 64, B, B, "none", 10, DEV)
    s["x"][1] = 0
    s["y"][1] = 0
    o = bl.bitlinear_residual_norm(**s, mode="quant")
    torch.cuda.synchronize()
    assert int(o["xq"][1].abs().max()) == 0 and float(o["sx"][1]) == float(np.float32(127) / np.float32(1e-5))
    assert float(o["xdq"][1].float().abs().max()) == 0


def test_repeatable_and_rows_independent(bl):
    """The same bits again, and a row's results do not depend on the rows beside it."""
    T, K = 900, 2048                          # many rows through the ring, one row without it
    s = ref.inputs(T, K, F, B, "channel", 11, DEV)
    o = bl.bitlinear_residual_norm(**s)
    dx, dh = torch.randn(T, K, device=DEV), torch.randn(T, K, device=DEV)
    g = run_backward(bl, s, o, dx, dh, 1.0, 1.0, True)
    for _ in range(5):
        o2 = bl.bitlinear_residual_norm(**s)
        g2 = run_backward(bl, s, o, dx, dh, 1.0, 1.0, True)
        assert all(torch.equal(o[k], o2[k]) for k in o) and all(torch.equal(g[k], g2[k]) for k in g)
    one = dict(s, x=s["x"][5:6].contiguous(), y=s["y"][5:6].contiguous())
    o1 = bl.bitlinear_residual_norm(**one)
    assert all(torch.equal(o[k][5:6], o1[k]) for k in o)
    g1 = run_backward(bl, one, o1, dx[5:6].contiguous(), dh[5:6].contiguous(), 1.0, 1.0, True)
    assert torch.equal(g["dx"][5:6], g1["dx"]) and torch.equal(g["dy"][5:6], g1["dy"])


def test_nothing_outside_is_written(bl):
    """Outputs at the end of larger buffers: what lies behind them stays."""
    for T, K in ((5, 72), (3, 1003), (2, 4096), (1700, 1001), (1600, 1000)):
        s = ref.inputs(T, K, F, F, "none", 12, DEV)
        pad = 64
        flat = {k: torch.full((T * K + pad,), 7.0, device=DEV) for k in ("x", "h", "dx", "dy")}
        v = {k: t[:T * K].view(T, K) for k, t in flat.items()}
        o = bl.bitlinear_residual_norm(**s, mode="norm", out={"x": v["x"], "h": v["h"]})
        run_backward(bl, s, o, torch.randn(T, K, device=DEV), torch.randn(T, K, device=DEV), 1.0, 1.0, True,
                     out={"dx": v["dx"], "dy": v["dy"]})
        torch.cuda.synchronize()
        for t in flat.values():
            assert bool((t[T * K:] == 7.0).all())


def test_graph_and_side_stream(bl):
    T, K = 64, 1024
    s = ref.inputs(T, K, B, B, "token", 13, DEV)
    dx, dh = torch.randn(T, K, device=DEV), torch.randn(T, K, device=DEV)
    o = bl.bitlinear_residual_norm(**s)
    want = run_backward(bl, s, o, dx, dh, 1.0, 1.0, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2_000_000)
        o2 = bl.bitlinear_residual_norm(**s)
        g2 = run_backward(bl, s, o2, dx, dh, 1.0, 1.0, True)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(o[k], o2[k]) for k in o) and all(torch.equal(want[k], g2[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3 = bl.bitlinear_residual_norm(**s)
        g3 = run_backward(bl, s, o3, dx, dh, 1.0, 1.0, True)
    for _ in range(3):
        for t in list(o3.values()) + list(g3.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], o3[k]) for k in o) and all(torch.equal(want[k], g3[k]) for k in want)
    del graph


def test_binding_refusals(bl):
    T, K = 4, 64
    s = ref.inputs(T, K, F, F, "none", 14, DEV)
    x, y = s["x"], s["y"]
    call = bl.bitlinear_residual_norm
    for kw in (dict(gate=torch.ones(K + 1, device=DEV)), dict(gate=torch.ones(T + 1, 1, device=DEV)),
               dict(gate=torch.ones(T, K, device=DEV, dtype=B)), dict(g_pre=torch.ones(K, device=DEV, dtype=B)),
               dict(g_post=torch.ones(K - 1, device=DEV)), dict(mode="codes"), dict(out={"x": x[:2]}),
               dict(gate=torch.ones(K))):
        with pytest.raises(ValueError):
            call(x, y, **kw)
    for a, b in ((x.t(), y), (x, y.t()), (x, y[:2]), (x.to(B), y), (x.cpu(), y), (x, y.double())):
        with pytest.raises(ValueError):
            call(a, b)
    with pytest.raises(_lib.BitLinearError):                        # g_post without the post norm
        call(x, y, post_norm=False, g_post=torch.ones(K, device=DEV))
    with pytest.raises(_lib.BitLinearError):                        # codes need K % 32 == 0
        call(x[:, :40].contiguous(), y[:, :40].contiguous(), mode="quant")
    o = call(x, y, mode="norm")
    with pytest.raises(_lib.BitLinearError):                        # no gradient comes in
        bl.bitlinear_residual_norm_backward(None, None, o["x"], y)
    with pytest.raises(ValueError):
        bl.bitlinear_residual_norm_backward(None, x, o["x"], y)     # dh needs r_pre
    with pytest.raises(ValueError):
        bl.bitlinear_residual_norm_backward(x.to(B), None, o["x"], y)
    torch.cuda.synchronize()
