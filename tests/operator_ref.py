"""fp64 forms of the residual norms and bounds on the kernels' rounding, for the tests.

The bounds count roundings: HALF is half an fp32 step relative to a value, STORE half a step of
the stored type.  A sum over K values is charged CHAIN additions (a thread's own chain, the
butterfly of a warp and the warps of a block: at most 16384 / 256 + 5 + 32 of them) of the sum of
magnitudes; a column sum over T rows the rows of one block's chain and the join behind it.
"""
import torch

HALF = 2.0 ** -24
STORE = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
CHAIN = 110.0
TINY = 1e-37          # below this fp32 products lose bits to the denormals


def f64(t):
    return None if t is None else t.detach().cpu().double()


def forward(x, y, g_post, gate, alpha, beta, post, eps=1e-6):
    """(x' before its rounding, its bound before rounding, r_post) in fp64."""
    x, y, g_post, gate = f64(x), f64(y), f64(g_post), f64(gate)
    n, r1 = y, None
    if post:
        r1 = 1.0 / torch.sqrt((y * y).mean(1) + eps)
        n = y * r1[:, None] * (1.0 if g_post is None else g_post)
    z = beta * n * (1.0 if gate is None else gate)
    new = alpha * x + z
    bound = HALF * (8.0 * z.abs() + 2.0 * (alpha * x).abs() + 2.0 * new.abs()) + TINY
    return new, bound, r1


def pre_norm(held, g_pre, eps=1e-6):
    """h and r_pre in fp64 from the residual as it is held."""
    held, g_pre = f64(held), f64(g_pre)
    r2 = 1.0 / torch.sqrt((held * held).mean(1) + eps)
    return held * r2[:, None] * (1.0 if g_pre is None else g_pre), r2


def backward(dx, dh, x, y, r_post, r_pre, g_post, g_pre, gate, alpha, beta, y_dtype, blocks=148):
    """{name: (value, bound)} of the gradients, from the formulas in fp64 with the saved
    statistics, and how far fp32 kernels may be off."""
    # a bf16 gate is an element gate also where it is [1, 1], and its gradient is held in bf16
    element = gate is not None and gate.dim() == 2 and (gate.shape[1] > 1 or gate.dtype is torch.bfloat16)
    dx, dh, x, y, g_post, g_pre, gate = (f64(t) for t in (dx, dh, x, y, g_post, g_pre, gate))
    r1, r2 = f64(r_post), f64(r_pre)
    T, K = y.shape
    cols = T / min(blocks, T) + 40.0               # a column's chain: its block's rows, then the join
    got = {}
    d = torch.zeros(T, K, dtype=torch.float64) if dx is None else dx
    ed = torch.zeros_like(d)                       # bound on d's error
    if dh is not None:
        g2 = 1.0 if g_pre is None else g_pre
        u, e = x * r2[:, None], dh * g2
        mag = (e * u).abs().mean(1, keepdim=True)
        d = d + r2[:, None] * (e - u * (e * u).mean(1, keepdim=True))
        ed = HALF * (2 * d.abs() + 6 * r2[:, None] * (e.abs() + u.abs() * mag) + CHAIN * r2[:, None] * u.abs() * mag)
        got["dpre_gain"] = ((dh * u).sum(0), HALF * (cols + 3) * (dh * u).abs().sum(0))
    got["dx"] = (alpha * d, abs(alpha) * (ed + HALF * 2 * d.abs()))
    p, ep = beta * d, abs(beta) * (ed + HALF * 2 * d.abs())
    g1 = 1.0 if g_post is None else g_post
    u = y if r1 is None else y * r1[:, None]
    n = u * g1
    if gate is not None:
        v, ev = p * n, ep * n.abs() + HALF * 5 * (p * n).abs()
        if element:
            got["dgate"] = (v, ev + STORE[y_dtype] * (v.abs() + ev))
        elif gate.dim() == 2:
            got["dgate"] = (v.sum(1, keepdim=True), (ev + HALF * CHAIN * v.abs()).sum(1, keepdim=True))
        elif gate.numel() == 1 and K > 1:
            got["dgate"] = (v.sum().reshape(1), (ev.sum() + HALF * CHAIN * v.abs().sum()).reshape(1))
        else:
            got["dgate"] = (v.sum(0), ev.sum(0) + HALF * cols * v.abs().sum(0))
        p, ep = p * gate, (ep + HALF * 2 * p.abs()) * gate.abs()
    if r1 is None:
        dy, edy = p, ep
    else:
        e, ee = g1 * p, abs(g1) * ep if g_post is None else g1.abs() * ep
        ee = ee + HALF * 2 * e.abs()
        mag = (e * u).abs().mean(1, keepdim=True)
        dy = r1[:, None] * (e - u * (e * u).mean(1, keepdim=True))
        emean = (ee * u.abs()).mean(1, keepdim=True) + HALF * CHAIN * mag
        edy = r1[:, None] * (ee + u.abs() * emean + HALF * 6 * (e.abs() + u.abs() * mag))
        got["dpost_gain"] = ((p * u).sum(0), (ep * u.abs()).sum(0) + HALF * (cols + 3) * (p * u).abs().sum(0))
    got["dy"] = (dy, edy + STORE[y_dtype] * (dy.abs() + edy))
    return {k: (v, b + TINY) for k, (v, b) in got.items()}


def inputs(T, K, x_dtype, y_dtype, gate, seed, dev, post=True, gains=True):
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)
    s = {"x": (randn(T, K) * torch.exp(0.5 * randn(K))).to(x_dtype), "y": (0.3 * randn(T, K)).to(y_dtype),
         "g_post": 1 + 0.2 * randn(K) if post and gains else None, "g_pre": 1 + 0.2 * randn(K) if gains else None,
         "gate": {"none": lambda: None, "scalar": lambda: 0.5 + 0.1 * randn(1), "channel": lambda: 0.5 + 0.1 * randn(K),
                  "token": lambda: torch.rand(T, 1, generator=gen),
                  "element": lambda: torch.sigmoid(randn(T, K)).to(y_dtype)}[gate]()}
    return {k: None if v is None else v.to(dev) for k, v in s.items()}
