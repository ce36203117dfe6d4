"""Workloads of the operators around a BitLinear block: the residual norms with their gradient,
the global gradient norm with clipping and the step behind it, and the 8-bit linear.

Each case names an operator and its sizes.  ``run`` is one pass: with ``own`` false the
operator's formulas in elementary torch operations (fp32, fp64 for the sums of squares whose
rounding decides 8-bit codes), with ``own`` true the framework's call.  ``exact`` restates the
definitions in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token between two blocks of a 4096-wide model: latency
        {"name": "norm_1x4096", "op": "norm", "T": 1, "K": 4096, "x": "bf16", "y": "bf16", "post": True,
         "gate": "none", "out": "quant", "alpha": 1.0, "beta": 1.0},
        # a training step's tokens, residual stream kept in fp32 around bf16 blocks
        {"name": "norm_16384x4096", "op": "norm", "T": 16384, "K": 4096, "x": "f32", "y": "bf16", "post": True,
         "gate": "channel", "out": "quant", "alpha": 1.0, "beta": 1.0},
        # an odd width and a gate for each token (a router's weight), plain norm output
        {"name": "norm_1021x1003", "op": "norm", "T": 1021, "K": 1003, "x": "f32", "y": "f32", "post": True,
         "gate": "token", "out": "norm", "alpha": 1.0, "beta": 0.7},
        # the gradients of the training step, every gain and the channel gate learned
        {"name": "norm_bwd_16384x4096", "op": "norm_bwd", "T": 16384, "K": 4096, "x": "bf16", "y": "bf16",
         "post": True, "gate": "channel", "out": "norm", "alpha": 1.0, "beta": 1.0},
        # a wide hidden activation gated element by element, a ragged batch of tokens
        {"name": "norm_bwd_777x11008", "op": "norm_bwd", "T": 777, "K": 11008, "x": "bf16", "y": "bf16",
         "post": True, "gate": "element", "out": "norm", "alpha": 0.8, "beta": 0.6},
        # all weight gradients of a 7B-shaped layer (q, k, v, o, gate, up, down), clipped
        {"name": "clip_layer", "op": "clip", "set": "layer", "count": 7, "total": 202375168, "types": "f32"},
        # gains, gates and small matrices of many layers, both types
        {"name": "clip_58_ragged", "op": "clip", "set": "ragged", "count": 58, "total": 1500007, "types": "mixed"},
        # global clip and optimizer step of an MLP's two matrices
        {"name": "step_2x11008x4096", "op": "step", "count": 2, "N": 11008, "K": 4096},
        # one decoded token through a large 8-bit matrix
        {"name": "int8_1x28672x8192", "op": "int8", "T": 1, "N": 28672, "K": 8192, "y": "bf16", "train": False},
        # a decode batch of odd size through a down projection
        {"name": "int8_37x4096x11008", "op": "int8", "T": 37, "N": 4096, "K": 11008, "y": "f32", "train": False},
        # a prompt through an up projection
        {"name": "int8_8192x11008x4096", "op": "int8", "T": 8192, "N": 11008, "K": 4096, "y": "bf16",
         "train": False},
        # a training forward: the latent weight quantised, then the product
        {"name": "int8_train_4096x2048x2048", "op": "int8", "T": 4096, "N": 2048, "K": 2048, "y": "bf16",
         "train": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "clip", "step", "int8", "int8"])
    if op in ("norm", "norm_bwd"):
        x, y = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
        out = rng.choice(["quant", "norm", "none"] if y == "bf16" and op == "norm" else ["norm", "norm", "none"])
        K = _log(rng, 8, 16384)
        if out == "quant":
            K = max(32, K // 32 * 32)
        elif rng.random() < 0.5:
            K = max(8, K // 8 * 8)
        T = _log(rng, 1, min(16384, 16384 * 4096 // K))
        return {"op": op, "T": T, "K": K, "x": x, "y": y, "post": rng.random() < 0.75,
                "gate": rng.choice(["none", "scalar", "channel", "token", "element"]), "out": out,
                "alpha": rng.choice([1.0, round(rng.uniform(0.5, 1.5), 3)]),
                "beta": rng.choice([1.0, round(rng.uniform(0.1, 1.0), 3)])}
    if op == "clip":
        count = _log(rng, 1, 58)
        return {"op": op, "set": "ragged", "count": count, "total": _log(rng, 4 * count, 1 << 27),
                "types": rng.choice(["f32", "bf16", "mixed"])}
    if op == "step":
        count = rng.randint(1, 4)
        K = max(32, _log(rng, 32, 11008) // 32 * 32)
        N = max(16, _log(rng, 16, min(11008, 90177536 // (K * count))) // 16 * 16)
        return {"op": op, "count": count, "N": N, "K": K}
    train = rng.random() < 0.25
    K = max(32, _log(rng, 32, 16384) // 32 * 32)
    N = max(16, _log(rng, 16, min(28672, (45088768 if train else 234881024) // K)) // 16 * 16)
    T = _log(rng, 1, min(8192, 8192 * 11008 * 4096 // (N * K)))
    return {"op": op, "T": T, "N": N, "K": K, "y": "bf16" if train else rng.choice(["f32", "bf16"]),
            "train": train}


def _sizes(case):
    """Element counts of a clip case's gradients."""
    if case["set"] == "layer":
        return [4096 * 4096] * 4 + [11008 * 4096] * 3
    r = random.Random(case["count"] * 1000003 + case["total"])
    w = [math.exp(r.uniform(0.0, 6.0)) for _ in range(case["count"])]
    return [max(1, int(case["total"] * v / sum(w))) for v in w]


def _types(case, i):
    if case["types"] == "mixed":
        return "bf16" if i % 3 == 1 else "f32"
    return case["types"]


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _randn(gen, shape, std, dtype="f32"):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(DTYPES[dtype])


def _inputs(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op in ("norm", "norm_bwd"):
        T, K = case["T"], case["K"]
        # a residual stream with a few channels of large values, a block's output of another scale
        s["x"] = (_randn(gen, (T, K), 1.0) * torch.exp(_randn(gen, (K,), 0.5))).to(DTYPES[case["x"]])
        s["y"] = _randn(gen, (T, K), 0.3, case["y"])
        s["g_post"] = 1.0 + _randn(gen, (K,), 0.2) if case["post"] else None
        s["g_pre"] = 1.0 + _randn(gen, (K,), 0.2) if case["out"] != "none" else None
        s["gate"] = {"none": lambda: None, "scalar": lambda: 0.5 + _randn(gen, (1,), 0.1),
                     "channel": lambda: 0.5 + _randn(gen, (K,), 0.1),
                     "token": lambda: torch.rand((T, 1), generator=gen, device=DEV),
                     "element": lambda: torch.sigmoid(_randn(gen, (T, K), 1.0)).to(DTYPES[case["y"]])}[case["gate"]]()
        if op == "norm_bwd":
            # what the forward saved: the new residual (here x stands for it) and both statistics
            s["r_post"] = _rinv(s["y"]) if case["post"] else None
            s["r_pre"] = _rinv(s["x"]) if case["out"] != "none" else None
            s["dx"] = _randn(gen, (T, K), 1e-2)
            s["dh"] = _randn(gen, (T, K), 1e-2) if case["out"] != "none" else None
    elif op == "clip":
        sizes = _sizes(case)
        std = torch.exp(_randn(gen, (len(sizes),), 1.0)).tolist()
        s["grads"] = [_randn(gen, (n,), 1e-2 * std[i], _types(case, i)) for i, n in enumerate(sizes)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        s["max_norm"] = 1.0
    elif op == "step":
        shape, n = (case["N"], case["K"]), case["count"]
        s["W"] = [_randn(gen, shape, 0.02) for _ in range(n)]
        s["dW"] = [_randn(gen, shape, 1e-2) for _ in range(n)]
        s["m"] = [_randn(gen, shape, 1e-3) for _ in range(n)]
        s["v"] = [_randn(gen, shape, 1e-3).square() for _ in range(n)]
        s["step"] = [torch.full((1,), 10, dtype=torch.int32, device=DEV) for _ in range(n)]
        s["max_norm"] = 1.0
    else:
        T, N, K = case["T"], case["N"], case["K"]
        # activations as the token quantiser leaves them; weights as the channel quantiser does
        s["xq"], s["sx"] = _codes(_randn(gen, (T, K), 1.0))
        W = _randn(gen, (N, K), 0.02) * torch.exp(_randn(gen, (N, 1), 0.3))
        if case["train"]:
            s["W"] = W
        else:
            s["wq"], scale = _codes(W)
            s["gamma"] = 1.0 / scale
    return s


def _rinv(v):
    return torch.rsqrt(v.double().square().mean(-1) + EPS).float()


def _codes(v):
    scale = 127.0 / v.abs().amax(-1).clamp_min(1e-5)
    return torch.round(v * scale[:, None]).to(torch.int8), scale


def prepare(case, seed):
    return _inputs(case, seed)


# ------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------
def _times(v, by):
    return v if by is None else v * by


def _plain_norm(s):
    c = s["case"]
    n = s["y"].float()
    if c["post"]:
        # fp64: the statistic's last bit can move a code across a border
        r_post = (1.0 / torch.sqrt(s["y"].double().square().mean(-1) + EPS)).float()
        n = n * r_post[:, None] * s["g_post"]
    n = _times(n, s["gate"] if s["gate"] is None else s["gate"].float()) * c["beta"]
    x = (s["x"].float() * c["alpha"] + n).to(s["x"].dtype)
    got = {"x": x}
    if c["post"]:
        got["r_post"] = r_post
    if c["out"] != "none":
        r_pre = (1.0 / torch.sqrt(x.double().square().mean(-1) + EPS)).float()
        h = x.float() * r_pre[:, None] * s["g_pre"]
        got["r_pre"] = r_pre
        if c["out"] == "norm":
            got["h"] = h.to(s["y"].dtype)
        else:
            sx = 127.0 / h.abs().amax(-1).clamp_min(1e-5)
            q = torch.round(h * sx[:, None]).clamp(-128, 127)
            got["sx"] = sx
            got["xdq"] = (q / sx[:, None]).to(s["y"].dtype)   # the codes' values
    return got


def _plain_norm_bwd(s):
    c = s["case"]
    d, got = s["dx"], {}
    if c["out"] != "none":
        u = s["x"].float() * s["r_pre"][:, None]
        e = s["dh"] * s["g_pre"]
        d = d + s["r_pre"][:, None] * (e - u * (e * u).mean(-1, keepdim=True))
        got["dpre_gain"] = (s["dh"] * u).sum(0)
    got["dx"] = d * c["alpha"]
    d = d * c["beta"]
    y = s["y"].float()
    u = y * s["r_post"][:, None] if c["post"] else y
    n = _times(u, s["g_post"])
    if c["gate"] != "none":
        p = d * n
        got["dgate"] = {"scalar": lambda: p.sum(dtype=torch.float64).float().reshape(1),
                        "channel": lambda: p.sum(0), "token": lambda: p.sum(1, keepdim=True), "element": lambda: p.to(s["y"].dtype)}[c["gate"]]()
        d = d * s["gate"].float()
    if c["post"]:
        got["dpost_gain"] = (d * u).sum(0)
        e = d * s["g_post"]
        d = s["r_post"][:, None] * (e - u * (e * u).mean(-1, keepdim=True))
    got["dy"] = d.to(s["y"].dtype)
    return got


def _plain_coef(grads, max_norm):
    norm = torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()
    return norm.float().reshape(1), (max_norm / (norm + 1e-6)).clamp(max=1.0).float().reshape(1)


def _plain_clip(s):
    norm, coef = _plain_coef(s["grads"], s["max_norm"])
    return {"norm": norm, "coef": coef, "grads": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}


LR, B1, B2, DECAY = 1e-3, 0.9, 0.95, 0.01


def _plain_adamw(W, dW, m, v, step, coef):
    g = dW * coef
    step += 1
    t = step.double()
    m.copy_(m * B1 + g * (1.0 - B1))
    v.copy_(v * B2 + g * g * (1.0 - B2))
    size = (LR / (1.0 - B1 ** t)).float()
    root = torch.sqrt(1.0 - B2 ** t).float()
    W.copy_((W * (1.0 - LR * DECAY) - size * m / (v.sqrt() / root + EPS)).clamp(-1.0, 1.0))


def _plain_step(s):
    norm, coef = _plain_coef(s["dW"], s["max_norm"])
    [_plain_adamw(*a, coef) for a in zip(s["W"], s["dW"], s["m"], s["v"], s["step"])]
    return {"norm": norm, "coef": coef, "W": s["W"], "m": s["m"], "v": s["v"]}


def _plain_int8(s):
    c, got = s["case"], {}
    if c["train"]:
        peak = s["W"].abs().amax(-1).clamp_min(1e-5)
        wq, gamma = torch.round(s["W"] * (127.0 / peak)[:, None]), peak / 127.0
        got = {"gamma_rows": gamma, "w": (wq * gamma.to(torch.bfloat16).float()[:, None]).to(torch.bfloat16)}
    else:
        wq, gamma = s["wq"].float(), s["gamma"]
    # sums of whole numbers below 2^24: fp32 holds them
    acc = s["xq"].float() @ wq.t()
    got["y"] = (acc * (gamma[None, :] / s["sx"][:, None])).to(DTYPES[c["y"]])
    return got


# ------------------------------------------------------------------------------------
# the framework's calls
# ------------------------------------------------------------------------------------
def _own(s):
    import bit_ternary_qat_b200 as bl
    c = s["case"]
    if c["op"] == "norm":
        o = bl.bitlinear_residual_norm(s["x"], s["y"], post_norm=c["post"], g_post=s["g_post"], gate=s["gate"],
                                       alpha=c["alpha"], beta=c["beta"], mode=c["out"], g_pre=s["g_pre"])
        return {k: o[k] for k in ("x", "r_post", "r_pre", "h", "sx", "xdq") if k in o}
    if c["op"] == "norm_bwd":
        o = bl.bitlinear_residual_norm_backward(s["dx"], s["dh"], s["x"], s["y"], r_post=s["r_post"],
                                                r_pre=s["r_pre"], g_post=s["g_post"], gate=s["gate"],
                                                alpha=c["alpha"], beta=c["beta"], g_pre=s["g_pre"])
        return {k: o[k] for k in ("dx", "dy", "dpre_gain", "dpost_gain", "dgate") if k in o}
    if c["op"] == "clip":
        return bl.bitlinear_clip_grads(s["grads"], s["max_norm"], out=s["out"])
    if c["op"] == "step":
        o = bl.bitlinear_grad_norm(s["dW"], s["max_norm"])
        [bl.bitlinear_optimizer_step(*a, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=DECAY, coef=o["coef"])
         for a in zip(s["W"], s["dW"], s["m"], s["v"], s["step"])]
        return {"norm": o["norm"], "coef": o["coef"], "W": s["W"], "m": s["m"], "v": s["v"]}
    if c["train"]:
        q = bl.bitlinear_quant_weight_int8(s["W"])
        y, _ = bl.bitlinear_linear_int8(s["xq"], s["sx"], q["wq_i8"], q["gamma_rows"], out_dtype=DTYPES[c["y"]])
        return {"gamma_rows": q["gamma_rows"], "w": q["wq_bf16"], "y": y}
    y, _ = bl.bitlinear_linear_int8(s["xq"], s["sx"], s["wq"], s["gamma"], out_dtype=DTYPES[c["y"]])
    return {"y": y}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "clip": _plain_clip, "step": _plain_step,
            "int8": _plain_int8}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        T, K, x, y = case["T"], case["K"], size[case["x"]], size[case["y"]]
        gate = {"none": 0, "scalar": 4, "channel": 4 * K, "token": 4 * T, "element": y * T * K}[case["gate"]]
        small = (4 * K + 4 * T) * ((1 if case["post"] else 0) + (1 if case["out"] != "none" else 0))
        if op == "norm":
            # x and y in; the new residual out, and the norm (or codes, scales and the codes' values)
            per = 2 * x + y + {"none": 0, "norm": y, "quant": 1 + y}[case["out"]]
            return {"bytes": per * T * K + gate + small + (4 * T if case["out"] == "quant" else 0),
                    "flops": 12 * T * K}
        # dx, dh, the new residual and y in; dx and dy out, and the gains' and gate's gradients
        per = 4 + y + 4 + y + (4 + x if case["out"] != "none" else 0)
        return {"bytes": per * T * K + 2 * gate + 2 * small, "flops": 24 * T * K}
    if op == "clip":
        b = sum(n * size[_types(case, i)] for i, n in enumerate(_sizes(case)))
        return {"bytes": 2 * b, "flops": 3 * sum(_sizes(case))}
    if op == "step":
        n = case["count"] * case["N"] * case["K"]
        return {"bytes": 28 * n, "flops": 17 * n}
    T, N, K = case["T"], case["N"], case["K"]
    w = (4 + 1 + 2) * N * K if case["train"] else N * K
    return {"bytes": w + T * K + 4 * T + 4 * N + size[case["y"]] * T * N, "flops": 2 * T * N * K}


# ------------------------------------------------------------------------------------
# the definitions in fp64
# ------------------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "clip": _exact_clip, "step": _exact_step,
            "int8": _exact_int8}[case["op"]](case, s)


def _f64(t):
    return None if t is None else t.to(torch.float64)


def _exact_norm(c, s):
    x, y, g1, g2, gate = (_f64(s[k]) for k in ("x", "y", "g_post", "g_pre", "gate"))
    K, got = c["K"], {}
    z = y
    if c["post"]:
        got["r_post"] = ((y * y).sum(1) / K + EPS) ** -0.5
        z = torch.einsum("tk,t,k->tk", y, got["r_post"], g1)
    if gate is not None:
        z = gate * z
    got["x"] = torch.add(c["alpha"] * x, z, alpha=c["beta"])
    # the next norm reads the residual as it is held
    held = _f64(got["x"].to(s["x"].dtype))
    if c["out"] != "none":
        got["r_pre"] = ((held * held).sum(1) / K + EPS) ** -0.5
        h = torch.einsum("tk,t,k->tk", held, got["r_pre"], g2)
        if c["out"] == "norm":
            got["h"] = h
        else:
            got["sx"] = 127.0 / torch.clamp(h.abs().max(1).values, min=1e-5)
            got["xdq"] = torch.round(h * got["sx"].unsqueeze(1)) / got["sx"].unsqueeze(1)
    return got


def _exact_norm_bwd(c, s):
    d, dh, x, y, r1, r2, g1, g2, gate = (_f64(s[k]) for k in
                                         ("dx", "dh", "x", "y", "r_post", "r_pre", "g_post", "g_pre", "gate"))
    K, got = c["K"], {}
    if dh is not None:
        # h = g2 x r2 with r2 = (mean x^2 + eps)^(-1/2): dr2/dx = -r2^3 x / K
        inner = torch.einsum("tk,tk,k->t", dh, x, g2)
        d = d + torch.einsum("tk,t,k->tk", dh, r2, g2) - x * (r2 ** 3 * inner / K).unsqueeze(1)
        got["dpre_gain"] = torch.einsum("tk,tk,t->k", dh, x, r2)
    got["dx"] = c["alpha"] * d
    n = y if r1 is None else torch.einsum("tk,t,k->tk", y, r1, g1)
    if gate is not None:
        full = c["beta"] * d * n
        got["dgate"] = {"scalar": lambda: full.sum().view(1), "channel": lambda: full.sum(0),
                        "token": lambda: full.sum(1).unsqueeze(1), "element": lambda: full}[c["gate"]]()
    dn = c["beta"] * d if gate is None else c["beta"] * d * gate
    if r1 is None:
        got["dy"] = dn
    else:
        inner = torch.einsum("tk,tk,k->t", dn, y, g1)
        got["dpost_gain"] = torch.einsum("tk,tk,t->k", dn, y, r1)
        got["dy"] = torch.einsum("tk,t,k->tk", dn, r1, g1) - y * (r1 ** 3 * inner / K).unsqueeze(1)
    return got


def _exact_coef(grads, max_norm):
    total = 0.0
    for g in grads:
        total += float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2
    norm = math.sqrt(total)
    return norm, min(1.0, max_norm / (norm + 1e-6))


def _exact_clip(c, s):
    norm, coef = _exact_coef(s["grads"], s["max_norm"])
    one = torch.ones(1, dtype=torch.float64)
    return {"norm": norm * one, "coef": coef * one, "grads": [_f64(g) * coef for g in s["grads"]]}


def _exact_step(c, s):
    norm, coef = _exact_coef(s["dW"], s["max_norm"])
    one, t = torch.ones(1, dtype=torch.float64), 11
    got = {"norm": norm * one, "coef": coef * one, "W": [], "m": [], "v": []}
    for W, dW, m, v in zip(s["W"], s["dW"], s["m"], s["v"]):
        g = coef * _f64(dW)
        m1 = B1 * _f64(m) + (1 - B1) * g
        v1 = B2 * _f64(v) + (1 - B2) * g ** 2
        new = _f64(W) * (1 - LR * DECAY) - LR * (m1 / (1 - B1 ** t)) / ((v1 / (1 - B2 ** t)) ** 0.5 + EPS)
        got["W"].append(new.clamp(-1, 1))
        got["m"].append(m1)
        got["v"].append(v1)
    return got


def _exact_int8(c, s):
    got = {}
    if c["train"]:
        top = torch.clamp(_f64(s["W"]).abs().max(1).values, min=1e-5)
        wq, gamma = torch.round(_f64(s["W"]) * 127.0 / top.unsqueeze(1)), top / 127.0
        got = {"gamma_rows": gamma, "w": wq * gamma.unsqueeze(1)}
    else:
        wq, gamma = _f64(s["wq"]), _f64(s["gamma"])
    y = torch.matmul(_f64(s["xq"]), wq.T)
    got["y"] = y * gamma / _f64(s["sx"]).unsqueeze(1)
    return got
