"""The `out` of the calls that are marshalled in C++: a dict, another mapping of names, or a TypeError."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def calls(bl):
    x, y = torch.ones(4, 32, device=DEV), torch.full((4, 32), 2.0, device=DEV)
    W = torch.randn(16, 32, device=DEV)
    step, coef = torch.zeros(1, dtype=torch.int32, device=DEV), torch.ones(1, device=DEV)
    return {"norm": (("x", torch.empty_like(x)), lambda out: bl.bitlinear_residual_norm(x, y, mode="norm", out=out)),
            "backward": (("dy", torch.empty_like(y)),
                         lambda out: bl.bitlinear_residual_norm_backward(x, None, x, y, out=out)),
            "weight": (("gamma_rows", torch.empty(16, device=DEV)),
                       lambda out: bl.bitlinear_quant_weight_int8(W, out=out)),
            "step": (("gamma", torch.empty(1, device=DEV)),
                     lambda out: bl.bitlinear_optimizer_step(W.clone(), W, W.clone(), W * W, step.clone(),
                                                             requantize=True, out=out, coef=coef))}


@pytest.mark.parametrize("name", ["norm", "backward", "weight", "step"])
def test_out(bl, name):
    (key, buf), call = calls(bl)[name]
    want = call(None)[key]
    for out in ({key: buf}, types.MappingProxyType({key: buf})):
        buf.fill_(7.0)
        got = call(out)
        assert got[key] is buf and torch.equal(buf, want) and got is not out
    for bad in (buf, 3, "x", [buf], object()):
        with pytest.raises(TypeError, match="out must be a dict"):
            call(bad)
    torch.cuda.synchronize()
