"""One `out` dictionary through calls that write different parts of it: what a call returns it has
written, and what it has not written it does not return."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


def same(got, want, out):
    assert set(got) == set(want)
    for k, v in want.items():
        assert torch.equal(got[k], v), k
        assert k not in out or got[k] is out[k], k


@pytest.mark.parametrize("T", [3, 900])             # the kernel for few rows, and the ring
def test_residual_norm(bl, T):
    gen = torch.Generator().manual_seed(T)
    x, y = (torch.randn(T, 2048, generator=gen).to(B).to(DEV) for _ in range(2))
    out = bl.bitlinear_residual_norm(x, y)
    out["h"] = torch.full((T, 2048), 9.0, dtype=B, device=DEV)
    out["other"] = 5
    for kw in (dict(mode="norm"), dict(mode="none"), dict(mode="none", post_norm=False), dict(mode="quant"),
               dict(mode="norm", post_norm=False, alpha=0.5)):
        for t in out.values():
            if isinstance(t, torch.Tensor):
                t.fill_(3)
        want = bl.bitlinear_residual_norm(x, y, **kw)
        same(bl.bitlinear_residual_norm(x, y, out=out, **kw), want, out)
    # an xdq that the caller gives is an output, as in bitlinear_act_quant
    want = bl.bitlinear_residual_norm(x, y)
    out["xdq"].fill_(3)
    same(bl.bitlinear_residual_norm(x, y, want_xdq=False, out=out), want, out)
    assert "xdq" not in bl.bitlinear_residual_norm(x, y, want_xdq=False, out={"xdq": None})


def test_backward(bl):
    T, K = 20, 96
    gen = torch.Generator().manual_seed(1)
    x, y, dx, dh = (torch.randn(T, K, generator=gen).to(DEV) for _ in range(4))
    gate = torch.rand(K, generator=gen).to(DEV)
    r = torch.ones(T, device=DEV)

    def call(out=None, **kw):
        a = dict(dx=dx, dh=dh, x=x, y=y, r_post=r, r_pre=r, gate=gate, out=out)
        return bl.bitlinear_residual_norm_backward(**dict(a, **kw))
    out = call()
    assert {"dpost_gain", "dpre_gain", "dgate"} < set(out)
    for kw in (dict(dh=None, r_pre=None), dict(gate=None), dict(r_post=None), {}):
        for t in out.values():
            t.fill_(3)
        same(call(out=out, **kw), call(**kw), out)
    for t in out.values():
        t.fill_(3)
    same(call(out=out, want_dgains=False, want_dgate=False), call(), out)
    assert set(call(want_dgains=False, want_dgate=False)) == {"dx", "dy"}
