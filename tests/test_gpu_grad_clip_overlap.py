"""Clips whose outputs would overlap a gradient or one another are refused before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, B = torch.float32, torch.bfloat16


@pytest.fixture
def flat():
    return torch.arange(1000, dtype=F, device=DEV) / 100


def refused(call, *a, **kw):
    with pytest.raises(ValueError, match="overlap"):
        call(*a, **kw)


def test_out_is_another_gradient(bl, flat):
    g = [flat[:100], flat[100:200]]
    refused(bl.bitlinear_clip_grads, g, 1.0, out=[g[1], g[0]])


def test_parts_overlap(bl, flat):
    other = torch.zeros(1000, device=DEV)
    clip = bl.bitlinear_clip_grads
    refused(clip, [flat[:100], flat[99:200]], 1.0)                           # both in place, one element shared
    refused(clip, [flat[:100]], 1.0, out=[flat[1:101]])                      # its own output, shifted
    refused(clip, [flat[:100], flat[100:200]], 1.0, out=[other[:100], other[50:150]])
    refused(clip, [flat[:100], flat[100:200]], 1.0, out=[other[:100], flat[20:120]])
    refused(clip, [flat[:100], flat[:100]], 1.0, out=[flat[:100], other[:100]])   # read while it is written
    refused(clip, [flat[:100], flat.view(B)[100:300]], 1.0)                  # another type over the same bytes
    refused(clip, [flat[:500], flat[100:101]], 1.0)                          # within


def test_norm_coef_and_workspace(bl, flat):
    for call in (bl.bitlinear_clip_grads, bl.bitlinear_grad_norm):
        refused(call, [flat[:100]], 1.0, norm=flat[4:5])
        refused(call, [flat[:100]], 1.0, coef=flat[99:100])
        refused(call, [flat[:100]], 1.0, norm=flat[500:501], coef=flat[500:501])
        big = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
        refused(call, [big.view(F)[8:20]], 1.0, ws=big)


def test_neighbours_are_taken(bl, flat):
    """Views that touch, the same gradient twice into separate outputs, and empty ones among them."""
    src, other = flat.clone(), torch.zeros(1000, device=DEV)
    o = bl.bitlinear_clip_grads([flat[:100], flat[100:350], flat[100:100]], 1.0, norm=flat[350:351], coef=flat[351:352])
    assert torch.equal(flat[:350], src[:350] * o["coef"]) and torch.equal(flat[352:], src[352:])
    assert o["norm"].data_ptr() == flat[350:351].data_ptr()
    o = bl.bitlinear_clip_grads([src[:100], src[:100], src[50:90]], 1.0, out=[other[:100], other[100:200], other[200:240]])
    for lo, hi, at in ((0, 100, 0), (0, 100, 100), (50, 90, 200)):
        assert torch.equal(other[at:at + hi - lo], src[lo:hi] * o["coef"])
    bl.bitlinear_grad_norm([src[:100], src[50:100]], 1.0, norm=src[500:501])
    # a buffer that is more than the workspace, with the results and a gradient behind that
    n = bl.workspace_bytes(1, 1, 1)
    buf = torch.zeros(n + 4096, dtype=torch.uint8, device=DEV)
    tail = buf[n:].view(F)
    tail[:100] = src[:100]
    o = bl.bitlinear_clip_grads([tail[:100]], 1.0, norm=tail[200:201], coef=tail[201:202], ws=buf)
    assert torch.equal(tail[:100], src[:100] * o["coef"])
    torch.cuda.synchronize()
    assert bl.check_device_status() == 0
