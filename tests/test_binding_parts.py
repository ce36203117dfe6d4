"""The library without the binding's C++ part: what needs only the library goes on working, the calls
marshalled in C++ say what is missing."""
import pytest
import torch

import bit_ternary_qat_b200 as pkg
from bit_ternary_qat_b200 import build, ops


@pytest.fixture
def no_marshal(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(ops, "_marshal_module", None)
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))


def test_library_alone(no_marshal):
    assert pkg.load().bl_abi_version() >= 1
    assert pkg.workspace_bytes(1, 16, 32) > 0
    x = torch.ones(2, 32)
    for call in (lambda: pkg.bitlinear_grad_norm([x]), lambda: pkg.bitlinear_residual_norm(x, x),
                 lambda: pkg.bitlinear_linear_int8(x, x, x, x), lambda: pkg.bitlinear_quant_weight_int8(x)):
        with pytest.raises(ImportError, match="_marshal.so is not built"):
            call()


def test_library_is_built_first(no_marshal, monkeypatch):
    def missing(*a):
        raise RuntimeError("no headers")
    order = []
    monkeypatch.setattr(build, "build_marshal", missing)
    monkeypatch.setattr(build, "build_lib", lambda *a: order.append("library"))
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert order == ["library"]


def test_another_torch(monkeypatch):
    """A C++ part built for another torch is neither loaded nor taken as built."""
    build.build()
    assert build.marshal_fits() and ops._marshal().built_for.encode() == build._torch_mark()
    monkeypatch.setattr(ops, "_marshal_module", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0")
        assert not build.marshal_fits()
        with pytest.raises(ImportError, match="another torch"):
            pkg.bitlinear_grad_norm([torch.ones(2)])
        asked = []
        m.setattr(build.subprocess, "run", lambda cmd, check: asked.append(cmd))
        m.setattr(build.os, "replace", lambda a, b: None)
        build.build_marshal()
        assert len(asked) == 1 and '-DBL_TORCH_MARK="%s"' % build._torch_mark().decode() in asked[0]
    assert ops._marshal().built_for.encode() == build._torch_mark()
