"""Argument handling of the module wrapper that needs no GPU."""

import pytest
import torch

from swiglu_activation_amd.autograd import MegatronSwiGLU


def test_unsupported_options_raise():
    m = MegatronSwiGLU()
    x = torch.zeros(4, 8)
    with pytest.raises(NotImplementedError):
        m(x, None, True)
    with pytest.raises(NotImplementedError):
        m(x, None, False, True)


def test_shape_validation():
    m = MegatronSwiGLU(in_place=True)
    assert "in_place=True" in repr(m)
    with pytest.raises(ValueError):
        m(torch.zeros(8))              # 1D
    with pytest.raises(ValueError):
        m(torch.zeros(2, 2, 2, 8))     # 4D
    with pytest.raises(ValueError):
        m(torch.zeros(4, 7))           # odd last dim
    with pytest.raises(ValueError):
        m(torch.zeros(4, 8))           # host tensor: device pointers only


def test_expert_mlps_refuse_forward_mode_tangents(monkeypatch):
    """On stand-ins for the kernels: a dual input, weight or router weight raises, as
    the op itself does, whether gradients are recorded or not; without one the
    inference path is taken."""
    from torch.autograd import forward_ad

    from swiglu_activation_amd import autograd as ag
    calls = []

    def product(a, w, ends):
        calls.append("mm")
        return a @ w[0].t()

    def fc1(a, w, ends, scale=None):
        calls.append("fc1")
        return (a @ w[0].t())[:, :w.shape[1] // 2]

    monkeypatch.setattr(ag, "swiglu_grouped_mm", product)
    monkeypatch.setattr(ag, "swiglu_grouped_fc1", fc1)
    monkeypatch.setattr(ag, "swiglu_ckpt8_fwd", lambda x, s: (x[:, :x.shape[1] // 2], x, x))
    mlp = ag.GroupedSwiGLUMLP(1, 8, 16).requires_grad_(False)
    a, s, ends = torch.ones(4, 8, dtype=torch.bfloat16), torch.ones(4), torch.tensor([4], dtype=torch.int32)

    def plain():
        calls.clear()
        out = mlp(a, ends, s)
        assert calls == ["fc1", "mm"] and forward_ad.unpack_dual(out).tangent is None

    plain()
    with forward_ad.dual_level():
        plain()
        dual_a, dual_s = forward_ad.make_dual(a, a), forward_ad.make_dual(s, s)
        with pytest.raises(NotImplementedError):
            ag.grouped_mm(dual_a, mlp.w1, ends)
        for args in ((dual_a, ends, s), (dual_a, ends), (a, ends, dual_s)):
            with pytest.raises(NotImplementedError):
                mlp(*args)
            with torch.no_grad(), pytest.raises(NotImplementedError):
                mlp(*args)
        w1 = mlp.w1.data
        del mlp.w1
        mlp.w1 = forward_ad.make_dual(w1, w1)
        with pytest.raises(NotImplementedError):
            mlp(a, ends, s)
