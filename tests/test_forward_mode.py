"""Derivatives in forward mode are refused, never dropped: the autograd functions have none. The library's calls are
replaced by stand-ins of the same outputs, so no GPU is needed."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import autograd as glue


@pytest.fixture(autouse=True)
def _stand_ins(monkeypatch):
    monkeypatch.setattr(glue._b, "delta_forward", lambda q, k, v, log_g, beta, S0=None, **kw: (v * 2, torch.ones(1, 2, 16, 16)))
    monkeypatch.setattr(glue._b, "qk_norm_rope_forward", lambda q, k, *a: (q * 2, None if k is None else k * 2))


def _delta():
    x = torch.randn(1, 2, 3, 16)
    return [x, x + 1, x + 2, -torch.rand(1, 2, 3), torch.rand(1, 2, 3), torch.ones(1, 2, 16, 16)]


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("grad", [True, False])
def test_delta_attention_refuses_a_dual(at, grad):
    x = _delta()
    with fwd.dual_level(), torch.set_grad_enabled(grad):
        x[at] = fwd.make_dual(x[at], torch.ones_like(x[at]))
        with pytest.raises((RuntimeError, NotImplementedError), match="(?i)forward|jvp"):
            gla.delta_attention(*x)


@pytest.mark.parametrize("at", range(4))
def test_qk_norm_rope_refuses_a_dual(at):
    x = [torch.randn(1, 2, 3, 16), torch.randn(1, 2, 3, 16), torch.ones(16), torch.ones(16)]
    with fwd.dual_level():
        x[at] = fwd.make_dual(x[at], torch.ones_like(x[at]))
        with pytest.raises((RuntimeError, NotImplementedError), match="(?i)forward|jvp"):
            gla.qk_norm_rope(x[0], x[1], w_q=x[2], w_k=x[3])


def test_other_calls_pass():
    x = _delta()
    assert not gla.delta_attention(*x)[0].requires_grad
    assert not gla.qk_norm_rope(x[0])[0].requires_grad
    with fwd.dual_level():             # a level is open, these inputs have no tangents
        assert torch.equal(gla.delta_attention(*x)[0], x[2] * 2)
        assert torch.equal(gla.qk_norm_rope(x[0], x[1])[1], x[1] * 2)
    x[2].requires_grad_(True)
    assert gla.delta_attention(*x)[0].requires_grad
    with torch.no_grad():
        assert not gla.delta_attention(*x)[0].requires_grad
