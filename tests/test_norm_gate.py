"""gla_norm_gate and its gradients against fp64. A row's sum of up to 1024 squares in fp32 (ten levels of adding), a root, a
sigmoid and a few products: below 30 roundings of 2^-24 of terms up to ten times the result's root mean square. The weight's
gradient sums rows in fp32: 1e-5 of its norm."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def make(B, H, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    gate = rnd(B, T, 2 * H * d).to(dtype)[:, :, H * d:].unflatten(2, (H, d)).transpose(1, 2)
    return rnd(B, H, T, d).to(dtype), gate, 1 + 0.2 * rnd(d), rnd(B, T, H, d).to(dtype)


CASES = [
    # B, H, T, d, norm, activation, gate first, gate, weight
    (1, 1, 1, 16, "rms", "silu", False, True, True),
    (2, 4, 7, 128, "rms", "silu", False, True, True),
    (2, 4, 33, 128, "rms", "silu", True, True, True),
    (1, 3, 130, 64, "l2", "sigmoid", False, True, True),
    (3, 2, 5, 512, "rms", "silu", True, True, False),
    (1, 2, 40, 272, None, "silu", False, True, True),
    (1, 2, 11, 1024, "rms", "sigmoid", True, True, True),
    (1, 1, 300, 784, "rms", "silu", False, True, True),
    (2, 3, 9, 128, "rms", "silu", False, False, True),
    (1, 1, 3, 48, None, "sigmoid", True, True, False),
    (2, 5, 700, 16, "rms", "silu", True, True, True),
    (1, 7, 333, 32, "l2", "silu", False, True, True),
    (1, 3, 2000, 512, "rms", "sigmoid", False, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,T,d,norm,act,first,gated,weight", CASES)
def test_forward_and_backward(B, H, T, d, norm, act, first, gated, weight, dtype):
    x, g, w, dy = make(B, H, T, d, dtype, 7 * T + d)
    g, w = g if gated else None, w if weight else None
    cx, cg, cw, cdy = ref.cuda((x, g, w, dy))
    kw = dict(norm=norm, eps=1e-6, activation=act, gate_first=first)
    y = gla.norm_gate_forward(cx, cg, cw, **kw)
    assert y.is_contiguous() and y.shape == (B, T, H, d)
    X, Gd, Wd = ref.double((x, g, w))
    want = ref.gate(X, Gd, Wd, norm, 1e-6, act, first)
    ref.near(y, want, "y")
    leaves = [t for t in (X, Gd, Wd) if t is not None]
    wg = dict(zip([n for n, t in zip("xgw", (X, Gd, Wd)) if t is not None], torch.autograd.grad((want * dy.double()).sum(), leaves)))
    got = gla.norm_gate_backward(cx, cg, cw, cdy, **kw)
    ref.near(got[0], wg["x"], "dx")
    if gated:
        ref.near(got[1], wg["g"], "dgate")
        assert got[1].stride() == cg.stride() or T == 1 or H == 1 or got[1].transpose(1, 2).is_contiguous()
    if weight:
        e = (got[2].double().cpu() - wg["w"]).norm() / wg["w"].norm()
        assert e <= 1e-5, f"dw: {e:.1e}"
        assert torch.equal(got[2], gla.norm_gate_backward(cx, cg, cw, cdy, **kw)[2])


@pytest.mark.gpu
@pytest.mark.parametrize("first", [False, True])
def test_closed_gates_and_zero_rows(first):
    """Gates at the infinities' sides and rows of zeros: finite values and gradients, with and without eps where the row
    is not zero."""
    x, g, w, dy = ref.cuda(make(1, 2, 20, 128, torch.float32, 5))
    g = g.contiguous()
    g[0, 0, 3] = -200.0
    g[0, 1, 4] = 200.0
    x[0, 0, 5] = 0
    y = gla.norm_gate(x, g, w, gate_first=first)
    got = gla.norm_gate_backward(x, g, w, dy, gate_first=first)
    assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in got)
    assert not y[0, 5, 0].any() and not y[0, 3, 0].any()
    y = gla.norm_gate(x[:, :, 6:], g[:, :, 6:], w, eps=0.0, gate_first=first)
    got = gla.norm_gate_backward(x[:, :, 6:], g[:, :, 6:], w, dy[:, 6:].contiguous(), eps=0.0, gate_first=first)
    assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in got)


@pytest.mark.gpu
def test_empty_sequence_and_broadcast_gate():
    x, g, w, dy = ref.cuda(make(2, 3, 6, 64, torch.bfloat16, 9))
    assert gla.norm_gate(x[:, :, :0], g[:, :, :0], w).shape == (2, 0, 3, 64)
    got = gla.norm_gate_backward(x[:, :, :0], g[:, :, :0], w, dy[:, :0].contiguous())
    assert not got[2].any()
    e = g[:1, :, :1].expand(2, 3, 6, 64)
    assert torch.equal(gla.norm_gate(x, e, w), gla.norm_gate(x, e.contiguous(), w))
    e = e.detach().requires_grad_(True)
    y = gla.norm_gate(x, e, w)
    full = torch.autograd.grad(y, e, dy)[0]
    assert full.shape == e.shape


@pytest.mark.gpu
@pytest.mark.parametrize("first,act", [(False, "silu"), (True, "silu"), (True, "sigmoid")])
def test_gradients_against_differences(first, act):
    x, g, w, dy = ref.cuda(make(1, 2, 5, 64, torch.float32, 8))
    kw = dict(activation=act, gate_first=first)
    loss = lambda *a: float((gla.norm_gate_forward(*a, **kw).double() * dy.double()).sum())  # noqa: E731
    ref.along(loss, (x, g.contiguous(), w), gla.norm_gate_backward(x, g.contiguous(), w, dy, **kw))


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(x=1 << 20, gate=2 << 20, x_stride=(512, 256, 128), gate_stride=(512, 128, 256), w=3 << 20, B=1, H=2, T=2, d=128,
             norm=gla.GLA_NORM_RMS, activation=gla.GLA_ACT_SILU, eps=1e-6, dtype=gla.GLA_BF16)
    a.update(kw)
    p = bnd.gla_norm_gate_params()
    for n, v in a.items():
        setattr(p, n, type(getattr(p, n))(*v) if isinstance(v, tuple) else v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(T=-1), 1), (dict(d=24), 1), (dict(d=1040), 2), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(norm=3), 1), (dict(activation=0), 1), (dict(dtype=2), 1), (dict(x=0), 1),
    (dict(x=(1 << 20) + 8), 1), (dict(gate=(2 << 20) + 8), 1), (dict(gate_stride=(512, 128, 252)), 1), (dict(w=(3 << 20) + 2), 1),
])
def test_refuses_before_launch(kw, want):
    p = _params(**kw)
    assert bnd.load().gla_norm_gate(p, 4 << 20, None) == want
    assert bnd.load().gla_norm_gate_bwd_workspace_size(p) == 0


def test_refuses_outputs():
    lib, p = bnd.load(), _params()
    assert lib.gla_norm_gate(None, 4 << 20, None) == 1
    assert lib.gla_norm_gate(p, None, None) == 1
    assert lib.gla_norm_gate(p, (2 << 20) + 16, None) == 1                 # y over the gate
    st = (512, 256, 128)
    for g in (bnd.gla_norm_gate_grads(4 << 20, 5 << 20, 5 << 20, st, st, 6 << 20),       # two gradients in one place
              bnd.gla_norm_gate_grads(4 << 20, 5 << 20, 7 << 20, (512, 64, 128), st, 6 << 20),   # rows share storage
              bnd.gla_norm_gate_grads(4 << 20, 5 << 20, None, st, st, 6 << 20)):         # no place for the gate's
        assert lib.gla_norm_gate_bwd(p, g, None, 0, None) == 1
    assert lib.gla_norm_gate_bwd(p, None, None, 0, None) == 1


def test_python_checks():
    x = torch.randn(1, 2, 3, 64)
    for a in ((x[0],), (x, x[:, :, :2]), (x, x.bfloat16()), (x, None, torch.ones(32)), (x.double(),), (x.transpose(2, 3),),
              (x, x, None, "max"), (x, x, None, "rms", 1e-6, "relu")):
        with pytest.raises(gla.GlaError):
            gla.norm_gate(*a)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.norm_gate(x, x)
