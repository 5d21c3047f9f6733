"""gla_residual_norm and its gradients against fp64. Sums of up to 16384 squares in fp32 over threads and lanes (at most 32
products in a row, then eleven levels of adding), roots and a few products: below 30 roundings of 2^-24 of terms up to ten
times the result's root mean square. Vector gradients sum rows in fp32: 1e-5 of their norm."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref

BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


CASES = [
    # rows, D, types, post norm, scale, residual, weight
    (1, 16, (BF, BF), False, None, True, True),
    (5, 256, (BF, FP), True, "vector", True, True),
    (33, 512, (FP, FP), True, "vector", True, True),
    (7, 1024, (BF, BF), False, 0.25, True, True),
    (40, 2048, (BF, BF), True, "vector", True, True),
    (700, 2048, (BF, FP), False, "vector", True, True),
    (9, 2064, (BF, BF), False, "vector", False, True),
    (6, 4096, (FP, FP), False, None, True, False),
    (3, 8192, (BF, BF), True, "vector", True, True),
    (2, 16384, (BF, FP), True, "vector", True, True),
    (1300, 48, (BF, BF), True, 2.0, True, True),
    (325, 8208, (BF, BF), True, "vector", True, True),       # the widest kernel, several rows to a block
    (160, 16384, (FP, FP), False, "vector", True, True),
    (311, 11008, (BF, FP), True, 0.5, True, False),
    (200, 6160, (FP, FP), True, "vector", False, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,D,types,post,scale,has_r,weight", CASES)
def test_forward_and_backward(rows, D, types, post, scale, has_r, weight):
    g = torch.Generator().manual_seed(rows + D)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, r = rnd(rows, D).to(types[0]), (2 * rnd(rows, D)).to(types[1]) if has_r else None
    w = 1 + 0.2 * rnd(D) if weight else None
    sc = 0.5 + 0.2 * rnd(D) if scale == "vector" else scale
    rt = types[1] if has_r else types[0]
    dh, dy = rnd(rows, D).to(rt), rnd(rows, D).to(types[0])
    vec = isinstance(sc, torch.Tensor)
    cx, cr, cw, csc, cdh, cdy = ref.cuda((x, r, w, sc if vec else None, dh, dy))
    csc = csc if vec else sc
    h, y = gla.residual_norm_forward(cx, cr, cw, csc, post_norm=post)
    assert h.dtype == rt and y.dtype == types[0]
    X, R, Wd, Sd = ref.double((x, r, w, sc if vec else None))
    H, Y = ref.residual(X, R, Wd, Sd if vec else sc, post, 1e-6)
    ref.near(h, H, "h")
    ref.near(y, Y, "y")
    if has_r:
        into = cr.clone()
        h2, y2 = gla.residual_norm_forward(cx, into, cw, csc, post_norm=post, h=into)
        assert h2 is into and torch.equal(h2, h) and torch.equal(y2, y)
    names = [n for n, t in zip(("x", "r", "w", "scale"), (X, R, Wd, Sd)) if t is not None]
    leaves = [t for t in (X, R, Wd, Sd) if t is not None]
    wg = dict(zip(names, torch.autograd.grad((H * dh.double()).sum() + (Y * dy.double()).sum(), leaves)))
    got = gla.residual_norm_backward(cx, cr, cw, csc, cdh, cdy, post_norm=post)
    ref.near(got[0], wg["x"], "dx")
    if has_r:
        ref.near(got[1], wg["r"], "dr")
    for n, a in (("w", got[2]), ("scale", got[3])):
        assert (a is None) == (n not in wg)
        if n in wg:
            e = (a.double().cpu() - wg[n]).norm() / wg[n].norm()
            assert e <= 1e-5, f"d{n}: {e:.1e}"
    again = gla.residual_norm_backward(cx, cr, cw, csc, cdh, cdy, post_norm=post)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.gpu
def test_one_gradient_alone_and_a_shared_one():
    x, r, dh, dy = (torch.randn(12, 256, device="cuda") for _ in range(4))
    w = torch.rand(256, device="cuda") + 0.5
    for t in (x, r, w):
        t.requires_grad_(True)
    h, y = gla.residual_norm(x, r, w)
    a = torch.autograd.grad((h, y), (x, r, w), (dh, dy), retain_graph=True)
    assert torch.equal(a[0], a[1])
    zero = torch.zeros_like(dh)
    b = torch.autograd.grad(h, (x, r), dh, retain_graph=True)
    c = torch.autograd.grad((h, y), (x, r), (dh, zero), retain_graph=True)
    assert torch.equal(b[0], dh) and torch.allclose(c[0], b[0], atol=1e-6)
    d = torch.autograd.grad(y, (r, w), dy)
    e = gla.residual_norm_backward(x.detach(), r.detach(), w.detach(), None, zero, dy)
    assert torch.equal(d[0], e[1]) and torch.equal(d[1], e[2])
    # accumulated into two leaves, the shared gradient is not shared by them
    p, q = (t.detach().clone().requires_grad_(True) for t in (x, r))
    h, y = gla.residual_norm(p, q, w.detach())
    torch.autograd.backward((h, y), (dh, dy))
    p.grad.add_(1)
    assert torch.allclose(q.grad + 1, p.grad)


@pytest.mark.gpu
def test_no_rows():
    x, w = torch.empty(0, 256, device="cuda"), torch.ones(256, device="cuda")
    h, y = gla.residual_norm(x, x, w, w)
    assert h.shape == y.shape == (0, 256)
    got = gla.residual_norm_backward(x, x, w, w, h, y)
    assert not got[2].any() and not got[3].any()


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
def test_gradients_against_differences(post):
    g = torch.Generator().manual_seed(3)
    x, r, dh, dy = (torch.randn(6, 80, generator=g).cuda() for _ in range(4))
    w, sc = (1 + 0.2 * torch.randn(80, generator=g).cuda() for _ in range(2))

    def loss(x, r, w, sc):
        h, y = gla.residual_norm_forward(x, r, w, sc, post_norm=post)
        return float((h.double() * dh.double()).sum() + (y.double() * dy.double()).sum())
    ref.along(loss, (x, r, w, sc), gla.residual_norm_backward(x, r, w, sc, dh, dy, post_norm=post))


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(x=1 << 20, residual=2 << 20, w=3 << 20, scale=4 << 20, alpha=1.0, rows=4, D=256, eps=1e-6, dtype=gla.GLA_BF16,
             residual_dtype=gla.GLA_FP32)
    a.update(kw)
    p = bnd.gla_residual_params()
    for n, v in a.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(D=0), 1), (dict(D=24), 1), (dict(D=16400), 2), (dict(eps=-1.0), 1), (dict(alpha=float("inf")), 1),
    (dict(dtype=2), 1), (dict(dtype=1, residual_dtype=0), 1), (dict(x=0), 1), (dict(x=(1 << 20) + 8), 1),
    (dict(w=(3 << 20) + 4), 1), (dict(scale=(4 << 20) + 4), 1), (dict(rows=1 << 40), 2),
])
def test_refuses_before_launch(kw, want):
    p = _params(**kw)
    assert bnd.load().gla_residual_norm(p, 5 << 20, 6 << 20, None) == want
    assert bnd.load().gla_residual_norm_bwd_workspace_size(p) == 0


def test_refuses_outputs():
    lib, p = bnd.load(), _params()
    assert lib.gla_residual_norm(None, 5 << 20, 6 << 20, None) == 1
    assert lib.gla_residual_norm(p, 5 << 20, None, None) == 1
    assert lib.gla_residual_norm(p, (2 << 20) + 16, 6 << 20, None) == 1    # over the residual, elsewhere
    assert lib.gla_residual_norm(p, 5 << 20, 2 << 20, None) == 1           # y over the residual
    assert lib.gla_residual_norm(p, 5 << 20, (5 << 20) + 16, None) == 1    # over each other
    g = bnd.gla_residual_grads(None, 7 << 20, 8 << 20, 8 << 20, None, None)
    assert lib.gla_residual_norm_bwd(p, g, None, 0, None) == 1             # two gradients in one place
    g = bnd.gla_residual_grads(None, 7 << 20, 8 << 20, 9 << 20, 10 << 20, None)
    assert lib.gla_residual_norm_bwd(_params(w=None), g, None, 0, None) == 1
    assert lib.gla_residual_norm_bwd(p, None, None, 0, None) == 1


def test_python_checks():
    x, w = torch.randn(3, 64), torch.ones(64)
    for a in ((x, x[:2]), (x, x.bfloat16()), (x, x, w[:32]), (x.double(),), (x.t(),), (x, x, w, w.double())):
        with pytest.raises(gla.GlaError):
            gla.residual_norm(*a)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.residual_norm(x, x, w)
