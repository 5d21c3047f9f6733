"""gla_conv_fwd and gla_conv_bwd against fp64. Sums of at most four products and a bias, a sigmoid of five roundings: below 30
roundings of 2^-24 of terms up to ten times the result's root mean square. Weight gradients are sums over all tokens in
fp32: 1e-5 of their norm."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def flat(t, heads):
    return t.transpose(1, 2).flatten(2) if heads else t


def make(B, H, T, d, W, dtype, seed, bias=True, s0=True):
    """x as a projection's slice, token-major (heads split off for H > 1)."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    D = H * d
    proj = rnd(B, T, D + 32).to(dtype)
    x = proj[:, :, 16:16 + D]
    x = x.unflatten(2, (H, d)).transpose(1, 2) if H > 1 else x
    return (x, rnd(D, W), rnd(D) if bias else None, rnd(B, W - 1, D).to(dtype) if s0 else None,
            rnd(*x.shape).to(dtype), rnd(B, W - 1, D).to(dtype))


CASES = [
    # B, H, T, d, W, act, bias, S0
    (1, 1, 1, 16, 4, "silu", True, True),
    (2, 1, 2, 48, 4, "silu", True, True),
    (3, 1, 3, 272, 4, "silu", False, True),
    (2, 1, 7, 1040, 3, None, True, False),
    (2, 3, 65, 64, 4, "silu", True, True),
    (1, 2, 130, 128, 2, "silu", False, False),
    (2, 1, 1031, 128, 4, "silu", True, True),
    (1, 5, 33, 16, 2, None, False, True),
    (2, 1, 2500, 2048, 4, "silu", True, True),       # long runs
    (3, 1, 1300, 2048, 3, None, True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,T,d,W,act,bias,s0", CASES)
def test_forward_and_backward(B, H, T, d, W, act, bias, s0, dtype):
    x, w, b, S0, dy, dST = make(B, H, T, d, W, dtype, 10 * T + W, bias, s0)
    heads = H > 1
    gx, gw, gb, gS, gdy, gdST = ref.cuda((x, w, b, S0, dy, dST))
    if heads:                                      # (cuda() of a transposed view keeps its strides)
        assert T == 1 or not gx.is_contiguous()
    y, ST = gla.causal_conv_forward(gx, gw, gb, gS, act)
    assert y.is_contiguous() and y.shape == gx.shape
    X, Wd, Bd, S0d = ref.double((x, w, b, S0))
    want, last = ref.conv(flat(X, heads), Wd, Bd, S0d, act)
    ref.near(flat(y, heads), want, "y")
    assert torch.equal(ST.double().cpu(), last.detach())
    leaves = [t for t in (X, Wd, Bd, S0d) if t is not None]
    wg = torch.autograd.grad((want * flat(dy.double(), heads)).sum() + (last * dST.double()).sum(), leaves)
    wg = dict(zip([n for n, t in zip(("x", "w", "bias", "S0"), (X, Wd, Bd, S0d)) if t is not None], wg))
    got = gla.causal_conv_backward(gx, gw, gb, gS, gdy, gdST, act)
    ref.near(got[0], wg["x"], "dx")
    for n, a in (("w", got[1]), ("bias", got[2])):
        if n in wg:
            e = (a.double().cpu() - wg[n]).norm() / wg[n].norm()
            assert e <= 1e-5, f"d{n}: {e:.1e}"
    if s0:
        ref.near(got[3], wg["S0"], "dS0")
    again = gla.causal_conv_backward(gx, gw, gb, gS, gdy, gdST, act)
    assert all(a is None or torch.equal(a, c) for a, c in zip(got, again))


@pytest.mark.gpu
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("cuts", [(1, 1, 1, 1, 1), (2, 5, 1, 40), (3, 0, 4)])
def test_pieces_with_the_state_carried_in_place(W, cuts):
    """A sequence in pieces gives what it gives in one call, bit for bit: the same sums in the same order."""
    T = sum(cuts)
    x, w, b, S0, _, _ = make(2, 1, T, 64, W, torch.bfloat16, T)
    x, w, b, S0 = ref.cuda((x, w, b, S0))
    y, ST = gla.causal_conv(x, w, b, S0)
    state, at, out = S0.clone(), 0, []
    for n in cuts:
        p, s = gla.causal_conv_forward(x[:, at:at + n], w, b, state, ST=state)
        assert s is state
        out.append(p)
        at += n
    assert torch.equal(torch.cat(out, 1), y) and torch.equal(state, ST)


@pytest.mark.gpu
def test_in_place_over_many_blocks():
    """The state carried in place while several blocks of the sequence run."""
    x, w, b, S0, _, _ = make(2, 1, 5000, 128, 4, torch.bfloat16, 1)
    x, w, b, S0 = ref.cuda((x, w, b, S0))
    y, ST = gla.causal_conv(x, w, b, S0)
    for _ in range(3):
        s = S0.clone()
        y2, _ = gla.causal_conv_forward(x, w, b, s, ST=s)
        assert torch.equal(y2, y) and torch.equal(s, ST)


@pytest.mark.gpu
def test_padding_in_front():
    """Rows of zeros in front of a prompt leave what a zero state leaves."""
    x, w, _, _, _, _ = make(1, 1, 20, 64, 4, torch.float32, 2)
    x, w = x.cuda(), w.cuda()
    a, sa = gla.causal_conv(x, w)
    b, sb = gla.causal_conv(torch.cat((torch.zeros(1, 9, 64, device="cuda"), x), 1), w)
    assert torch.equal(b[:, 9:], a) and torch.equal(sa, sb)


@pytest.mark.gpu
def test_empty_sequence_and_broadcast():
    x, w, b, S0, _, dST = ref.cuda(make(2, 1, 4, 64, 4, torch.bfloat16, 3))
    y, ST = gla.causal_conv(x[:, :0], w, b, S0)
    assert y.shape == (2, 0, 64) and torch.equal(ST, S0)
    _, ST = gla.causal_conv(x[:, :0], w, b)
    assert not ST.any()
    got = gla.causal_conv_backward(x[:, :0], w, b, S0, y, dST)
    assert torch.equal(got[3], dST) and not got[1].any() and not got[2].any()
    e = x[:1].expand(3, 4, 64)
    y, _ = gla.causal_conv(e, w, b)
    one, _ = gla.causal_conv(x[:1], w, b)
    assert torch.equal(y, one.expand(3, 4, 64))


@pytest.mark.gpu
def test_not_finite_values_stay_in_their_channel_and_window():
    x, w, b, S0, _, _ = ref.cuda(make(1, 1, 300, 64, 4, torch.bfloat16, 4))
    y, _ = gla.causal_conv(x, w, b, S0)
    v = x.contiguous()
    v[0, 100, 5], v[0, 200, 9] = float("nan"), float("inf")
    z, _ = gla.causal_conv(v, w, b, S0)
    same = torch.ones_like(y, dtype=torch.bool)
    same[0, 100:104, 5] = False
    same[0, 200:204, 9] = False
    assert torch.equal(z[same], y[same]) and torch.isnan(z[0, 100:104, 5]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [1, 2])
def test_gradients_against_differences(H):
    x, w, b, S0, dy, dST = ref.cuda(make(2, H, 9, 32, 4, torch.float32, 6))
    x = x.contiguous()

    def loss(*a):
        y, ST = gla.causal_conv_forward(*a)
        return float((y.double() * dy.double()).sum() + (ST.double() * dST.double()).sum())
    ref.along(loss, (x, w, b, S0), gla.causal_conv_backward(x, w, b, S0, dy, dST))


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(x=1 << 20, x_stride=(512, 128, 256), w=2 << 20, bias=3 << 20, S0=4 << 20, B=1, H=2, T=2, d=128, W=4,
             activation=gla.GLA_ACT_SILU, dtype=gla.GLA_BF16)
    a.update(kw)
    p = bnd.gla_conv_params()
    for n, v in a.items():
        setattr(p, n, type(getattr(p, n))(*v) if isinstance(v, tuple) else v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(T=-1), 1), (dict(d=24), 1), (dict(W=0), 1), (dict(W=1), 2), (dict(W=5), 2),
    (dict(activation=2), 1), (dict(dtype=2), 1), (dict(x=0), 1), (dict(w=0), 1), (dict(x=(1 << 20) + 2), 1),
    (dict(x_stride=(512, 128, 252)), 1), (dict(w=(2 << 20) + 4), 1), (dict(S0=(4 << 20) + 2), 1),
    (dict(T=1 << 30, B=1 << 20), 2), (dict(H=1 << 20, d=128), 2),
])
def test_refuses_before_launch(kw, want):
    p = _params(**kw)
    assert bnd.load().gla_conv_fwd(p, 5 << 20, 6 << 20, None) == want
    assert bnd.load().gla_conv_bwd_workspace_size(p) == 0


def test_refuses_outputs():
    lib, p = bnd.load(), _params()
    assert lib.gla_conv_fwd(None, 5 << 20, None, None) == 1
    assert lib.gla_conv_fwd(p, None, 6 << 20, None) == 1
    assert lib.gla_conv_fwd(p, 1 << 20, 6 << 20, None) == 1              # y over x
    assert lib.gla_conv_fwd(p, 5 << 20, (4 << 20) + 16, None) == 1       # ST over S0, elsewhere
    assert lib.gla_conv_fwd(p, 5 << 20, 5 << 20, None) == 1              # over each other
    g = bnd.gla_conv_grads(5 << 20, None, 7 << 20, (512, 128, 64), 8 << 20, 9 << 20, None)
    assert lib.gla_conv_bwd(p, g, None, 0, None) == 1                    # rows of grad_x share storage
    g = bnd.gla_conv_grads(5 << 20, None, 7 << 20, (512, 128, 256), 8 << 20, 9 << 20, None)
    assert lib.gla_conv_bwd(_params(bias=None), g, None, 0, None) == 1   # a bias's gradient without the bias
    assert lib.gla_conv_bwd(p, None, None, 0, None) == 1


def test_python_checks():
    x, w = torch.randn(1, 3, 64), torch.randn(64, 4)
    for a in ((x[0], w), (x, w[0]), (x, w[:32]), (x.double(), w), (x.transpose(1, 2), w), (x, w.bfloat16()),
              (x, w, torch.ones(32)), (x, w, None, torch.zeros(1, 4, 64)), (x, w, None, None, "relu")):
        with pytest.raises(gla.GlaError):
            gla.causal_conv(*a)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.causal_conv(x, w)
