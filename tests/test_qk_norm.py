"""gla_qk_norm_rope and its gradients against fp64.

Tolerances: bf16 results are rounded once, at most 2^-8 relative of each value's own size; the
pair of a rotation adds fp32 errors of both, so 2^-8 of |y| plus 2^-20 of the row's norm. fp32: a
row's sum of 256 squares, a square root, a division, a product, the angle to 2^-24 turns and a
rotation: below 16 roundings of 2^-24 relative to the row's norm, 1e-6. Weight gradients sum rows in
fp32: 1e-5 of their norm."""
import math
from fractions import Fraction

import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _delta_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def rows_close(got, want, dtype, what):
    got, want = got.detach().double().cpu(), want.detach().double()
    assert torch.isfinite(got).all(), what
    row = want.norm(dim=-1, keepdim=True)
    tol = want.abs() * 2.0 ** -8 + row * 2.0 ** -20 if dtype == torch.bfloat16 else row * 1e-6
    worst = ((got - want).abs() / (tol + 1e-30)).max()
    assert worst <= 1, f"{what}: {worst:.2f} of its bound"


def case(B, H, Hk, T, d, rot, dtype, seed, positions, weights):
    g = torch.Generator().manual_seed(seed)
    proj = torch.randn((B, T, (H + 2 * Hk) * d), generator=g).to(dtype)
    q = proj[..., :H * d].unflatten(2, (H, d)).transpose(1, 2)
    k = proj[..., H * d:(H + Hk) * d].unflatten(2, (Hk, d)).transpose(1, 2)
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)] if weights else [None, None]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else None
    pos = torch.randint(-5, 2 ** 31 - 1, (B, T), generator=g) if positions else None
    return proj, q, k, w, f, pos, g


CASES = [
    # B, H, Hk, T, d, rot, norm, interleaved, weights, positions
    (1, 1, 1, 1, 128, 128, "l2", False, False, False),
    (2, 4, 2, 7, 128, 64, "rms", False, True, True),
    (2, 4, 2, 33, 64, 64, "rms", True, True, True),
    (1, 3, 1, 130, 256, 32, "l2", True, False, False),
    (1, 5, 5, 9, 48, 16, "rms", False, True, False),
    (3, 2, 1, 5, 208, 208, None, False, False, True),
    (1, 2, 2, 300, 16, 16, None, True, True, False),
    (1, 2, 1, 40, 128, 0, "l2", False, True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,Hk,T,d,rot,norm,inter,weights,positions", CASES)
def test_forward_and_backward(B, H, Hk, T, d, rot, norm, inter, weights, positions, dtype):
    proj, q, k, w, f, pos, g = case(B, H, Hk, T, d, rot, dtype, T, positions, weights)
    at = pos if positions else 11 + torch.arange(T).expand(B, T)
    gp = proj.cuda()
    gq = gp[..., :H * d].unflatten(2, (H, d)).transpose(1, 2)
    gk = gp[..., H * d:(H + Hk) * d].unflatten(2, (Hk, d)).transpose(1, 2)
    assert not gq.is_contiguous() or T == 1 or H == 1
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(norm=norm, w_q=cu(w[0]), w_k=cu(w[1]), eps=1e-6, inv_freq=cu(f), positions=cu(pos), start=11,
              interleaved=inter)
    oq, ok = gla.qk_norm_rope_forward(gq, gk, **kw)
    xs = [t.double().requires_grad_(True) for t in (q, k)]
    ws = [None if t is None else t.double().requires_grad_(True) for t in w]
    want = [ref.norm_rope(x, norm, ww, 1e-6, f, at, inter) for x, ww in zip(xs, ws)]
    for a, b, n in ((oq, want[0], "q"), (ok, want[1], "k")):
        assert a.is_contiguous() and a.dtype == dtype
        rows_close(a, b, dtype, n)
    dq, dk = torch.randn(oq.shape, generator=g).to(dtype), torch.randn(ok.shape, generator=g).to(dtype)
    leaves = xs + [x for x in ws if x is not None]
    ref_g = torch.autograd.grad((want[0] * dq.double()).sum() + (want[1] * dk.double()).sum(), leaves)
    got = gla.qk_norm_rope_backward(gq, gk, dq.cuda(), dk.cuda(), **kw)
    rows_close(got[0], ref_g[0], dtype, "dq")
    rows_close(got[1], ref_g[1], dtype, "dk")
    if weights:
        for a, b, n in ((got[2], ref_g[2], "dw_q"), (got[3], ref_g[3], "dw_k")):
            e = (a.double().cpu() - b).norm() / b.norm()
            assert e <= 1e-5, f"{n}: {e:.1e}"
        again = gla.qk_norm_rope_backward(gq, gk, dq.cuda(), dk.cuda(), **kw)
        assert torch.equal(again[2], got[2]) and torch.equal(again[3], got[3])


@pytest.mark.gpu
def test_far_positions_keep_their_angle():
    """Positions to 2^40 against the same frequencies rounded to 2^-60 turns, in exact integers."""
    import math
    from fractions import Fraction
    d = 32
    f = torch.tensor([1.0, 0.3, 0.01, 1e-4] * 4, dtype=torch.float64)
    pos = torch.tensor([[0, 1, 12345, 2 ** 20 + 1, 2 ** 31 + 7, 2 ** 40 + 3]])
    x = torch.zeros(1, 1, 6, d)
    x[..., :16] = 1                      # pairs (1, 0): the result is (cos, sin)
    y = gla.qk_norm_rope_forward(x.cuda(), None, norm=None, inv_freq=f.cuda(), positions=pos.cuda())[0].cpu()
    for t, p in enumerate(pos[0].tolist()):
        for i in range(16):
            # the turns per position as the kernel defines them: f / (2 pi) in fp64
            turn = Fraction(float(f[i]) * 0.15915494309189533577) * p
            th = float(turn - math.floor(turn)) * 2 * math.pi
            assert abs(float(y[0, 0, t, i]) - math.cos(th)) < 1e-6 and abs(float(y[0, 0, t, i + 16]) - math.sin(th)) < 1e-6


# 2 pi to 60 digits
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_true_angles_of_far_positions(interleaved):
    """Positions on both sides of zero against pos * f reduced by 2 pi in exact fractions. f / (2 pi) is rounded twice in
    fp64 (the constant and the product, 2^-53 each) and once to units of 2^-64 turns (half of one, 2^-62.3 radians): the
    angle is off by |pos| times that. The rest is fp32: the turn's upper 32 bits rounded to 24 (2^-25 of half a turn,
    9.4e-8) and the two functions' 2 ulp (1.2e-7)."""
    d = 32
    f = torch.tensor([1.0, 0.3, 0.01, 1e-4, 7e-9, 2.5, 0.7390851332151607, 1e-2 / 3] * 2, dtype=torch.float64)
    pos = torch.tensor([[0, 1, -1, 12345, 2 ** 20 + 1, -(2 ** 31) - 7, 2 ** 40 + 3, -(2 ** 40) - 3, 2 ** 46 + 1]])
    n = pos.shape[1]
    x = torch.zeros(1, 1, n, d)
    x[..., 0::2 if interleaved else 1] = 1
    if not interleaved:
        x[..., d // 2:] = 0              # pairs (1, 0): the result is (cos, sin)
    y = gla.qk_norm_rope_forward(x.cuda(), None, norm=None, inv_freq=f.cuda(), positions=pos.cuda(),
                                 interleaved=interleaved)[0].cpu()[0, 0].double()
    c, s = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :d // 2], y[:, d // 2:])
    for t, p in enumerate(pos[0].tolist()):
        for i in range(d // 2):
            tol = 4e-7 + abs(p * float(f[i])) * 2.0 ** -52 + abs(p) * 2.0 ** -62
            turn = p * Fraction(float(f[i])) / TWO_PI
            th = float(turn - math.floor(turn)) * 2 * math.pi
            assert abs(float(c[t, i]) - math.cos(th)) <= tol and abs(float(s[t, i]) - math.sin(th)) <= tol, (p, float(f[i]))


@pytest.mark.gpu
def test_one_tensor_alone_dense_and_broadcast():
    x = torch.randn(1, 1, 6, 64, device="cuda")
    a = gla.qk_norm_rope_forward(x, None)[0]
    assert torch.allclose(a, x / x.norm(dim=-1, keepdim=True), atol=1e-6)
    e = x.expand(3, 4, 6, 64)
    b = gla.qk_norm_rope_forward(e, None)[0]
    assert b.shape == e.shape and all(torch.equal(b[i, j], a[0, 0]) for i in range(3) for j in range(4))
    z = gla.qk_norm_rope_forward(torch.zeros(1, 1, 2, 64, device="cuda"), None)[0]
    assert not z.any()                  # a zero row stays zero: eps


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 1), (1, 5), (3, 40)])
def test_gradients_of_one_tensor_alone(B, T, weights):
    """Without k: q's gradient as beside one, bit for bit, and the weight's to its sums' order."""
    proj, q, k, w, f, pos, g = case(B, 3, 2, T, 64, 32, torch.bfloat16, 3 * B + T, False, True)
    q, k, dq, dk = (t.bfloat16().cuda() for t in (q, k, torch.randn(q.shape, generator=g), torch.randn(k.shape, generator=g)))
    wq = w[0].cuda() if weights else None
    leaves = [t.requires_grad_(True) for t in ([q, wq] if weights else [q])]
    y, none = gla.qk_norm_rope(q, None, w_q=wq, inv_freq=f.cuda())
    assert none is None
    got = torch.autograd.grad(y, leaves, dq)
    want = gla.qk_norm_rope_backward(q.detach(), k, dq, dk, w_q=None if wq is None else wq.detach(), inv_freq=f.cuda())
    assert torch.equal(got[0], want[0])
    if weights:
        assert torch.allclose(got[1], want[2], rtol=0, atol=1e-5 * float(want[2].norm()))


@pytest.mark.gpu
def test_autograd_through_both_operators():
    """A layer's run: projection -> norms and rotation -> gated delta rule -> loss, against fp64."""
    B, H, Hk, T, d = 1, 4, 2, 100, 64
    proj, q, k, w, f, pos, g = case(B, H, Hk, T, d, d, torch.bfloat16, 21, False, True)
    v = torch.randn((B, H, T, d), generator=g).bfloat16()
    be, lg = torch.sigmoid(torch.randn((B, H, T), generator=g)).bfloat16(), -torch.rand((B, H, T), generator=g) / 8
    dO = torch.randn((B, H, T, d), generator=g).bfloat16()
    P = proj.cuda().requires_grad_(True)
    W = [t.cuda().requires_grad_(True) for t in w]
    V, Be, Lg = (t.cuda().requires_grad_(True) for t in (v, be, lg))
    cut = lambda t, a, n: t[..., a * d:(a + n) * d].unflatten(2, (n, d)).transpose(1, 2)  # noqa: E731
    qq, kk = gla.qk_norm_rope(cut(P, 0, H)[:, ::2], cut(P, H, Hk), norm="l2", w_q=W[0], w_k=W[1], inv_freq=f.cuda())
    O, ST = gla.delta_attention(qq, kk, V, Lg, Be)
    O.backward(dO.cuda())
    R = [t.double().requires_grad_(True) for t in (proj, *w, v, be, lg)]
    at = torch.arange(T).expand(B, T)
    rq = ref.norm_rope(cut(R[0], 0, H)[:, ::2], "l2", R[1], 1e-6, f, at, False)
    rk = ref.norm_rope(cut(R[0], H, Hk), "l2", R[2], 1e-6, f, at, False)
    o, _ = ref.delta(rq, rk, R[3], R[5], R[4], None, d ** -0.5)
    (o * dO.double()).sum().backward()
    # q and k are rounded to bf16 on the way (2^-8) and their gradients again: a few such steps
    for a, b, n in ((O, o, "O"), (P.grad, R[0].grad, "dproj"), (W[0].grad, R[1].grad, "dw_q"), (W[1].grad, R[2].grad, "dw_k"),
                    (V.grad, R[3].grad, "dv"), (Be.grad, R[4].grad, "dbeta"), (Lg.grad, R[5].grad, "dlog_g")):
        e = (a.detach().double().cpu() - b.detach()).norm() / b.norm()
        assert e <= 4 * 2.0 ** -8, f"{n}: {e:.1e}"


@pytest.mark.gpu
def test_replays_from_a_cuda_graph_with_new_positions():
    proj, q, k, w, f, pos, g = case(4, 4, 2, 1, 128, 128, torch.bfloat16, 5, True, True)
    gq, gk, gw, gf, gpos = q.cuda(), k.cuda(), [t.cuda() for t in w], f.cuda(), pos.cuda()
    run = lambda: gla.qk_norm_rope_forward(gq, gk, norm="rms", w_q=gw[0], w_k=gw[1], inv_freq=gf, positions=gpos)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    gpos.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, run()):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("d,T", [(64, 7), (128, 17), (256, 3)])
def test_gradients_without_eps(d, T, norm, dtype):
    """eps = 0 and tokens that do not fill the last block: its idle rows hold zeros, of which no inverse norm exists."""
    proj, q, k, w, f, pos, g = case(1, 3, 1, T, d, 32, dtype, d + T, False, True)
    kw = dict(norm=norm, w_q=w[0].cuda(), w_k=w[1].cuda(), eps=0.0, inv_freq=f.cuda())
    oq, ok = gla.qk_norm_rope_forward(q.cuda(), k.cuda(), **kw)
    xs = [t.double().requires_grad_(True) for t in (q, k, *w)]
    at = torch.arange(T).expand(1, T)
    want = [ref.norm_rope(xs[i], norm, xs[2 + i], 0.0, f, at, False) for i in (0, 1)]
    rows_close(oq, want[0], dtype, "q")
    rows_close(ok, want[1], dtype, "k")
    dq, dk = torch.randn(oq.shape, generator=g).to(dtype), torch.randn(ok.shape, generator=g).to(dtype)
    ref_g = torch.autograd.grad((want[0] * dq.double()).sum() + (want[1] * dk.double()).sum(), xs)
    got = gla.qk_norm_rope_backward(q.cuda(), k.cuda(), dq.cuda(), dk.cuda(), **kw)
    rows_close(got[0], ref_g[0], dtype, "dq")
    rows_close(got[1], ref_g[1], dtype, "dk")
    for a, b, n in ((got[2], ref_g[2], "dw_q"), (got[3], ref_g[3], "dw_k")):
        assert torch.isfinite(a).all(), n
        e = (a.double().cpu() - b).norm() / b.norm()
        assert e <= 1e-5, f"{n}: {e:.1e}"


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(q=1 << 16, k=2 << 16, q_stride=(512, 128, 256), k_stride=(512, 128, 256), B=1, H=2, Hk=2, T=2, d=128, rot=0,
             norm=gla.GLA_NORM_L2, eps=1e-6, dtype=gla.GLA_BF16)
    a.update(kw)
    p = bnd.gla_qk_norm_params()
    for n, v in a.items():
        setattr(p, n, type(getattr(p, n))(*v) if isinstance(v, tuple) else v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hk=-1), 1), (dict(d=24), 1), (dict(d=272), 2), (dict(rot=24, inv_freq=1 << 8), 1),
    (dict(rot=144, inv_freq=1 << 8), 1), (dict(rot=64), 1), (dict(inv_freq=1 << 8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(norm=3), 1), (dict(dtype=2), 1), (dict(q=0), 1), (dict(k=0), 1),
    (dict(q=(1 << 16) + 8), 1), (dict(q_stride=(512, 128, 252)), 1), (dict(w_q=(1 << 14) + 4), 1),
    (dict(positions=(1 << 14) + 4), 1),
])
def test_refuses_before_launch(kw, want):
    p = _params(**kw)
    assert bnd.load().gla_qk_norm_rope(p, 3 << 16, 4 << 16, None) == want


def test_refuses_outputs():
    lib = bnd.load()
    p = _params()
    assert lib.gla_qk_norm_rope(None, 3 << 16, 4 << 16, None) == 1
    assert lib.gla_qk_norm_rope(p, None, 4 << 16, None) == 1
    assert lib.gla_qk_norm_rope(p, 1 << 16, 4 << 16, None) == 1          # over q
    assert lib.gla_qk_norm_rope(p, 3 << 16, (3 << 16) + 16, None) == 1   # over each other
    g = bnd.gla_qk_norm_grads(3 << 16, 4 << 16, 5 << 16, 6 << 16, (512, 128, 256), (512, 128, 64), None, None)
    assert lib.gla_qk_norm_rope_bwd(p, g, None, 0, None) == 1            # rows of grad_k share storage
    g = bnd.gla_qk_norm_grads(3 << 16, 4 << 16, 5 << 16, 6 << 16, (512, 128, 256), (512, 128, 256), 7 << 16, None)
    assert lib.gla_qk_norm_rope_bwd(p, g, None, 0, None) == 1            # a weight's gradient without the weight
    assert lib.gla_qk_norm_rope_bwd(p, None, None, 0, None) == 1


def test_python_checks():
    x = torch.randn(1, 2, 3, 64)
    for q, k, kw in ((x[0], x, {}), (x, x[:, :, :2], {}), (x, x.bfloat16(), {}), (x.transpose(2, 3), None, {}),
                     (x, x, dict(norm="max")), (x, x, dict(w_q=torch.ones(32))), (x.double(), None, {}),
                     (x, x, dict(inv_freq=torch.ones(32))), (x, x, dict(positions=torch.zeros(1, 3)))):
        with pytest.raises(gla.GlaError):
            gla.qk_norm_rope_forward(q, k, **kw)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.qk_norm_rope_forward(x, x)
