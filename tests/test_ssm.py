"""gla_ssm_fwd and gla_ssm_bwd against fp64, token by token.

Tolerances: a decay is good to 2^-22 (the exponential) and |delta A| 2^-23 (its argument), of either sign, and a state remembers
tau = 1 / |delta A| tokens: sqrt(tau) 2^-22 + 2^-23, below 4e-6 of the states' size for the tau <= 200 of these inputs; sums of
up to 64 states and 1040 channels add below 30 roundings of 2^-24. So 2e-5 of each tensor's root mean square, values of heavy
tails (a channel's gradients among all) included, plus one rounding to bf16 where the type is bf16. Sums over tokens: 1e-5 of
their norm."""
import math

import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref

NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def make(B, T, D, N, G, dtype, seed, without=(), steep=False):
    """x dense, z and dt slices of wider rows, B and C slices of one projection's output; all on the GPU if there is one."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    x, xz, low = (t.to(dtype).to(dev) for t in (rnd(B, T, D), rnd(B, T, 2 * D + 16), rnd(B, T, 16 + 2 * G * N)))
    step = torch.exp(torch.rand(D, generator=g) * math.log(20) + math.log(5e-3))
    t = {"x": x, "dt": xz[:, :, :D], "A": -(1 + torch.arange(N) % 16) * torch.exp(0.1 * rnd(D, N)),
         "B": low[:, :, 16:16 + G * N].unflatten(2, (G, N)), "C": low[:, :, 16 + G * N:].unflatten(2, (G, N)),
         "D": 1 + 0.1 * rnd(D), "z": xz[:, :, D + 16:], "dt_bias": step + torch.log(-torch.expm1(-step)),
         "S0": rnd(B, D, N) * 0.3}
    if steep:
        t["A"] = t["A"] * 40
    t = {n: None if n in without else a.to(dev) for n, a in t.items()}
    return t, rnd(B, T, D).to(dtype).to(dev), (rnd(B, D, N) * 0.3).to(dev)


def check(t, dy, dST, softplus=True, **kw):
    args = [t[n] for n in NAMES]
    y, ST = gla.selective_scan_forward(*args, softplus=softplus, **kw)
    leaves = dict(zip(NAMES, ref.double(args)))
    want, last = ref.scan(*leaves.values(), softplus)
    ref.near(y, want, "y")
    ref.near(ST, last, "ST")
    given = [n for n in NAMES if leaves[n] is not None]
    loss = (want * dy.double().cpu()).sum() + (0 if dST is None else (last * dST.double().cpu()).sum())
    wg = dict(zip(given, torch.autograd.grad(loss, [leaves[n] for n in given], allow_unused=True)))
    got = dict(zip(NAMES, gla.selective_scan_backward(*args, dy, dST, softplus=softplus, **kw)))
    for n in NAMES:
        if n not in wg:
            assert got[n] is None or n == "S0", n
        elif n in ("A", "D", "dt_bias"):
            e = (got[n].double().cpu() - wg[n]).norm() / wg[n].norm()
            assert e <= 1e-5, f"d{n}: {e:.1e}"
        else:
            ref.near(got[n], wg[n], "d" + n)
    return y, ST, got


CASES = [
    # B, T, D, N, G, segments, left out
    (1, 1, 16, 16, 1, 0, ()),
    (3, 2, 48, 8, 1, 0, ("z",)),
    (2, 8, 144, 16, 3, 0, ("S0", "dt_bias")),
    (2, 9, 32, 64, 2, 0, ("D",)),
    (1, 16, 16, 32, 1, 1, ()),
    (2, 17, 272, 16, 1, 1, ()),
    (1, 33, 1040, 16, 1, 1, ("D", "z", "dt_bias", "S0")),
    (2, 50, 96, 8, 2, 2, ()),
    (1, 100, 80, 64, 1, 3, ("z",)),
    (1, 161, 64, 16, 4, 5, ("S0",)),
    (3, 130, 160, 32, 2, 9, ()),
    (1, 320, 48, 16, 1, 0, ()),
    (2, 35, 72, 64, 3, 2, ()),
    (1, 40, 8, 8, 1, 1, ()),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,D,N,G,segments,without", CASES)
def test_forward_and_backward(B, T, D, N, G, segments, without, dtype):
    t, dy, dST = make(B, T, D, N, G, dtype, 3 * T + D, without)
    _, _, got = check(t, dy, dST if T % 2 else None, force_segments=segments)
    again = gla.selective_scan_backward(*[t[n] for n in NAMES], dy, dST if T % 2 else None, force_segments=segments)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got.values(), again))


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [1, 4])
def test_steep_decays_keep_their_gradients(segments):
    """Decays down to exp(-60): the gradients of A and dt hold terms of every size."""
    t, dy, dST = make(1, 70, 32, 16, 1, torch.float32, 6, steep=True)
    check(t, dy, dST, force_segments=segments)


@pytest.mark.gpu
def test_steps_given_directly():
    t, dy, dST = make(2, 40, 64, 16, 1, torch.float32, 8, ("dt_bias",))
    t["dt"] = t["dt"].abs() * 0.05
    check(t, dy, dST, softplus=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_small_and_large_steps(dtype):
    """softplus over its whole range: steps from 1e-9 to 80."""
    t, dy, _ = make(1, 24, 16, 8, 1, dtype, 9, ("S0", "dt_bias"))
    t["dt"] = torch.linspace(-20, 80, 24 * 16, device="cuda").reshape(1, 24, 16).to(dtype)
    check(t, dy, None)


@pytest.mark.gpu
@pytest.mark.parametrize("T,pad", [(5, 2), (40, 16), (33, 70)])
def test_padded_tokens_leave_the_state(T, pad):
    """Tokens with dt = -inf in front, between and behind: the state passes them unchanged."""
    t, dy, dST = make(2, T, 32, 16, 1, torch.float32, T)
    y, ST = gla.selective_scan(**t)
    longer = {n: a for n, a in t.items()}
    for n in ("x", "dt", "B", "C", "z"):
        a = t[n]
        fill = torch.full((2, pad, *a.shape[2:]), -math.inf if n == "dt" else 0.5, dtype=a.dtype, device="cuda")
        longer[n] = torch.cat((fill, a, fill), 1)
    y2, ST2 = gla.selective_scan(**longer)
    assert torch.allclose(ST2, ST, rtol=0, atol=1e-5) and torch.allclose(y2[:, pad:pad + T], y, rtol=0, atol=1e-4)
    zero = torch.zeros(2, pad, 32, device="cuda")
    got = gla.selective_scan_backward(*[longer[n] for n in NAMES], torch.cat((zero, dy, zero), 1), dST)
    want = gla.selective_scan_backward(*[t[n] for n in NAMES], dy, dST)
    assert all(torch.isfinite(a).all() for a in got)
    for n, a, b in zip(NAMES, got, want):
        a = a[:, pad:pad + T] if n in ("x", "dt", "B", "C", "z") else a
        assert torch.allclose(a, b, rtol=0, atol=2e-5 * float(b.square().mean().sqrt()) * 10), n


@pytest.mark.gpu
def test_decoding_carries_the_state_in_place():
    t, _, _ = make(4, 30, 96, 16, 1, torch.bfloat16, 11)
    y, ST = gla.selective_scan(**t)
    state, out, at = t["S0"].clone(), [], 0
    for n in (1, 1, 7, 0, 20, 1):
        p = {k: (a[:, at:at + n] if k in ("x", "dt", "B", "C", "z") else a) for k, a in t.items()}
        o, s = gla.selective_scan_forward(**{**p, "S0": state}, ST=state)
        assert s is state
        out.append(o)
        at += n
    ref.near(torch.cat(out, 1), y.double().cpu(), "y", 2.0 ** -7)     # (each rounded once, from sums of other order)
    assert torch.allclose(state, ST, rtol=0, atol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [2, 3, 20])
def test_state_in_place_over_segments(segments):
    """The last segment's blocks write the state that the first's read, in one launch and in any order."""
    t, _, _ = make(8, 320, 4096, 16, 1, torch.bfloat16, 14)
    y, ST = gla.selective_scan_forward(**t, force_segments=segments)
    for _ in range(3):
        state = t["S0"].clone()
        y2, _ = gla.selective_scan_forward(**{**t, "S0": state}, ST=state, force_segments=segments)
        assert torch.equal(y2, y) and torch.equal(state, ST)


@pytest.mark.gpu
def test_empty_sequence_and_broadcast_rows():
    t, dy, dST = make(2, 4, 32, 16, 1, torch.float32, 12)
    none = {k: (a[:, :0] if k in ("x", "dt", "B", "C", "z") else a) for k, a in t.items()}
    y, ST = gla.selective_scan(**none)
    assert y.shape == (2, 0, 32) and torch.equal(ST, t["S0"])
    got = gla.selective_scan_backward(*[none[n] for n in NAMES], y, dST)
    assert torch.equal(got[8], dST) and not got[2].any() and not got[5].any() and not got[7].any()
    e = {**t, "B": t["B"][:1, :1].expand(2, 4, 1, 16), "z": t["z"][:, :1].expand(2, 4, 32)}
    full = {k: None if a is None else a.contiguous() for k, a in e.items()}
    assert torch.equal(gla.selective_scan(**e)[0], gla.selective_scan(**full)[0])


@pytest.mark.gpu
def test_gradients_against_differences():
    """Directional derivatives in fp64 differences of the kernel's own fp32 results: a step of 2^-7 is off by its square times
    the third derivative (1e-4) and by the results' rounding over the step (1e-4 of the sum's terms)."""
    t, dy, dST = make(1, 40, 16, 8, 1, torch.float32, 13)
    args = [t[n].contiguous() for n in NAMES]
    got = gla.selective_scan_backward(*args, dy, dST)
    g = torch.Generator().manual_seed(1)
    for i, n in enumerate(NAMES):
        way = torch.randn(args[i].shape, generator=g).cuda() * (0.01 if n == "A" else 0.1)
        def loss(s):
            y, ST = gla.selective_scan_forward(*args[:i], args[i] + s * way, *args[i + 1:])
            return float((y.double() * dy.double()).sum() + (ST.double() * dST.double()).sum())
        diff = (loss(2.0 ** -7) - loss(-2.0 ** -7)) * 2 ** 6
        want = float((got[i].double() * way.double()).sum())
        size = float((got[i].double() * way.double()).square().sum().sqrt()) + 1
        assert abs(diff - want) <= 2e-2 * size, f"{n}: {diff} {want}"


@pytest.mark.gpu
@pytest.mark.parametrize("T,segments", [(5, 0), (70, 1), (70, 3)])
def test_not_finite_values_stay_in_their_channel_and_after_their_token(T, segments):
    """A NaN or an infinity in one channel's x, dt or z, or in its state, reaches no other channel and no token before it."""
    t, _, _ = make(1, T, 64, 16, 1, torch.float32, 14)
    t = {n: a.contiguous() for n, a in t.items()}
    y, ST = gla.selective_scan_forward(**t, force_segments=segments)
    v = {n: a.clone() for n, a in t.items()}
    at = T - 3
    v["x"][0, at, 3], v["dt"][0, at, 17], v["z"][0, at, 33], v["S0"][0, 50, 2] = float("nan"), float("inf"), float("nan"), float("inf")
    z, SZ = gla.selective_scan_forward(**v, force_segments=segments)
    same = torch.ones_like(y, dtype=torch.bool)
    same[0, at:, [3, 17, 33]] = False
    same[0, :, 50] = False
    assert torch.equal(z[same], y[same]) and torch.isnan(z[0, at:, 3]).all() and torch.isnan(z[0, at, 33])
    assert torch.equal(z[0, at + 1:, 33], y[0, at + 1:, 33])
    rows = [c for c in range(64) if c not in (3, 17, 50)]
    assert torch.equal(SZ[0, rows], ST[0, rows])


@pytest.mark.gpu
@pytest.mark.parametrize("tiny", [False, True])
def test_states_that_grow_over_segments(tiny):
    """exp(delta A) = e^2 a token: the growth of a segment of 64 tokens is no fp32 number, while the states are: none until the
    last two tokens, or so small that they fit after 48 tokens of it. A token's growth is off by 2^-22 + 2 2^-23, so 48 tokens' by
    below 48 2^-21 = 2.3e-5 if all erred one way; held to 2.5e-5."""
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, D, N = 256, 16, 16
    x, dt, A, B, C, S0 = rnd(1, T, D), torch.full((1, T, D), 2.0), torch.ones(D, N), rnd(1, T, 1, N), rnd(1, T, 1, N), None
    x[:, :T - 2] = 0
    if tiny:
        x, S0 = torch.zeros_like(x), 1e-30 * rnd(1, D, N)
        dt[:, :64], dt[:, 112:] = 0, 0
    args = (x, dt, A, B, C, None, None, None, S0)
    want, last = ref.scan(*ref.double(args), False)
    for segments in (1, 4):
        y, ST = gla.selective_scan_forward(*ref.cuda(args), softplus=False, force_segments=segments)
        ref.near(y, want, "y", 2.5e-5)
        ref.near(ST, last, "ST", 2.5e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [1, 4])
def test_gradients_across_growing_segments(segments):
    """The gradients of the first four tokens' outputs and the states of the last four tokens, with growth between them that neither
    meets and that is no fp32 number."""
    g = torch.Generator().manual_seed(22)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, D, N = 256, 16, 16
    x, dt, A, B, C, dy = rnd(1, T, D), torch.full((1, T, D), 2.0), torch.ones(D, N), rnd(1, T, 1, N), rnd(1, T, 1, N), rnd(1, T, D)
    x[:, :T - 4] = 0
    dy[:, 4:] = 0
    args = (x, dt, A, B, C, None, None, None, None)
    leaves = ref.double(args)
    want, _ = ref.scan(*leaves, False)
    wg = torch.autograd.grad((want * dy.double()).sum(), leaves[:5])
    got = gla.selective_scan_backward(*ref.cuda(args), dy.cuda(), softplus=False, force_segments=segments)
    for n, a, b in zip(NAMES, got, wg):
        ref.near(a, b, "d" + n)


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(x=1 << 24, dt=2 << 24, z=3 << 24, Bm=4 << 24, Cm=5 << 24, x_stride=(512, 64), dt_stride=(512, 64), z_stride=(512, 64),
             B_stride=(128, 16), C_stride=(128, 16), A=6 << 24, D_skip=7 << 24, dt_bias=8 << 24, S0=9 << 24, B=2, T=8, D=64, G=1,
             N=16, softplus=1, dtype=gla.GLA_BF16)
    a.update(kw)
    p = bnd.gla_ssm_params()
    for n, v in a.items():
        setattr(p, n, type(getattr(p, n))(*v) if isinstance(v, tuple) else v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(D=20), 1), (dict(G=16), 1), (dict(N=0), 1),
    (dict(N=12), 2), (dict(N=128), 2), (dict(dtype=2), 1), (dict(force_segments=-1), 1), (dict(x=0), 1), (dict(dt=0), 1),
    (dict(Bm=0), 1), (dict(Cm=0), 1), (dict(A=0), 1), (dict(x=(1 << 24) + 2), 1), (dict(B_stride=(128, 20)), 1),
    (dict(z_stride=(512, 60)), 1), (dict(A=(6 << 24) + 4), 1), (dict(S0=(9 << 24) + 4), 1), (dict(D=1 << 21), 2),
    (dict(T=1 << 30, B=1 << 14), 2),
])
def test_refuses_before_launch(kw, want):
    p = _params(**kw)
    lib = bnd.load()
    assert lib.gla_ssm_fwd(p, 10 << 24, 11 << 24, None, 0, None) == want
    assert lib.gla_ssm_fwd_workspace_size(p) == 0 and lib.gla_ssm_bwd_workspace_size(p) == 0


def test_refuses_outputs():
    lib, p = bnd.load(), _params()
    assert lib.gla_ssm_fwd(None, 10 << 24, None, None, 0, None) == 1
    assert lib.gla_ssm_fwd(p, None, 11 << 24, None, 0, None) == 1
    assert lib.gla_ssm_fwd(p, 1 << 24, 11 << 24, None, 0, None) == 1               # y over x
    assert lib.gla_ssm_fwd(p, 10 << 24, (9 << 24) + 16, None, 0, None) == 1        # ST over S0, elsewhere
    assert lib.gla_ssm_fwd(p, 10 << 24, 11 << 24, 8, 0, None) == 1                 # a workspace off its boundary
    at = [(20 + i) << 24 for i in range(11)]
    assert lib.gla_ssm_bwd(p, bnd.gla_ssm_grads(*at[:7], None, *at[8:]), None, 0, None) == 1      # A's gradient is always formed
    assert lib.gla_ssm_bwd(p, bnd.gla_ssm_grads(*at[:4], None, *at[5:]), None, 0, None) == 1      # z without a place
    assert lib.gla_ssm_bwd(_params(z=None), bnd.gla_ssm_grads(*at), None, 0, None) == 1           # a gradient without z
    assert lib.gla_ssm_bwd(p, bnd.gla_ssm_grads(*at[:3], at[2], *at[4:]), None, 0, None) == 1     # two in one place
    assert lib.gla_ssm_bwd(p, None, None, 0, None) == 1


def test_workspaces():
    lib = bnd.load()
    big = _params(T=2048, D=4096, B=8, x=1 << 40, dt=2 << 40, z=3 << 40, Bm=4 << 40, Cm=5 << 40, A=6 << 40, D_skip=7 << 40,
                  dt_bias=8 << 40, S0=9 << 40)
    assert lib.gla_ssm_fwd_workspace_size(big) == 0                                # channels enough: one walk
    few = _params(T=2048, force_segments=4)
    assert lib.gla_ssm_fwd_workspace_size(few) >= 3 * 2 * 64 * 16 * 4
    # three segments' states and sums, and a copy of S0 for the call that writes ST over it
    assert lib.gla_ssm_fwd_workspace_size(few) >= (3 + 1) * 2 * 64 * 16 * 4 + 3 * 2 * 64 * 4
    assert lib.gla_ssm_fwd_workspace_size(_params()) == 0                          # eight tokens: the step form
    assert lib.gla_ssm_bwd_workspace_size(_params(T=17)) >= 2 * 2 * 64 * 16 * 4    # the states of two tiles


def test_python_checks():
    D, N = 32, 16
    x, A, b = torch.randn(1, 3, D), -torch.rand(D, N), torch.randn(1, 3, 1, N)
    for a in ((x[0], x, A, b, b), (x, x[:, :2], A, b, b), (x, x.bfloat16(), A, b, b), (x, x, A[:8], b, b), (x, x, A.double(), b, b),
              (x, x, A, b[..., 0], b), (x, x, A, b, b[:, :2]), (x, x, A, b, b, torch.ones(8)), (x, x, A, b, b, None, x[0]),
              (x, x, A, b, b, None, None, torch.ones(D).double()), (x, x, A, b, b, None, None, None, torch.zeros(1, D, 8)),
              (x, x, A, torch.randn(1, 3, N, 2).transpose(2, 3)[:, :, :1], b), (x.transpose(1, 2), x, A, b, b)):
        with pytest.raises(gla.GlaError):
            gla.selective_scan(*a)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.selective_scan(x, x, A, b, b)
