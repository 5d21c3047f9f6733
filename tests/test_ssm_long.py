"""The selective scan where the form taken or the arithmetic differs from a short call's: few tokens of many rows, long prompts cut
as the planner does, memories longer than the call, steps so small that 1 + exp(dt) is 1."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref
from test_ssm import NAMES, make

U = 2.0 ** -24                 # half a step of fp32 at one


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T,over,without", [(8, 1, 1, ()), (16, 2, 3, ("z", "S0")), (32, 1, 2, ("D", "dt_bias")), (64, 8, 1, ()),
                                              (16, 1, 0, ())])
def test_few_tokens_of_many_rows(N, T, over, without, dtype):
    """Four batch rows to a thread, taken from 16384 states a multiprocessor on; `over` rows are left over. Two groups of B and C,
    channels that end inside a block, the state carried in place. Tolerances as for the other calls, of less than eight decays."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    D = 65536 // N + 16
    B = -(-16384 * sms // (D * N))
    B += (over - B) % 4
    t, _, _ = make(B, T, D, N, 2, dtype, N + T, without)
    y, ST = gla.selective_scan(**t)
    with torch.no_grad():
        want, last = ref.scan(*ref.double(t.values(), False), True)
    ref.near(y, want, "y")
    ref.near(ST, last, "ST")
    if t["S0"] is not None:
        state = t["S0"].clone()
        y2, _ = gla.selective_scan_forward(**{**t, "S0": state}, ST=state)
        assert torch.equal(y2, y) and torch.equal(state, ST)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,N,G,dtype", [(1, 4099, 64, 16, 1, torch.float32), (1, 2600, 48, 8, 1, torch.bfloat16),
                                             (2, 1500, 32, 64, 2, torch.float32), (1, 2053, 96, 32, 3, torch.bfloat16)])
def test_long_prompts_of_few_channels(B, T, D, N, G, dtype):
    """Cut into many segments by the planner, forward and backward. The states' decays are good to 4e-6 of their size (memories of
    up to 200 tokens) and the sums add 30 roundings, each of terms of up to ten times a tensor's root mean square: 6e-5 of it; sums over
    the tokens 1e-5 of their norm."""
    t, dy, dST = make(B, T, D, N, G, dtype, T)
    args = [t[n] for n in NAMES]
    packed, _, _ = bnd._ssm_params(*args, True)
    assert bnd._workspace("gla_ssm_fwd_workspace_size", packed, dy.device)[2] > 16 * B * D * N * 4      # 16 segments and more
    y, ST = gla.selective_scan_forward(*args)
    got = gla.selective_scan_backward(*args, dy, dST)
    leaves = ref.double(args)
    want, last = ref.scan(*leaves, True)
    ref.near(y, want, "y", 6e-5)
    ref.near(ST, last, "ST", 6e-5)
    wg = torch.autograd.grad((want * dy.double().cpu()).sum() + (last * dST.double().cpu()).sum(), leaves)
    for n, a, b in zip(NAMES, got, wg):
        if n in ("A", "D", "dt_bias"):
            e = float((a.double().cpu() - b).norm() / b.norm())
            assert e <= 1e-5, f"d{n}: {e:.1e}"
        else:
            ref.near(a, b, "d" + n, 6e-5)


@pytest.mark.gpu
def test_memories_longer_than_the_call():
    """States that only decay, by exp(-1e-3) or so a token, and the gradients of those that enter: S0 exp(A sum of delta), and dST
    times the same. A walk multiplies by one decay every 16 tokens (2048 of them: 128 decays, each good to 2^-23, and a rounding:
    2.3e-5 if all erred one way), a call of up to eight tokens by one a token, for which that is 3.7e-4. Roundings of a state at every
    token are common to both, sqrt(2048) U = 2.7e-6 at most; what 16 times fewer decays add is a fourth if they err at random and a
    sixteenth if not. So the walks' error is held to half of what the same tokens give in calls of eight."""
    g = torch.Generator().manual_seed(31)
    B, T, D, N = 1, 2048, 64, 16
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt, A = rnd(B, T, D) * 0.3 - 6.9, -(0.5 + torch.rand(D, N, generator=g))
    S0, dST = rnd(B, D, N), rnd(B, D, N)
    decay = torch.exp(A.double() * torch.nn.functional.softplus(dt.double()).sum(1).unsqueeze(2))
    none, bc = torch.zeros(B, T, D), rnd(B, T, 1, N)
    x, dt, A, bc, S0, dST = (t.cuda() for t in (none, dt, A, bc, S0, dST))
    off = lambda got, start: float(((got.double() - start.double() * decay.cuda()).norm() / (start.double() * decay.cuda()).norm()))  # noqa: E731
    state = S0.clone()
    for t in range(0, T, 8):
        p = slice(t, t + 8)
        gla.selective_scan_forward(x[:, p], dt[:, p], A, bc[:, p], bc[:, p], S0=state, ST=state)
    singly = off(state, S0)
    for segments in (0, 1, 8):
        _, ST = gla.selective_scan_forward(x, dt, A, bc, bc, S0=S0, force_segments=segments)
        dS0 = gla.selective_scan_backward(x, dt, A, bc, bc, None, None, None, S0, x, dST, force_segments=segments)[8]
        for n, e in (("ST", off(ST, S0)), ("dS0", off(dS0, dST))):
            assert e <= min(2.3e-5, singly / 2), f"{n} in {segments} segments: {e:.1e}, {singly:.1e} in calls of eight tokens"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,segments", [(5, 0), (20, 1), (20, 2)])
def test_small_steps_keep_their_digits(T, segments, dtype):
    """dt from -20 to -6, steps of 2e-9 to 2.5e-3: every value relative to itself. All terms are positive, so a sum is as good as its
    terms. exp(dt) is off by 4 U and |dt| (U + 1.3e-8) (its argument's rounding, and that of log2 e), softplus by 6 U more, a
    decay by 6 U, of at most 20 tokens; products and sums over tokens and 8 states 30 U: 160 U + |dt| 7.3e-8 in all. A gradient holds
    as much of its own side, and the sigmoid as much as exp(dt) again; what cancels is a twentieth (delta A of 20 tokens). A
    logarithm of the rounded 1 + exp(dt) is off by 400 U at dt = -6 and by everything at -17."""
    g = torch.Generator().manual_seed(T)
    D, N = 64, 8
    pos = lambda *s: (0.5 + torch.rand(s, generator=g)).to(dtype)  # noqa: E731
    dt = (torch.linspace(-20, -6, D) + 0.05 * torch.rand(1, T, D, generator=g)).to(dtype)
    x, A, Bm, C, dy = pos(1, T, D), -pos(D, N).float(), pos(1, T, 1, N), pos(1, T, 1, N), pos(1, T, D)
    args = (x, dt, A, Bm, C, None, None, None, None)
    y, ST = gla.selective_scan_forward(*ref.cuda(args), force_segments=segments)
    got = gla.selective_scan_backward(*ref.cuda(args), dy.cuda(), force_segments=segments)
    leaves = ref.double(args)
    want, last = ref.scan(*leaves, True)
    wg = torch.autograd.grad((want * dy.double()).sum(), leaves[:5])
    v = 20.0 - (14.0 / (D - 1)) * torch.arange(D, dtype=torch.float64)      # |dt| of a channel, at most
    one = 160 * U + 7.3e-8 * v
    for n, a, b, tol in (("y", y, want, one), ("ST", ST, last, one[:, None]), ("dx", got[0], wg[0], 1.1 * one),
                         ("ddt", got[1], wg[1], 1.1 * one + 20 * U + 7.3e-8 * v), ("dA", got[2], wg[2], 2.1 * one[:, None])):
        tol = tol + (2.0 ** -8 if a.dtype == torch.bfloat16 else 0)
        worst = float(((a.double().cpu() - b.detach()).abs() / (b.detach().abs() * tol)).max())
        assert (b > 0).all() and worst <= 1, f"{n}: {worst:.2f} of its bound"
