"""The gated delta rule (gla_delta_fwd, gla_delta_bwd) against the fp64 recurrence.

Tolerances. O, dq, dk, dv and dbeta in bf16: the library's bf16 contract (_util.TOL; a final
rounding of at most 2^-8 relative and two operand roundings of that size in O). The chunk form's
fp32 results pass through products of two-part bf16 operands, each part pair good to 2^-17: S_T
and dS0 go through four of them (state, right-hand side, inverse, correction), so 4 x 2^-17 of the
norm; dlog_g sums products of two such operands, twice that. The recurrent form is fp32 throughout:
sums of at most 256 terms a token, 1e-5."""
import ctypes

import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _delta_ref as ref
from _util import assert_close, errors, to_np

PARTS = 2.0 ** -17
NAMES = ("dq", "dk", "dv", "dlog_g", "dbeta", "dS0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def close(got, want, tol, what):
    e, _ = errors(to_np(got), to_np(want))
    assert e <= tol, f"{what}: relative error {e:.2e} > {tol:.2e}"


def check_forward(x, scale=None, path=gla.GLA_PATH_AUTO):
    sc = x[0].shape[3] ** -0.5 if scale is None else scale
    O, S = ref.delta(*ref.f64(x), sc)
    got_O, got_S = gla.delta_forward(*ref.cuda(x), scale=scale, path=path)
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    chunk = path == gla.GLA_PATH_TENSOR
    if x[0].dtype == torch.bfloat16:
        assert_close(to_np(got_O), to_np(O), torch.bfloat16, "O")
    else:
        close(got_O, O, 1e-5, "O")
    close(got_S, S, 4 * PARTS if chunk else 1e-5, "S_T")


def reference_grads(x, dO, dST, scale):
    leaves = [None if t is None else t.double().requires_grad_(True) for t in x]
    O, S = ref.delta(*leaves, scale)
    loss = (O * dO.double()).sum() + (0 if dST is None else (S * dST.double()).sum())
    want = torch.autograd.grad(loss, [t for t in leaves if t is not None], allow_unused=True)
    it = iter(want)
    return [None if t is None else next(it) for t in leaves]


def check_backward(x, dO, dST, path=gla.GLA_PATH_AUTO):
    want = reference_grads(x, dO, dST, x[0].shape[3] ** -0.5)
    got = gla.delta_backward(*ref.cuda(x), dO.cuda(), None if dST is None else dST.cuda(), path=path)
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    chunk = path == gla.GLA_PATH_TENSOR
    bf = x[0].dtype == torch.bfloat16
    for name, g, w in zip(NAMES, got, want):
        if w is None:
            continue
        assert torch.isfinite(g).all(), name
        if bf and name in ("dq", "dk", "dv", "dbeta"):
            assert_close(to_np(g), to_np(w), torch.bfloat16, name)
        else:
            close(g, w, ((8 if name == "dlog_g" else 4) * PARTS) if chunk else 2e-5, name)


def test_reference_gradient_against_differences():
    x, g = ref.make(1, 2, 1, 5, 16, 16, torch.float64, seed=3, keys="unit")
    x = ref.f64(x)
    dO = torch.randn(x[2].shape, generator=g, dtype=torch.float64)
    dST = torch.randn(x[5].shape, generator=g, dtype=torch.float64)
    want = reference_grads(x, dO, dST, 0.25)
    f = lambda y: sum((a * b).sum() for a, b in zip(ref.delta(*y, 0.25), (dO, dST)))  # noqa: E731
    for i, t in enumerate(x):
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        up, down = list(x), list(x)
        up[i], down[i] = t + 1e-5 * d, t - 1e-5 * d
        assert abs((f(up) - f(down)) / 2e-5 - (want[i] * d).sum()) <= 1e-7 * (1 + want[i].norm() * d.norm())


# ---------------------------------------------------------------- refusals, no GPU needed

def _params(**kw):
    a = dict(q=1 << 12, k=2 << 12, v=3 << 12, log_g=4 << 12, beta=5 << 12, S0=0, O=6 << 12, ST=7 << 12,
             B=1, H=2, Hk=1, T=4, dk=64, dv=64, scale=0.125, dtype=gla.GLA_BF16, path=gla.GLA_PATH_AUTO)
    a.update(kw)
    p = bnd.gla_delta_params()
    for n, v in a.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 1),
    (dict(H=3, Hk=2), 1), (dict(Hk=0), 1), (dict(T=-1), 1), (dict(dk=24), 1), (dict(dv=8), 1),
    (dict(dtype=7), 1), (dict(path=gla.GLA_PATH_FUSED), 1), (dict(scale=float("nan")), 1), (dict(dk=272), 2),
    (dict(q=0), 1), (dict(beta=0), 1), (dict(O=0), 1), (dict(q=(1 << 12) + 8), 1), (dict(ST=(7 << 12) + 4), 1),
    (dict(O=3 << 12), 1), (dict(ST=1 << 12), 1), (dict(S0=(7 << 12) + 64), 1),
    (dict(path=gla.GLA_PATH_TENSOR, dk=128, dv=80), 2), (dict(path=gla.GLA_PATH_TENSOR, dtype=gla.GLA_FP32), 2),
    (dict(path=gla.GLA_PATH_TENSOR, dk=256), 2), (dict(path=gla.GLA_PATH_TENSOR, T=(1 << 25) + 1), 2),
])
def test_forward_refuses_before_launch(kw, want):
    assert bnd.gla_delta_fwd(_params(**kw), 0, check=False) == want


@pytest.mark.parametrize("T,want", [(2 ** 31 - 1, 2), (2 ** 31 - 15, 2), (2 ** 31 - 16, 1)])
def test_the_longest_sequences(T, want):
    """The step of 16 past the last token is an int up to 2^31 - 16 (nothing runs: q is missing, which is looked at next)."""
    assert bnd.gla_delta_fwd(_params(T=T, q=0), 0, check=False) == want
    p = bnd.gla_delta_bwd_params()
    for n, v in dict(B=1, H=1, Hk=1, T=T, dk=16, dv=16, scale=1.0, dtype=gla.GLA_BF16).items():
        setattr(p, n, v)
    assert bnd.gla_delta_bwd(p, 0, check=False) == want
    assert (bnd.gla_delta_bwd_workspace_size(p) > 0) == (want == 1)


def test_null_params_are_refused():
    lib = bnd.load()
    assert lib.gla_delta_fwd(None, None) == 1 and lib.gla_delta_bwd(None, None) == 1
    assert lib.gla_delta_fwd_workspace_size(None) == 0 and lib.gla_delta_bwd_workspace_size(None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(grad_q=0), 1), (dict(grad_O=0), 1), (dict(log_g=0, grad_log_g=13 << 12), 1), (dict(grad_v=3 << 12), 1),
    (dict(grad_k=9 << 12), 1), (dict(dk=272), 2), (dict(grad_S0=(15 << 12) + 4), 1),
])
def test_backward_refuses_before_launch(kw, want):
    p = bnd.gla_delta_bwd_params()
    a = dict(q=1 << 12, k=2 << 12, v=3 << 12, log_g=4 << 12, beta=5 << 12, grad_O=6 << 12, grad_q=9 << 12,
             grad_k=10 << 12, grad_v=11 << 12, grad_beta=12 << 12, B=1, H=2, Hk=1, T=4, dk=64, dv=64, scale=0.125,
             dtype=gla.GLA_BF16)
    a.update(kw)
    for n, v in a.items():
        setattr(p, n, v)
    assert bnd.gla_delta_bwd(p, 0, check=False) == want


def test_struct_layout():
    assert ctypes.sizeof(bnd.gla_delta_params) == 8 * 8 + 9 * 4 + 4 + 16 + 8
    assert ctypes.sizeof(bnd.gla_delta_bwd_params) == 14 * 8 + 9 * 4 + 4 + 16


def test_python_checks_shapes():
    x, _ = ref.make(1, 2, 1, 4, 64, 64, torch.bfloat16)
    for i, bad in ((1, x[1][:, :, :3]), (2, x[2].float()), (3, x[3].double()), (4, x[4].transpose(1, 2)),
                   (5, x[5].transpose(2, 3)), (0, x[0][0])):
        y = list(x)
        y[i] = bad
        with pytest.raises(gla.GlaError):
            gla.delta_forward(*y)
    with pytest.raises(gla.GlaError, match="not on a GPU"):
        gla.delta_forward(*x)


def test_plans_on_host():
    """Workspace only for the segments of a cut sequence: a state and a transition each but the last, and a state
    entering each."""
    seg = 2 * (3 * (64 * 64 + 64 * 64) + 4 * 64 * 64) * 4     # H = 2, four segments
    assert bnd.gla_delta_fwd_workspace_size(_params(T=500, force_segments=4)) == seg
    assert bnd.gla_delta_fwd_workspace_size(_params(T=500, force_segments=1)) == 0
    assert bnd.gla_delta_fwd(_params(T=500, force_segments=-1), 0, check=False) == 1
    assert bnd.gla_delta_fwd_workspace_size(_params(T=1)) == 0
    assert bnd.gla_delta_fwd_workspace_size(_params(T=500, dtype=gla.GLA_FP32)) == 0
    assert bnd.gla_delta_fwd_workspace_size(_params(T=500, dk=80)) == 0


# ---------------------------------------------------------------- forward

SHAPES = [(1, 1, 1, 1), (2, 3, 1, 2), (1, 2, 2, 63), (1, 2, 1, 64), (2, 2, 1, 65), (1, 4, 2, 200)]


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["sigmoid", "none", "steep", "resets"])
@pytest.mark.parametrize("B,H,Hk,T", SHAPES)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 192), (64, 256)])
def test_chunk_form(B, H, Hk, T, dk, dv, gate):
    check_forward(ref.make(B, H, Hk, T, dk, dv, torch.bfloat16, seed=T, gate=gate, s0=T % 2 == 0)[0],
                  path=gla.GLA_PATH_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("keys,beta", [("same", "one"), ("same", "sigmoid"), ("unit", "holes"), ("unit", "one")])
def test_chunk_form_of_dependent_keys(keys, beta):
    x = ref.make(1, 2, 1, 150, 128, 128, torch.bfloat16, seed=9, keys=keys, beta=beta)[0]
    check_forward(x, path=gla.GLA_PATH_TENSOR)
    check_forward(x, path=gla.GLA_PATH_SIMT)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["sigmoid", "none", "steep", "resets"])
@pytest.mark.parametrize("T,dk,dv", [(1, 128, 128), (1, 16, 16), (5, 64, 80), (17, 256, 64), (40, 48, 144), (2, 208, 128)])
def test_recurrent_form(T, dk, dv, gate, dtype):
    check_forward(ref.make(2, 4, 2, T, dk, dv, dtype, seed=T, gate=gate)[0], path=gla.GLA_PATH_SIMT)


@pytest.mark.gpu
@pytest.mark.parametrize("segments", [2, 3, 7])
@pytest.mark.parametrize("gate", ["sigmoid", "steep", "resets"])
@pytest.mark.parametrize("dk,dv,T", [(128, 128, 430), (64, 192, 449), (128, 64, 131)])
def test_cut_sequences(dk, dv, T, gate, segments):
    x = ref.make(1, 2, 1, T, dk, dv, torch.bfloat16, seed=T, gate=gate, s0=segments != 3)[0]
    O, S = ref.delta(*ref.f64(x), dk ** -0.5)
    got_O, got_S = gla.delta_forward(*ref.cuda(x), path=gla.GLA_PATH_TENSOR, force_segments=segments)
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    assert_close(to_np(got_O), to_np(O), torch.bfloat16, "O")
    close(got_S, S, 6 * PARTS, "S_T")        # the transition's two-part operands too


@pytest.mark.gpu
@pytest.mark.parametrize("H,segments", [(40, 3), (24, 5), (24, 6), (24, 7), (20, 4), (16, 8), (16, 9)])
@pytest.mark.parametrize("T", [320, 900])
def test_cut_sequences_of_more_heads(H, segments, T):
    """Two segments to a CTA of the first walk where one wave would not hold them singly; odd and even numbers."""
    x = ref.make(1, H, H // 2, T, 64, 64, torch.bfloat16, seed=T + segments)[0]
    O, S = ref.delta(*ref.f64(x), 64 ** -0.5)
    got_O, got_S = gla.delta_forward(*ref.cuda(x), path=gla.GLA_PATH_TENSOR, force_segments=segments)
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    assert_close(to_np(got_O), to_np(O), torch.bfloat16, "O")
    close(got_S, S, 6 * PARTS, "S_T")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 64, 65, 100, 127, 128])
def test_more_segments_than_chunks(T):
    x = ref.make(1, 2, 2, T, 64, 64, torch.bfloat16, seed=T)[0]
    O, S = ref.delta(*ref.f64(x), 64 ** -0.5)
    got_O, got_S = gla.delta_forward(*ref.cuda(x), path=gla.GLA_PATH_TENSOR, force_segments=3)
    assert_close(to_np(got_O), to_np(O), torch.bfloat16, "O")
    close(got_S, S, 6 * PARTS, "S_T")


@pytest.mark.gpu
def test_recurrent_form_with_wide_tiles():
    """More tiles than multiprocessors: the wide tile."""
    check_forward(ref.make(40, 8, 4, 3, 128, 128, torch.bfloat16, seed=1)[0])
    check_forward(ref.make(40, 8, 8, 2, 64, 128, torch.float32, seed=2)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("path", [gla.GLA_PATH_TENSOR, gla.GLA_PATH_SIMT])
def test_carried_in_place_over_calls(path):
    """A sequence in pieces, the state carried in place, equals the sequence at once; its scale is the caller's."""
    x, _ = ref.make(1, 2, 1, 150, 128, 128, torch.bfloat16, seed=5)
    O, S = ref.delta(*ref.f64(x), 0.5)
    q, k, v, lg, be, S0 = ref.cuda(x)
    state, outs = S0.clone(), []
    for a, b in ((0, 70), (70, 71), (71, 150)):
        cut = lambda t: t[:, :, a:b].contiguous()  # noqa: E731
        o, s = gla.delta_forward(cut(q), cut(k), cut(v), cut(lg), cut(be), state, scale=0.5, path=path, ST=state)
        assert s is state
        outs.append(o)
    assert_close(to_np(torch.cat(outs, 2)), to_np(O), torch.bfloat16, "O")
    close(state, S, 8 * PARTS, "state")


@pytest.mark.gpu
def test_empty_sequence():
    x, _ = ref.make(1, 2, 1, 0, 64, 64, torch.bfloat16)
    O, S = gla.delta_forward(*ref.cuda(x))
    assert O.shape == (1, 2, 0, 64) and torch.equal(S.cpu(), x[5])
    x[5] = None
    assert not gla.delta_forward(*ref.cuda(x))[1].any()
    dST = torch.randn(1, 2, 64, 64)
    assert torch.equal(gla.delta_backward(*ref.cuda(x), torch.zeros(1, 2, 0, 64).bfloat16().cuda(), dST.cuda())[5].cpu(), dST)


@pytest.mark.gpu
def test_passed_over_tokens_leave_the_state():
    """beta = 0 and log_g = 0: bitwise the state of before, whatever q, k and v hold."""
    x, _ = ref.make(1, 2, 1, 64, 128, 128, torch.bfloat16, seed=4)
    x[3], x[4] = torch.zeros_like(x[3]), torch.zeros_like(x[4])
    for path in (gla.GLA_PATH_TENSOR, gla.GLA_PATH_SIMT):
        assert torch.equal(gla.delta_forward(*ref.cuda(x), path=path)[1].cpu(), x[5])


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("path", [gla.GLA_PATH_TENSOR, gla.GLA_PATH_SIMT])
def test_how_far_a_bad_value_reaches(path, bad):
    x, _ = ref.make(1, 2, 2, 150, 128, 128, torch.bfloat16, seed=18)
    O, S = gla.delta_forward(*ref.cuda(x), path=path)
    first = 64 if path == gla.GLA_PATH_TENSOR else 70      # the first token that it may reach
    y = [t.clone() for t in x]
    y[2][0, 1, 70, 3] = bad
    got_O, got_S = gla.delta_forward(*ref.cuda(y), path=path)
    assert torch.equal(got_O[:, 0], O[:, 0]) and torch.equal(got_S[:, 0], S[:, 0])
    rest = [c for c in range(128) if c != 3]
    assert torch.equal(got_O[0, 1][:, rest], O[0, 1][:, rest]) and torch.equal(got_S[0, 1][:, rest], S[0, 1][:, rest])
    assert torch.equal(got_O[0, 1, :first], O[0, 1, :first])
    assert not torch.isfinite(got_O[0, 1, 70:, 3]).any() and not torch.isfinite(got_S[0, 1, :, 3]).any()
    y = [t.clone() for t in x]
    y[1][0, 1, 70, 5] = bad
    got_O, got_S = gla.delta_forward(*ref.cuda(y), path=path)
    assert torch.equal(got_O[:, 0], O[:, 0]) and torch.equal(got_O[0, 1, :first], O[0, 1, :first])
    assert not torch.isfinite(got_S[0, 1]).any()
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0


@pytest.mark.gpu
def test_streams_and_bitwise_repeats():
    x, g = ref.make(2, 4, 2, 130, 128, 128, torch.bfloat16, seed=6)
    dO = torch.randn(x[2].shape, generator=g).bfloat16().cuda()
    c = ref.cuda(x)
    first = [*gla.delta_forward(*c), *gla.delta_backward(*c, dO)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        again = [*gla.delta_forward(*c, stream=s), *gla.delta_backward(*c, dO, stream=s)]
        torch.cuda.synchronize()
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 200])
def test_replays_from_a_cuda_graph(T):
    """Forward and backward captured at the binding's level, replayed on new inputs."""
    x, g = ref.make(1, 4, 2, T, 128, 128, torch.bfloat16, seed=7)
    buf = ref.cuda(x)
    dO = torch.randn(x[2].shape, generator=g).bfloat16()
    dbuf = dO.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gla.delta_forward(*buf)
        gla.delta_backward(*buf, dbuf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = [*gla.delta_forward(*buf), *gla.delta_backward(*buf, dbuf)]
    for seed in (8, 9):
        y, _ = ref.make(1, 4, 2, T, 128, 128, torch.bfloat16, seed=seed)
        for b, t in zip(buf, y):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = [*gla.delta_forward(*ref.cuda(y)), *gla.delta_backward(*ref.cuda(y), dbuf)]
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- backward

@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["sigmoid", "none", "steep", "resets"])
@pytest.mark.parametrize("B,H,Hk,T", [(1, 1, 1, 1), (2, 4, 2, 64), (1, 2, 1, 65), (1, 2, 2, 200)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 192)])
def test_chunk_backward(B, H, Hk, T, dk, dv, gate):
    x, g = ref.make(B, H, Hk, T, dk, dv, torch.bfloat16, seed=T + 1, gate=gate, s0=T != 64)
    dO = torch.randn(x[2].shape, generator=g).bfloat16()
    dST = torch.randn((B, H, dk, dv), generator=g) if T % 2 else None
    check_backward(x, dO, dST, path=gla.GLA_PATH_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,dk,dv", [(1, 64, 64), (17, 128, 80), (33, 48, 144), (16, 256, 32)])
def test_recurrent_backward(T, dk, dv, dtype):
    x, g = ref.make(2, 4, 2, T, dk, dv, dtype, seed=T, gate="resets" if T == 33 else "sigmoid")
    dO = torch.randn(x[2].shape, generator=g).to(dtype)
    dST = torch.randn((2, 4, dk, dv), generator=g)
    check_backward(x, dO, dST, path=gla.GLA_PATH_SIMT)


@pytest.mark.gpu
@pytest.mark.parametrize("keys,beta", [("same", "one"), ("unit", "holes")])
def test_backward_of_dependent_keys_and_holes(keys, beta):
    """beta = 0 included: dbeta there is not zero (the chunk form takes it as 2^-40)."""
    x, g = ref.make(1, 2, 1, 100, 64, 64, torch.bfloat16, seed=11, keys=keys, beta=beta)
    dO = torch.randn(x[2].shape, generator=g).bfloat16()
    check_backward(x, dO, None, path=gla.GLA_PATH_TENSOR)
    check_backward(x, dO, None, path=gla.GLA_PATH_SIMT)


@pytest.mark.gpu
def test_backward_against_differences_of_the_forward():
    """fp32, recurrent form: the directional derivative by central differences of the kernel itself. With a step of
    2^-6 the differences are off by a third derivative's 2^-12 / 6 and by fp32 rounding over the step, 2^-24 2^6."""
    x, g = ref.make(1, 2, 1, 20, 64, 64, torch.float32, seed=12)
    dO = torch.randn(x[2].shape, generator=g)
    grads = gla.delta_backward(*ref.cuda(x), dO.cuda())
    f = lambda y: (gla.delta_forward(*ref.cuda(y))[0].double().cpu() * dO).sum()  # noqa: E731
    for i in (0, 1, 2, 3, 4, 5):
        d = torch.randn(x[i].shape, generator=g) * x[i].norm() / x[i].numel() ** 0.5
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + d / 64, x[i] - d / 64
        want = (grads[i].double().cpu() * d).sum()
        assert abs((f(up) - f(down)) * 32 - want) <= 4e-3 * grads[i].double().norm().cpu() * d.norm() ** 1


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hk,T,dk,dv,gate,keys", [
    (1, 1, 1, 6000, 128, 128, "sigmoid", "unit"), (1, 2, 1, 4100, 64, 128, "none", "unit"),
    (2, 2, 2, 2999, 128, 64, "none", "same"), (1, 4, 2, 5000, 64, 64, "resets", "unit")])
def test_long_prompts_are_cut_by_the_planner(B, H, Hk, T, dk, dv, gate, keys):
    """AUTO's own split of a long prompt of few heads (its workspace shows that there is one) against fp64. Every increment
    of the state is good to four two-part operands' 2^-17 and so are the joins; the errors do not grow along the sequence,
    as no step of unit keys grows the state."""
    x = ref.make(B, H, Hk, T, dk, dv, torch.bfloat16, seed=T, gate=gate, keys=keys)[0]
    p = _params(B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv)
    state = B * H * dk * dv * 4
    assert bnd.gla_delta_fwd_workspace_size(p) >= 2 * 3 * state     # three segments or more
    O, S = ref.delta(*ref.f64(x), dk ** -0.5)
    got_O, got_S = gla.delta_forward(*ref.cuda(x))
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    assert_close(to_np(got_O), to_np(O), torch.bfloat16, "O")
    close(got_S, S, 6 * PARTS, "S_T")


@pytest.mark.gpu
@pytest.mark.parametrize("T,dk,dv,gate", [(1300, 128, 128, "sigmoid"), (1100, 64, 192, "none"), (900, 128, 64, "resets")])
def test_chunk_backward_of_many_chunks(T, dk, dv, gate):
    x, g = ref.make(1, 2, 1, T, dk, dv, torch.bfloat16, seed=T, gate=gate)
    dO = torch.randn(x[2].shape, generator=g).bfloat16()
    check_backward(x, dO, torch.randn((1, 2, dk, dv), generator=g), path=gla.GLA_PATH_TENSOR)


@pytest.mark.gpu
@pytest.mark.parametrize("path", [gla.GLA_PATH_TENSOR, gla.GLA_PATH_SIMT])
def test_gradients_that_are_not_wanted(path):
    """grad_log_g, grad_beta and grad_S0 absent: the others are the same, bit for bit; a short workspace is refused."""
    x, _ = ref.make(1, 4, 2, 70, 64, 64, torch.bfloat16, seed=3)
    c = ref.cuda(x)
    dO = torch.ones_like(c[2])
    want = gla.delta_backward(*c, dO, path=path)
    out = [torch.empty_like(t) for t in c[:3]]
    p = bnd.gla_delta_bwd_params(*(t.data_ptr() for t in c), dO.data_ptr(), None, *(t.data_ptr() for t in out),
                                 None, None, None, 1, 4, 2, 70, 64, 64, 0.125, gla.GLA_BF16, path)
    ws = torch.empty(bnd.gla_delta_bwd_workspace_size(p), dtype=torch.uint8, device="cuda")
    p.workspace, p.workspace_bytes = ws.data_ptr(), ws.numel()
    bnd.gla_delta_bwd(p)
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    p.workspace_bytes -= 1
    assert bnd.gla_delta_bwd(p, check=False) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("path", [gla.GLA_PATH_TENSOR, gla.GLA_PATH_SIMT])
@pytest.mark.parametrize("T,dk,dv", [(6, 128, 192), (84, 128, 192), (200, 64, 64), (70, 64, 320)])
@pytest.mark.parametrize("decay", [2.0, 6.0, 14.0])
def test_gradients_of_a_steep_gate(decay, T, dk, dv, path):
    """Every token decays by about exp(-decay): what is left to differentiate is as small as that, and has all its digits
    (the same bound relative to its own size as for any gate)."""
    x, g = ref.make(1, 3, 3, T, dk, dv, torch.bfloat16, seed=T)
    x[3] = -decay * (1 + torch.rand(x[3].shape, generator=g) / 4)
    dO = torch.randn(x[2].shape, generator=g).bfloat16()
    want = reference_grads(x, dO, None, dk ** -0.5)
    got = gla.delta_backward(*ref.cuda(x), dO.cuda(), path=path)
    for n in (3, 5):
        close(got[n], want[n], (8 if n == 3 else 4) * PARTS, NAMES[n])
    for n in (0, 1, 2, 4):
        assert_close(to_np(got[n]), to_np(want[n]), torch.bfloat16, NAMES[n])


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(6))
def test_backward_against_differences_along_the_gradient(i):
    """fp32, recurrent form, one input at a time, moved along its own gradient, so that the derivative is |grad| |d| and a
    wrong part of it shows in full. Central differences of <dO, O> with a step of 2^-6 of the input's norm: in fp64 the
    reference's own are off by 7.7e-5 of the derivative for k, 2.6e-5 for log_g, below 1e-8 for the others (O is linear
    or nearly so in them). O's rounding in fp32, 16 x 2^-24 of each value, over the step: at most 6e-5 (log_g). Together
    below 2^-12."""
    x, g = ref.make(1, 2, 1, 20, 64, 64, torch.float32, seed=12)
    dO = torch.randn(x[2].shape, generator=g)
    grad = gla.delta_backward(*ref.cuda(x), dO.cuda())[i].double().cpu()
    f = lambda y: (gla.delta_forward(*ref.cuda(y))[0].double().cpu() * dO.double()).sum()  # noqa: E731
    d = (grad / grad.norm() * x[i].norm()).float()
    up, down = list(x), list(x)
    up[i], down[i] = x[i] + d / 64, x[i] - d / 64
    got = (f(up) - f(down)) * 32
    want = (grad * d.double()).sum()
    assert abs(got - want) <= 2.0 ** -12 * abs(want), (got, want)


@pytest.mark.gpu
def test_autograd_and_unused_outputs():
    x, g = ref.make(1, 2, 1, 70, 64, 64, torch.bfloat16, seed=13)
    leaves = [t.cuda().requires_grad_(True) for t in x]
    O, ST = gla.delta_attention(*leaves)
    dO, dST = torch.randn(O.shape, generator=g).bfloat16(), torch.randn(ST.shape, generator=g)
    got = torch.autograd.grad((O, ST), leaves, (dO.cuda(), dST.cuda()), retain_graph=True)
    direct = gla.delta_backward(*[t.detach() for t in leaves], dO.cuda(), dST.cuda())
    for a, b, t in zip(got, direct, leaves):
        assert a.dtype == t.dtype and torch.equal(a, b)
    only_state = torch.autograd.grad(ST, leaves, dST.cuda(), retain_graph=True)
    zero = gla.delta_backward(*[t.detach() for t in leaves], torch.zeros_like(O), dST.cuda())
    for a, b in zip(only_state, zero):
        assert torch.equal(a, b)
    (O.float().square().sum()).backward()
    assert all(t.grad is not None for t in leaves)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 100])
def test_training_step_replays_from_a_cuda_graph(T):
    """The norms and the delta rule with their gradients through autograd, captured and replayed on new inputs."""
    def inputs(seed):
        x, g = ref.make(1, 4, 2, T, 64, 64, torch.bfloat16, seed=seed)
        return [*(t.cuda() for t in x), torch.randn(x[2].shape, generator=g).bfloat16().cuda()]

    def step(q, k, v, log_g, beta, S0, dO):
        leaves = [t.detach().requires_grad_(True) for t in (q, k, v, log_g, beta, S0)]
        O, ST = gla.delta_attention(*gla.qk_norm_rope(*leaves[:2]), *leaves[2:])
        return [O.detach(), ST.detach(), *torch.autograd.grad((O, ST), leaves, (dO, torch.ones_like(ST)))]

    buf = inputs(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(*buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(*buf)
    for seed in (2, 3):
        new = inputs(seed)
        for b, t in zip(buf, new):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step(*new)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_outputs_that_are_given_count_as_written():
    """A state carried in place is seen by a graph that saved it, as with any torch operation."""
    x, _ = ref.make(1, 2, 1, 3, 64, 64, torch.bfloat16, seed=15)
    q, k, v, lg, be, S0 = ref.cuda(x)
    O, ST = torch.empty_like(v), S0.clone()
    seen = O._version, ST._version
    gla.delta_forward(q, k, v, lg, be, S0, O=O, ST=ST)
    assert (O._version, ST._version) == (seen[0] + 1, seen[1] + 1)
    leaf = v.clone().requires_grad_(True)
    out, _ = gla.delta_attention(q, k, leaf, lg, be, S0)
    gla.delta_forward(q, k, v, lg, be, S0, ST=S0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    with torch.inference_mode():                       # tensors without versions
        S = S0.clone()
        want = gla.delta_forward(q, k, v, lg, be, S)
        got = gla.delta_forward(q, k, v, lg, be, S, O=torch.empty_like(v), ST=S)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_given_outputs_that_require_gradients_are_refused():
    x, _ = ref.make(1, 2, 1, 3, 64, 64, torch.bfloat16, seed=15)
    for kw in (dict(ST=x[5].clone().requires_grad_(True)), dict(O=x[2].clone().requires_grad_(True))):
        with pytest.raises(gla.GlaError, match="requires grad"):
            gla.delta_forward(*x, **kw)
        with torch.no_grad(), pytest.raises(gla.GlaError, match="not on a GPU"):
            gla.delta_forward(*x, **kw)


@pytest.mark.gpu
def test_gradients_that_arrive_anywhere():
    """What autograd hands to the backward may be a slice that starts at any element (here of a concatenation's)."""
    x, g = ref.make(1, 2, 1, 5, 64, 64, torch.bfloat16, seed=16)
    leaves = [t.cuda().requires_grad_(True) for t in x]
    O, ST = gla.delta_attention(*leaves)
    dO, dST = torch.randn(O.shape, generator=g).bfloat16().cuda(), torch.randn(ST.shape, generator=g).cuda()
    one = lambda t: torch.ones(1, dtype=t.dtype, device="cuda")  # noqa: E731
    after = [torch.cat([one(t), t.flatten()]) for t in (O, ST)]
    got = torch.autograd.grad(after, leaves, [torch.cat([one(t), t.flatten()]) for t in (dO, dST)])
    for a, b in zip(got, gla.delta_backward(*[t.detach() for t in leaves], dO, dST)):
        assert torch.equal(a, b)
    q, k = (torch.randn(1, h, 5, 64, generator=g).bfloat16().cuda().requires_grad_(True) for h in (2, 1))
    qo, ko = gla.qk_norm_rope(q, k)
    dq, dk = torch.randn(q.shape, generator=g).bfloat16().cuda(), torch.randn(k.shape, generator=g).bfloat16().cuda()
    after = [torch.cat([one(t), t.flatten()]) for t in (qo, ko)]
    got = torch.autograd.grad(after, (q, k), [torch.cat([one(t), t.flatten()]) for t in (dq, dk)])
    for a, b in zip(got, gla.qk_norm_rope_backward(q.detach(), k.detach(), dq, dk)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_thread_keeps_its_own_driver_context():
    """A thread that works in a context of its own (made through the driver) finds it current after a call. The call
    launches nothing: no token, no state asked for."""
    import threading
    drv = ctypes.CDLL("libcuda.so.1")
    said = []

    def work():
        ctx, now = ctypes.c_void_p(), ctypes.c_void_p()
        said.append(drv.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))
        p = _params(T=0, ST=0)
        said.append(bnd.load().gla_delta_fwd(ctypes.byref(p), None))
        drv.cuCtxGetCurrent(ctypes.byref(now))
        said.append(now.value == ctx.value)
        drv.cuCtxDestroy_v2(ctx)

    torch.cuda.synchronize()
    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert said == [0, 0, True]


@pytest.mark.gpu
def test_a_thread_without_a_context_gets_one():
    """The first thing that a new thread does is a call in the chunk form (an autograd worker's case)."""
    import threading
    x, _ = ref.make(1, 2, 1, 70, 64, 64, torch.bfloat16, seed=17)
    c = ref.cuda(x)
    O, ST = gla.delta_forward(*c)
    torch.cuda.synchronize()
    got = torch.empty_like(O)
    p = bnd.gla_delta_params(*(t.data_ptr() for t in c), got.data_ptr(), None, 1, 2, 1, 70, 64, 64, 0.125, gla.GLA_BF16,
                             gla.GLA_PATH_TENSOR, None, 0, 1)
    said = []
    t = threading.Thread(target=lambda: said.append(bnd.load().gla_delta_fwd(ctypes.byref(p), None)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert said == [0] and torch.equal(got, O)


@pytest.mark.gpu
def test_calls_in_flight_on_two_streams():
    """Two passes and their gradients at once: neither sees the other's workspace or status."""
    sets = [ref.cuda(ref.make(1, 4, 2, T, 128, 128, torch.bfloat16, seed=T)[0]) for T in (300, 2000)]
    dO = [torch.ones_like(x[2]) for x in sets]
    want = [[*gla.delta_forward(*x), *gla.delta_backward(*x, d)] for x, d in zip(sets, dO)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([*gla.delta_forward(*sets[i]), *gla.delta_backward(*sets[i], dO[i])])
    torch.cuda.synchronize()
    assert gla.gla_device_status() == 0
    for i in range(2):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)


@pytest.mark.gpu
def test_second_device_or_stream_state_is_left_alone():
    """Inputs on the current device, called with another stream current: results are usable after its own sync."""
    x, _ = ref.make(1, 2, 1, 65, 64, 64, torch.bfloat16, seed=14)
    c = ref.cuda(x)
    want = gla.delta_forward(*c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = gla.delta_forward(*c)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
