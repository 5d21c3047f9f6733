"""The operators around the recurrences together, as a layer uses them: a gated delta net's block (residual norm, projection,
short convolutions, unit queries and keys, delta rule, gated norm, projection, residual norm), a selective-scan block, both with
gradients against fp64, decoded token by token, captured into CUDA graphs, and on other streams."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import autograd as glue
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _delta_ref as dref
import _layer_ref as ref


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def weights(shapes, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return {n: (torch.randn(s, generator=g) * (s[-1] ** -0.5 if len(s) > 1 else 0.1) + (1 if n.startswith("norm") else 0)).to(
        dtype if n.startswith("proj") else torch.float32) for n, s in shapes.items()}


H, DH, M = 4, 64, 128                            # heads, head width, model width
DELTA = dict(norm_in=(M,), proj_qkv=(3 * H * DH, M), proj_g=(H * DH, M), proj_ab=(2 * H, M), conv_q=(H * DH, 4), conv_k=(H * DH, 4),
             conv_v=(H * DH, 4), norm_o=(DH,), proj_o=(M, H * DH), norm_out=(M,))


def delta_block(w, x, r, lib, states=None):
    """One block over x [B,T,M] with residual r: (residual, normed). lib: the kernels, or their fp64 definitions."""
    B, T, _ = x.shape
    r, a = lib.residual(x, r, w["norm_in"])
    qkv, gate, ab = (lib.out(a @ w[n].t()) for n in ("proj_qkv", "proj_g", "proj_ab"))
    heads = lambda t: t.unflatten(2, (H, DH)).transpose(1, 2)  # noqa: E731
    new, c = [], []
    for i, n in enumerate(("conv_q", "conv_k", "conv_v")):
        y, s = lib.conv(heads(qkv[:, :, i * H * DH:(i + 1) * H * DH]), w[n], states[i] if states else None)
        c.append(y)
        new.append(s)
    ab = ab.transpose(1, 2).contiguous()
    q, k = lib.qk(c[0], c[1])
    o, s = lib.delta(q, k, c[2].contiguous(), torch.nn.functional.logsigmoid(ab[:, :H].to(lib.wide)) / 4,
                     lib.out(torch.sigmoid(ab[:, H:]).contiguous()), states[3] if states else None)
    new.append(s)
    y = lib.out(lib.gate(o, heads(gate), w["norm_o"]).flatten(2) @ w["proj_o"].t())
    return (*lib.residual(y, r, w["norm_out"]), new)


class Kernels:
    wide = torch.float32
    out = staticmethod(lambda t: t)
    residual = staticmethod(lambda *a: gla.residual_norm(*a))
    conv = staticmethod(lambda x, w, s, b=None: gla.causal_conv(x, w, b, s))
    qk = staticmethod(lambda q, k: gla.qk_norm_rope(q, k))
    delta = staticmethod(lambda q, k, v, g, b, s: gla.delta_attention(q, k, v, g.contiguous(), b, s))
    gate = staticmethod(lambda o, g, w: gla.norm_gate(o, g, w))
    scan = staticmethod(lambda *a: gla.selective_scan(*a)[0])


class Plain:
    """The definitions; `out` is what becomes of each operator's and product's result."""
    wide = torch.float64
    out = staticmethod(lambda t: t)

    @classmethod
    def residual(cls, x, r, w, scale=None, post=False):
        return tuple(cls.out(t) for t in ref.residual(x, r, w, scale, post, 1e-6))

    @classmethod
    def conv(cls, x, w, s, b=None):
        heads = x.dim() == 4
        y, s = ref.conv(x.transpose(1, 2).flatten(2) if heads else x, w, b, s, "silu")
        return cls.out(y.unflatten(2, x.shape[1::2]).transpose(1, 2) if heads else y), s

    @classmethod
    def qk(cls, *rows):
        return [cls.out(dref.norm_rope(t, "l2", None, 1e-6, None, None, False)) for t in rows]

    @classmethod
    def delta(cls, q, k, v, g, b, s):
        o, s = dref.delta(q, k, v, g, b, s, DH ** -0.5)
        return cls.out(o), s

    @classmethod
    def gate(cls, o, g, w):
        return cls.out(ref.gate(o, g, w, "rms", 1e-6, "silu", False))

    @classmethod
    def scan(cls, *a):
        return cls.out(ref.scan(*a, None, True)[0])


class _Round(torch.autograd.Function):
    @staticmethod
    def forward(ctx, t):
        return t.bfloat16().double()

    @staticmethod
    def backward(ctx, g):
        return g.bfloat16().double()


class Rounded(Plain):
    """The definitions with each result, and its gradient, rounded to bf16, as every bf16 run must."""
    out = staticmethod(_Round.apply)


def against_fp64(block, shapes, T, dtype, seed):
    """The block's results and gradients against fp64. fp32: 1e-4 (the delta rule's own 1e-5, the projections', and those
    meeting again). bf16: what the roundings of the results between the operators alone do to each output differs from
    output to output (sums of cancelling terms grow them); it is what the rounded definitions are off by, and roundings that
    fall differently are off by as much again: twice that, and the last rounding."""
    w, g = weights(shapes, seed, dtype), torch.Generator().manual_seed(seed + 1)
    x, r, dy = (torch.randn(2, T, M, generator=g).to(dtype) for _ in range(3))
    torch.backends.cuda.matmul.allow_tf32 = False

    def run(lib, place):
        leaves = [place(t).requires_grad_(True) for t in (x, r, *w.values())]
        h, y = block(dict(zip(w, leaves[2:])), *leaves[:2], lib)[:2]
        return (h, y, *torch.autograd.grad((h, y), leaves, (place(dy), place(dy))))

    got, want = run(Kernels, lambda t: t.cuda()), run(Plain, lambda t: t.double())
    off = [1e-4] * len(got)
    if dtype == torch.bfloat16:
        off = [2 * rel(a, b) + 2.0 ** -8 for a, b in zip(run(Rounded, lambda t: t.double()), want)]
    for n, a, b, tol in zip(("h", "y", "dx", "dr", *("d" + n for n in w)), got, want, off):
        assert rel(a, b) <= tol, f"{n}: {rel(a, b):.1e} of {tol:.1e}"


def rel(a, b):
    return float((a.detach().double().cpu() - b.detach()).norm() / b.detach().norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_delta_block_against_fp64(dtype):
    against_fp64(delta_block, DELTA, 70, dtype, 1)


@pytest.mark.gpu
def test_delta_block_decodes_as_it_prefills():
    w = {n: t.cuda() for n, t in weights(DELTA, 3, torch.float32).items()}
    g = torch.Generator().manual_seed(4)
    x, r = (torch.randn(2, 12, M, generator=g).cuda() for _ in range(2))
    torch.backends.cuda.matmul.allow_tf32 = False
    h, y, last = delta_block(w, x, r, Kernels)
    state = [torch.zeros(2, 3, H * DH, device="cuda") for _ in range(3)] + [torch.zeros(2, H, DH, DH, device="cuda")]
    out = []
    for t in range(12):
        a, b, state = delta_block(w, x[:, t:t + 1].contiguous(), r[:, t:t + 1].contiguous(), Kernels, state)
        out.append(b)
    assert torch.allclose(torch.cat(out, 1), y, atol=1e-4)
    for a, b in zip(state, last):
        assert torch.allclose(a, b, atol=1e-4)


RANK, N, D2 = 16, 16, 256
SCAN = dict(norm_in=(M,), proj_in=(2 * D2, M), conv=(D2, 4), bias_conv=(D2,), proj_low=(RANK + 2 * N, D2), proj_dt=(D2, RANK),
            bias_dt=(D2,), A_log=(D2, N), skip=(D2,), proj_o=(M, D2), norm_out=(M,))


def scan_block(w, x, r, lib):
    r, a = lib.residual(x, r, w["norm_in"])
    xz = lib.out(a @ w["proj_in"].t())
    u, _ = lib.conv(xz[:, :, :D2], w["conv"], None, w["bias_conv"])
    low = lib.out(u @ w["proj_low"].t())
    B, C = (low[:, :, RANK + i * N:RANK + (i + 1) * N].unflatten(2, (1, N)) for i in (0, 1))
    dt = lib.out(low[:, :, :RANK] @ w["proj_dt"].t())
    y = lib.scan(u, dt, -torch.exp(w["A_log"] + 1), B, C, w["skip"], xz[:, :, D2:], w["bias_dt"])
    return lib.residual(lib.out(y @ w["proj_o"].t()), r, w["norm_out"], 0.5, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scan_block_against_fp64(dtype):
    against_fp64(scan_block, SCAN, 50, dtype, 5)


def _scan_inputs(T, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    return dict(x=rnd(2, T, 64), dt=rnd(2, T, 64) - 2, A=-1 - rnd(64, 16).abs(), B=rnd(2, T, 1, 16), C=rnd(2, T, 1, 16), D=rnd(64),
                z=rnd(2, T, 64), dt_bias=rnd(64) * 0.1, S0=rnd(2, 64, 16))


def _all(t, w, x4):
    """Every operator once, forward."""
    y, ST = gla.selective_scan(**t)
    c, cs = gla.causal_conv(t["x"], w)
    return (y, ST, c, cs, gla.norm_gate(x4, x4), *gla.residual_norm(t["x"], t["z"], t["dt_bias"]))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 300])
def test_replays_from_a_cuda_graph(T):
    t, w, x4 = _scan_inputs(T, 7), torch.randn(64, 4, device="cuda"), torch.randn(2, 2, T, 64, device="cuda")
    _all(t, w, x4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all(t, w, x4)
    for a in (*t.values(), w, x4):
        a.mul_(0.75)
    want = _all(t, w, x4)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_training_step_replays_from_a_cuda_graph():
    def step(t, w, x4):
        leaves = [a.detach().requires_grad_(True) for a in (*t.values(), w, x4)]
        out = _all(dict(zip(t, leaves)), leaves[-2], leaves[-1])
        return torch.autograd.grad(out, leaves, [torch.ones_like(o) for o in out])
    t, w, x4 = _scan_inputs(200, 8), torch.randn(64, 4, device="cuda"), torch.randn(2, 2, 200, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(t, w, x4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(t, w, x4)
    for a in (*t.values(), w, x4):
        a.mul_(0.75)
    want = step(t, w, x4)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_other_streams_and_two_at_once():
    t, w, x4 = _scan_inputs(500, 9), torch.randn(64, 4, device="cuda"), torch.randn(2, 2, 500, 64, device="cuda")
    want = _all(t, w, x4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for s in streams * 3:
        y, ST = gla.selective_scan_forward(**t, stream=s)
        c, cs = gla.causal_conv_forward(t["x"], w, stream=s)
        got.append((y, ST, c, cs, gla.norm_gate_forward(x4, x4, stream=s.cuda_stream), *gla.residual_norm_forward(t["x"], t["z"], t["dt_bias"], stream=s)))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_rows_beyond_32_bits():
    """Rows 2^30 values apart in one tensor of 2^33 bytes: offsets pass 2^31 elements and 2^32 bytes."""
    T, far = 4, 1 << 30
    store = torch.empty(T * far, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(11)
    rows = torch.randn(T, 256, generator=g).bfloat16().cuda()
    wide = store.as_strided((T, 256), (far, 1))
    wide.copy_(rows)
    x, near = wide.unsqueeze(0), rows.unsqueeze(0)
    w = torch.randn(256, 4, generator=g).cuda()
    dy = torch.randn(1, T, 256, generator=g).bfloat16().cuda()
    for a, b in ((gla.causal_conv(x, w), gla.causal_conv(near, w)),
                 (gla.causal_conv_backward(x, w, None, None, dy), gla.causal_conv_backward(near, w, None, None, dy))):
        assert all(p is q or torch.equal(p, q) for p, q in zip(a, b))
    heads = lambda t: t.unflatten(2, (2, 128)).transpose(1, 2)  # noqa: E731
    dg = dy.unflatten(2, (2, 128)).contiguous()
    assert torch.equal(gla.norm_gate(heads(x), heads(x)), gla.norm_gate(heads(near), heads(near)))
    for p, q in zip(gla.norm_gate_backward(heads(x), heads(x), None, dg), gla.norm_gate_backward(heads(near), heads(near), None, dg)):
        assert p is q or torch.equal(p, q)
    A, S0 = -torch.rand(64, 16, generator=g).cuda(), torch.randn(1, 64, 16, generator=g).cuda()
    cut = lambda t: (t[..., :64], t[..., 64:128], A, t[..., 128:144].unflatten(2, (1, 16)), t[..., 144:160].unflatten(2, (1, 16)), None,  # noqa: E731
                     t[..., 160:224], None, S0)
    for kw in ({}, {"force_segments": 1}):
        assert all(torch.equal(p, q) for p, q in zip(gla.selective_scan_forward(*cut(x), **kw), gla.selective_scan_forward(*cut(near), **kw)))
    d = dy[..., :64].contiguous()
    for p, q in zip(gla.selective_scan_backward(*cut(x), d), gla.selective_scan_backward(*cut(near), d)):
        assert p is q or torch.equal(p, q)


@pytest.mark.gpu
def test_long_tensors_pass_32_bits():
    """2^31 + values in one dense tensor: the last rows against the same rows alone."""
    g = torch.Generator(device="cuda").manual_seed(12)
    T, D = (1 << 20) + 40, 2048
    x = torch.randn(64, D, generator=g, device="cuda").bfloat16().repeat((T + 63) // 64, 1)[:T]
    w, tail = torch.randn(D, 4, generator=g, device="cuda"), slice(T - 70, T)
    y, ST = gla.causal_conv(x.unsqueeze(0), w)
    y2, ST2 = gla.causal_conv(x[tail].unsqueeze(0), w, S0=x[T - 73:T - 70].unsqueeze(0).contiguous())
    assert torch.equal(y[0, tail], y2[0]) and torch.equal(ST, ST2)
    del y, y2
    h, n = gla.residual_norm(x, x, w[:, 0].contiguous())
    h2, n2 = gla.residual_norm(x[tail].contiguous(), x[tail].contiguous(), w[:, 0].contiguous())
    assert torch.equal(h[tail], h2) and torch.equal(n[tail], n2)
    del h, n
    v = x.unflatten(1, (16, 128)).transpose(0, 1).unsqueeze(0)
    y = gla.norm_gate(v, v)
    assert torch.equal(y[0, tail], gla.norm_gate(v[:, :, tail], v[:, :, tail])[0])
    del y
    # a step of a decay that forgets: the last tokens of a long scan are those of a short one
    args = lambda t: (t, t, torch.full((D, 8), -8.0, device="cuda"), t[..., :8].unsqueeze(2), t[..., 8:16].unsqueeze(2))  # noqa: E731
    y, S = gla.selective_scan(*args(x.unsqueeze(0)))
    y2, S2 = gla.selective_scan(*args(x[T - 320:].unsqueeze(0)))
    assert torch.allclose(S, S2, rtol=1e-4, atol=1e-4) and torch.allclose(y[0, tail].float(), y2[0, -70:].float(), rtol=2.0 ** -7, atol=1e-3)


@pytest.mark.gpu
def test_gradients_of_broadcast_inputs():
    """B and C of one row for the whole batch, a gate and a convolved row shared by all tokens: their gradients are the sums."""
    t, w, x4 = _scan_inputs(40, 10), torch.randn(64, 4, device="cuda"), torch.randn(2, 2, 40, 64, device="cuda")
    one = {n: t[n][:1].detach().requires_grad_(True) for n in ("B", "C")}
    full = {n: a.detach().expand(2, -1, -1, -1).contiguous().requires_grad_(True) for n, a in one.items()}
    dy = torch.randn(2, 40, 64, device="cuda")
    a = torch.autograd.grad(gla.selective_scan(**{**t, **{n: b.expand(2, -1, -1, -1) for n, b in one.items()}})[0], list(one.values()), dy)
    b = torch.autograd.grad(gla.selective_scan(**{**t, **full})[0], list(full.values()), dy)
    for p, q in zip(a, b):
        assert torch.allclose(p, q.sum(0, keepdim=True), rtol=1e-5, atol=1e-5)
    g1 = torch.randn(2, 2, 1, 64, device="cuda", requires_grad=True)
    g2 = g1.detach().expand(2, 2, 40, 64).contiguous().requires_grad_(True)
    do = torch.randn(2, 40, 2, 64, device="cuda")
    p, = torch.autograd.grad(gla.norm_gate(x4, g1.expand(2, 2, 40, 64)), g1, do)
    q, = torch.autograd.grad(gla.norm_gate(x4, g2), g2, do)
    assert torch.allclose(p, q.sum(2, keepdim=True), rtol=1e-5, atol=1e-4)


# ---------------------------------------------------------------- no GPU needed

def test_given_outputs_that_require_grad_are_refused():
    x, w = torch.randn(1, 3, 64), torch.randn(64, 4)
    A, b = -torch.rand(64, 16), torch.randn(1, 3, 1, 16)
    out = torch.empty(1, 3, 64, requires_grad=True)
    for call in (lambda: gla.residual_norm_forward(x, x, h=out), lambda: gla.causal_conv_forward(x, w, y=out),
                 lambda: gla.selective_scan_forward(x, x, A, b, b, y=out)):
        with pytest.raises(gla.GlaError):
            call()


@pytest.fixture
def _stand_ins(monkeypatch):
    b = glue._b
    monkeypatch.setattr(b, "causal_conv_forward", lambda x, w, *a: (x * 2, None))
    monkeypatch.setattr(b, "selective_scan_forward", lambda x, *a: (x * 2, None))
    monkeypatch.setattr(b, "norm_gate_forward", lambda x, *a: x * 2)
    monkeypatch.setattr(b, "residual_norm_forward", lambda x, *a: (x * 2, x * 3))


CALLS = {
    "conv": (gla.causal_conv, 4), "scan": (gla.selective_scan, 9), "gate": (gla.norm_gate, 3), "residual": (gla.residual_norm, 4),
}


@pytest.mark.parametrize("name,at", [(n, i) for n, (_, k) in CALLS.items() for i in range(k)])
def test_forward_mode_is_refused(name, at, _stand_ins):
    call, k = CALLS[name]
    x = [torch.randn(2, 3, 16) for _ in range(k)]
    with fwd.dual_level():
        x[at] = fwd.make_dual(x[at], torch.ones_like(x[at]))
        with pytest.raises((RuntimeError, NotImplementedError), match="(?i)forward|jvp"):
            call(*x)


@pytest.mark.parametrize("name", CALLS)
def test_plain_calls_take_no_graph(name, _stand_ins):
    call, k = CALLS[name]
    x = [torch.randn(2, 3, 16) for _ in range(k)]
    first = lambda r: r[0] if isinstance(r, tuple) else r  # noqa: E731
    assert not first(call(*x)).requires_grad
    x[0].requires_grad_(True)
    assert first(call(*x)).requires_grad
    with torch.no_grad():
        assert not first(call(*x)).requires_grad


@pytest.mark.parametrize("name", CALLS)
def test_second_derivatives_are_refused(name, _stand_ins, monkeypatch):
    b = glue._b
    monkeypatch.setattr(b, "causal_conv_backward", lambda x, w, bias, S0, dy, *a, **k: (dy * 2, None, None, None))
    monkeypatch.setattr(b, "selective_scan_backward", lambda *a, **k: (a[9] * 2, *(None,) * 8))
    monkeypatch.setattr(b, "norm_gate_backward", lambda x, gate, w, dy, *a: (dy * 2, None, None))
    monkeypatch.setattr(b, "residual_norm_backward", lambda x, r, w, s, dh, dy, *a, **k: (dh * 2, None, None, None))
    call, k = CALLS[name]
    x = [torch.randn(2, 3, 16) for _ in range(k)]
    x[0].requires_grad_(True)
    first = lambda r: r[0] if isinstance(r, tuple) else r  # noqa: E731
    (g,) = torch.autograd.grad(first(call(*x)).square().sum(), x[:1])
    assert not g.requires_grad and torch.equal(g, 8 * x[0])
    (g,) = torch.autograd.grad(first(call(*x)).square().sum(), x[:1], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()
