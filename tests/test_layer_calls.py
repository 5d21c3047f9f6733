"""How the operators around the recurrences are called: what the Python functions pack is what the C structs say, field by field
(no GPU needed), and the calls under the C names give what the functions give."""

import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


def at(t):
    return None if t is None else t.data_ptr()


def conv_inputs(dev="cpu"):
    """[B,H,T,d] as a slice of a projection: no two strides alike."""
    x = torch.randn(2, 5, 80).to(dev)[:, :, 16:64].unflatten(2, (3, 16)).transpose(1, 2)
    return dict(x=x, w=torch.randn(48, 4).to(dev), bias=torch.randn(48).to(dev), S0=torch.randn(2, 3, 48).to(dev))


def scan_inputs(dev="cpu"):
    B, T, D, N, G = 2, 20, 48, 8, 2
    rows = lambda wide, n, o=0: torch.randn(B, T, wide).to(BF).to(dev)[:, :, o:o + n]  # noqa: E731
    return dict(x=rows(48, D), dt=rows(56, D), A=-torch.rand(D, N).to(dev), B=rows(64, G * N, 16).unflatten(2, (G, N)),
                C=rows(72, G * N, 32).unflatten(2, (G, N)), D=torch.randn(D).to(dev), z=rows(80, D, 24),
                dt_bias=torch.randn(D).to(dev), S0=torch.randn(B, D, N).to(dev))


def gate_inputs(dev="cpu"):
    x = torch.randn(2, 3, 5, 64).to(BF).to(dev)[..., :48]
    gate = torch.randn(2, 5, 160).to(BF).to(dev)[:, :, 16:].unflatten(2, (3, 48)).transpose(1, 2)
    return dict(x=x, gate=gate, w=torch.randn(48).to(dev))


def residual_inputs(dev="cpu"):
    return dict(x=torch.randn(6, 48).to(BF).to(dev), residual=torch.randn(6, 48).to(dev), w=torch.randn(48).to(dev),
                scale=torch.randn(48).to(dev))


def struct_of(cls, **kw):
    """A struct with these fields, tensors by their addresses."""
    p = cls()
    for n, v in kw.items():
        setattr(p, n, at(v) if isinstance(v, torch.Tensor) else type(getattr(p, n))(*v) if isinstance(v, tuple) else v)
    return p


def conv_struct(x, w, bias, S0):
    return struct_of(bnd.gla_conv_params, x=x, x_stride=x.stride()[:3], w=w, bias=bias, S0=S0, B=2, H=3, T=5, d=16, W=4,
                     activation=gla.GLA_ACT_SILU, dtype=gla.GLA_FP32)


def scan_struct(x, dt, A, B, C, D, z, dt_bias, S0):
    return struct_of(bnd.gla_ssm_params, x=x, dt=dt, z=z, Bm=B, Cm=C, x_stride=x.stride()[:2], dt_stride=dt.stride()[:2],
                     z_stride=z.stride()[:2], B_stride=B.stride()[:2], C_stride=C.stride()[:2], A=A, D_skip=D, dt_bias=dt_bias,
                     S0=S0, B=2, T=20, D=48, G=2, N=8, softplus=1, dtype=gla.GLA_BF16, force_segments=0)


def gate_struct(x, gate, w):
    return struct_of(bnd.gla_norm_gate_params, x=x, gate=gate, x_stride=x.stride()[:3], gate_stride=gate.stride()[:3], w=w, B=2,
                     H=3, T=5, d=48, norm=gla.GLA_NORM_L2, activation=gla.GLA_ACT_SIGMOID, gate_first=1, eps=0.25,
                     dtype=gla.GLA_BF16)


def residual_struct(x, residual, w, scale, alpha=1.0):
    return struct_of(bnd.gla_residual_params, x=x, residual=residual, w=w, scale=scale, alpha=alpha, rows=6, D=48, post_norm=1, eps=0.5,
                     dtype=gla.GLA_BF16, residual_dtype=gla.GLA_FP32)


# ---------------------------------------------------------------- packed as the structs say, no GPU needed

@pytest.fixture
def calls(monkeypatch):
    """The library calls that the functions make: (name, their arguments but the stream)."""
    made = []
    monkeypatch.setattr(bnd, "_on_gpu", lambda t, what: None)
    monkeypatch.setattr(bnd, "_workspace", lambda name, packed, device: (None, 64, 128))
    monkeypatch.setattr(bnd, "_call", lambda name, device, stream, tensors, *args: made.append((name, args)))
    return made


def same(packed, want):
    got = type(want).from_buffer_copy(packed)
    assert len(packed) == len(bytes(want))
    for n, *_ in want._fields_:
        a, b = getattr(got, n), getattr(want, n)
        assert (list(a) == list(b) if hasattr(a, "_length_") else a == b), f"{n}: {a} is not {b}"


def test_conv_packs_its_structs(calls):
    t = conv_inputs()
    p = conv_struct(**t)
    assert len({*p.x_stride}) == 3
    y, ST = gla.causal_conv_forward(**t)
    dy, dST = torch.randn(2, 3, 5, 16), torch.randn(2, 3, 48)
    g = gla.causal_conv_backward(**t, dy=dy, dST=dST)
    (f, (packed, *out)), (b, (packed2, grads, *ws)) = calls
    assert (f, b) == ("gla_conv_fwd", "gla_conv_bwd") and out == [at(y), at(ST)] and ws == [64, 128]
    same(packed, p)
    same(packed2, p)
    same(grads, struct_of(bnd.gla_conv_grads, grad_y=dy, grad_ST=dST, grad_x=g[0], x_stride=g[0].stride()[:3], grad_w=g[1],
                          grad_bias=g[2], grad_S0=g[3]))


def test_scan_packs_its_structs(calls):
    t = scan_inputs()
    p = scan_struct(**t)
    assert len({t[n].stride(1) for n in ("x", "dt", "z", "B", "C")}) == 5
    y, ST = gla.selective_scan_forward(**t)
    dy, dST = torch.randn(2, 20, 48).to(BF), torch.randn(2, 48, 8)
    dx, ddt, dA, dB, dC, dD, dz, db, dS0 = gla.selective_scan_backward(**t, dy=dy, dST=dST)
    (f, (packed, *out)), (b, (packed2, grads, *ws)) = calls
    assert (f, b) == ("gla_ssm_fwd", "gla_ssm_bwd") and out == [at(y), at(ST), 64, 128] and ws == [64, 128]
    same(packed, p)
    same(packed2, p)
    same(grads, struct_of(bnd.gla_ssm_grads, grad_y=dy, grad_ST=dST, grad_x=dx, grad_dt=ddt, grad_z=dz, grad_B=dB, grad_C=dC, grad_A=dA,
                          grad_D=dD, grad_dt_bias=db, grad_S0=dS0))


def test_gate_packs_its_structs(calls):
    t, kw = gate_inputs(), dict(norm="l2", eps=0.25, activation="sigmoid", gate_first=True)
    p = gate_struct(**t)
    assert list(p.x_stride) != list(p.gate_stride)
    y = gla.norm_gate_forward(**t, **kw)
    dy = torch.randn(2, 5, 3, 48).to(BF)
    dx, dg, dw = gla.norm_gate_backward(**t, dy=dy, **kw)
    (f, (packed, *out)), (b, (packed2, grads, *ws)) = calls
    assert (f, b) == ("gla_norm_gate", "gla_norm_gate_bwd") and out == [at(y)] and ws == [64, 128]
    same(packed, p)
    same(packed2, p)
    assert dx.stride() != dg.stride()
    same(grads, struct_of(bnd.gla_norm_gate_grads, grad_y=dy, grad_x=dx, grad_gate=dg, x_stride=dx.stride()[:3],
                          gate_stride=dg.stride()[:3], grad_w=dw))


def test_residual_packs_its_structs(calls):
    t, kw = residual_inputs(), dict(post_norm=True, eps=0.5)
    h, y = gla.residual_norm_forward(**t, **kw)
    dh, dy = torch.randn(6, 48), torch.randn(6, 48).to(BF)
    dx, dr, dw, ds = gla.residual_norm_backward(**t, dh=dh, dy=dy, **kw)
    gla.residual_norm_forward(**{**t, "scale": 0.75}, **kw)
    (f, (packed, *out)), (b, (packed2, grads, *ws)), (_, (packed3, *_)) = calls
    assert (f, b) == ("gla_residual_norm", "gla_residual_norm_bwd") and out == [at(h), at(y)] and ws == [64, 128]
    same(packed, residual_struct(**t))
    same(packed2, residual_struct(**t))
    same(packed3, residual_struct(**{**t, "scale": None}, alpha=0.75))
    same(grads, struct_of(bnd.gla_residual_grads, grad_h=dh, grad_y=dy, grad_x=dx, grad_residual=dr, grad_w=dw, grad_scale=ds))


def test_calls_under_the_c_names_tell_their_status():
    for call, p in ((lambda p, **k: gla.gla_conv_fwd(p, None, **k), bnd.gla_conv_params()),
                    (lambda p, **k: gla.gla_conv_bwd(p, bnd.gla_conv_grads(), **k), bnd.gla_conv_params()),
                    (lambda p, **k: gla.gla_ssm_fwd(p, None, **k), bnd.gla_ssm_params()),
                    (lambda p, **k: gla.gla_ssm_bwd(p, bnd.gla_ssm_grads(), **k), bnd.gla_ssm_params()),
                    (lambda p, **k: gla.gla_norm_gate(p, None, **k), bnd.gla_norm_gate_params()),
                    (lambda p, **k: gla.gla_norm_gate_bwd(p, bnd.gla_norm_gate_grads(), **k), bnd.gla_norm_gate_params()),
                    (lambda p, **k: gla.gla_residual_norm(p, None, None, **k), bnd.gla_residual_params()),
                    (lambda p, **k: gla.gla_residual_norm_bwd(p, bnd.gla_residual_grads(), **k), bnd.gla_residual_params())):
        assert call(p, stream=0, check=False) == bnd.GLA_ERR_INVALID_ARG
        with pytest.raises(gla.GlaError):
            call(p, stream=0)


def test_a_filter_without_taps_is_refused():
    """Its state would have minus one row."""
    with pytest.raises(gla.GlaError, match="no taps"):
        gla.causal_conv(torch.randn(1, 3, 64), torch.empty(64, 0))


# ---------------------------------------------------------------- the same results under both names

def _ws(n):
    assert n > 0
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _equal(got, want):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.gpu
def test_conv_under_its_c_name():
    t = conv_inputs("cuda")
    p, want = conv_struct(**t), gla.causal_conv_forward(**t)
    out = [torch.empty_like(a) for a in want]
    gla.gla_conv_fwd(p, *out)
    _equal(out, want)
    dy, dST = torch.randn(2, 3, 5, 16, device="cuda"), torch.randn(2, 3, 48, device="cuda")
    want = gla.causal_conv_backward(**t, dy=dy, dST=dST)
    g = [torch.empty_like(a) for a in want]
    grads = struct_of(bnd.gla_conv_grads, grad_y=dy, grad_ST=dST, grad_x=g[0], x_stride=g[0].stride()[:3], grad_w=g[1], grad_bias=g[2],
                      grad_S0=g[3])
    gla.gla_conv_bwd(p, grads, _ws(gla.gla_conv_bwd_workspace_size(p)))
    _equal(g, want)


@pytest.mark.gpu
def test_scan_under_its_c_name():
    t = scan_inputs("cuda")
    p, want = scan_struct(**t), gla.selective_scan_forward(**t, force_segments=2)
    p.force_segments = 2
    out = [torch.empty_like(a) for a in want]
    gla.gla_ssm_fwd(p, *out, _ws(gla.gla_ssm_fwd_workspace_size(p)))
    _equal(out, want)
    dy, dST = torch.randn(2, 20, 48, device="cuda").to(BF), torch.randn(2, 48, 8, device="cuda")
    want = gla.selective_scan_backward(**t, dy=dy, dST=dST, force_segments=2)
    g = [torch.empty(a.shape, dtype=a.dtype, device="cuda") for a in want]
    names = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_S0")
    grads = struct_of(bnd.gla_ssm_grads, grad_y=dy, grad_ST=dST, **dict(zip(names, g)))
    gla.gla_ssm_bwd(p, grads, _ws(gla.gla_ssm_bwd_workspace_size(p)))
    _equal(g, want)


@pytest.mark.gpu
def test_gate_under_its_c_name():
    t, kw = gate_inputs("cuda"), dict(norm="l2", eps=0.25, activation="sigmoid", gate_first=True)
    p, want = gate_struct(**t), gla.norm_gate_forward(**t, **kw)
    y = torch.empty_like(want)
    gla.gla_norm_gate(p, y)
    _equal([y], [want])
    dy = torch.randn(2, 5, 3, 48, device="cuda").to(BF)
    want = gla.norm_gate_backward(**t, dy=dy, **kw)
    g = [torch.empty_like(a) for a in want]
    grads = struct_of(bnd.gla_norm_gate_grads, grad_y=dy, grad_x=g[0], grad_gate=g[1], x_stride=g[0].stride()[:3],
                      gate_stride=g[1].stride()[:3], grad_w=g[2])
    gla.gla_norm_gate_bwd(p, grads, _ws(gla.gla_norm_gate_bwd_workspace_size(p)))
    _equal(g, want)


@pytest.mark.gpu
def test_residual_under_its_c_name():
    t, kw = residual_inputs("cuda"), dict(post_norm=True, eps=0.5)
    p, want = residual_struct(**t), gla.residual_norm_forward(**t, **kw)
    out = [torch.empty_like(a) for a in want]
    gla.gla_residual_norm(p, *out)
    _equal(out, want)
    dh, dy = torch.randn(6, 48, device="cuda"), torch.randn(6, 48, device="cuda").to(BF)
    want = gla.residual_norm_backward(**t, dh=dh, dy=dy, **kw)
    g = [torch.empty_like(a) for a in want]
    grads = struct_of(bnd.gla_residual_grads, grad_h=dh, grad_y=dy, grad_x=g[0], grad_residual=g[1], grad_w=g[2], grad_scale=g[3])
    gla.gla_residual_norm_bwd(p, grads, _ws(gla.gla_residual_norm_bwd_workspace_size(p)))
    _equal(g, want)
