"""torch.autograd glue: gated linear attention whose forward runs gla_fwd_ex and whose
backward runs gla_bwd, both through the C ABI. Argument marshalling only: every step of
both passes runs in the library's kernels.

    O, ST = gla_attention(q, k, v, log_g, S0)   # q, k, v bf16 or fp32; log_g, S0 fp32

Gradients reach q, k, v (in their dtype: the library returns fp32 gradients, cast here),
log_g and S0 (fp32), for every gate mode but the bilinear one. Nothing is kept from the
forward pass but its inputs: the backward recomputes the chunk states (gla_bwd's design).

    O, ST = delta_attention(q, k, v, log_g, beta, S0)     # the gated delta rule
    q, k = qk_norm_rope(q, k, norm="l2", inv_freq=f)      # norms of q and k, position rotation

delta_attention's backward runs gla_delta_bwd and qk_norm_rope's gla_qk_norm_rope_bwd; both
keep their inputs only. So do, each with the _bwd call of its kernel,

    y, ST = causal_conv(x, w, bias, S0)                   # the short causal convolution
    y, ST = selective_scan(x, dt, A, B, C, D, z, dt_bias, S0)
    y = norm_gate(x, gate, w)                             # the heads' norm with its gate
    h, y = residual_norm(x, residual, w, scale)           # the residual with its norm
"""
from __future__ import annotations

from . import binding as _b


def _function():
    import torch

    class GLAFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_g, S0, gate):
            O, ST = _b.forward(q, k, v, log_g, S0, gate=gate)
            ctx.gate = gate
            ctx.save_for_backward(q, k, v, log_g, S0)
            return O, ST

        @staticmethod
        def backward(ctx, dO, dST):
            q, k, v, log_g, S0 = ctx.saved_tensors
            if dO is None:
                dO = torch.zeros((q.shape[0], q.shape[1], q.shape[2], v.shape[-1]), dtype=q.dtype, device=q.device)
            dO = dO.to(q.dtype).contiguous()
            dST = None if dST is None else dST.to(torch.float32).contiguous()
            want = ctx.needs_input_grad
            dq, dk, dv, dg, dS0 = _b.backward(q, k, v, log_g, S0, dO, dST, gate=ctx.gate,
                                              want_dS0=S0 is not None and want[4])
            cast = lambda g, like, need: g.to(like.dtype) if need and g is not None else None
            return (cast(dq, q, want[0]), cast(dk, k, want[1]), cast(dv, v, want[2]),
                    cast(dg, log_g, want[3]) if log_g is not None else None,
                    cast(dS0, S0, want[4]) if S0 is not None else None, None)

    return GLAFunction


def _placed(g):
    """A gradient as the library takes it: dense and from a 16-byte boundary. What autograd hands over may be a slice of
    another tensor that starts at any element."""
    g = g.contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


def _delta_function():
    import torch

    class DeltaFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_g, beta, S0, scale, path):
            O, ST = _b.delta_forward(q, k, v, log_g, beta, S0, scale=scale, path=path)
            ctx.scale, ctx.path = scale, path
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(q, k, v, log_g, beta, S0)
            return O, ST

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dO, dST):
            q, k, v, log_g, beta, S0 = ctx.saved_tensors
            if dO is None and dST is None:
                return (None,) * 8
            dO = torch.zeros_like(v) if dO is None else _placed(dO)
            dST = None if dST is None else _placed(dST)
            want = ctx.needs_input_grad
            g = _b.delta_backward(q, k, v, log_g, beta, S0, dO, dST, scale=ctx.scale,
                                  want_dS0=S0 is not None and want[5], path=ctx.path)
            return (*(x if w else None for x, w in zip(g, want)), None, None)

    return DeltaFunction


def _qk_function():
    import torch

    class QkNormRopeFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, w_q, w_k, inv_freq, positions, norm, eps, start, interleaved):
            qo, ko = _b.qk_norm_rope_forward(q, k, norm, w_q, w_k, eps, inv_freq, positions, start, interleaved)
            ctx.how = norm, eps, start, interleaved
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(q, k, w_q, w_k, inv_freq, positions)
            return qo, ko

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dqo, dko):
            q, k, w_q, w_k, inv_freq, positions = ctx.saved_tensors
            if dqo is None and dko is None:
                return (None,) * 10
            norm, eps, start, interleaved = ctx.how
            want = ctx.needs_input_grad
            dense = lambda g, x: (torch.zeros(x.shape, dtype=x.dtype, device=x.device) if g is None
                                  else _placed(g))
            g = _b.qk_norm_rope_backward(q, k, dense(dqo, q), None if k is None else dense(dko, k), norm, w_q, w_k,
                                         eps, inv_freq, positions, start, interleaved)
            return (*(x if w else None for x, w in zip(g, want)), None, None, None, None, None, None)

    return QkNormRopeFunction


def _conv_function():
    import torch

    class CausalConvFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, S0, activation, want_state):
            y, ST = _b.causal_conv_forward(x, w, bias, S0, activation, want_state)
            ctx.activation = activation
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(x, w, bias, S0)
            return y, ST

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dST):
            x, w, bias, S0 = ctx.saved_tensors
            if dy is None and dST is None:
                return (None,) * 6
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _placed(dy)
            want = ctx.needs_input_grad
            g = _b.causal_conv_backward(x, w, bias, S0, dy, None if dST is None else _placed(dST), ctx.activation,
                                        want_dw=want[1] or want[2], want_dS0=want[3])
            return (*(x if w else None for x, w in zip(g, want)), None, None)

    return CausalConvFunction


def _scan_function():
    import torch

    class SelectiveScanFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A, B, C, D, z, dt_bias, S0, softplus, want_state):
            y, ST = _b.selective_scan_forward(x, dt, A, B, C, D, z, dt_bias, S0, softplus, want_state)
            ctx.softplus = softplus
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, S0)
            return y, ST

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dST):
            t = ctx.saved_tensors
            if dy is None and dST is None:
                return (None,) * 11
            x = t[0]
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _placed(dy)
            want = ctx.needs_input_grad
            g = _b.selective_scan_backward(*t, dy, None if dST is None else _placed(dST), ctx.softplus, want_dS0=want[8])
            return (*(x if w else None for x, w in zip(g, want)), None, None)

    return SelectiveScanFunction


def _gate_function():
    import torch

    class NormGateFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, w, norm, eps, activation, gate_first):
            ctx.how = norm, eps, activation, gate_first
            ctx.save_for_backward(x, gate, w)
            return _b.norm_gate_forward(x, gate, w, norm, eps, activation, gate_first)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, gate, w = ctx.saved_tensors
            g = _b.norm_gate_backward(x, gate, w, _placed(dy), *ctx.how)
            return (*(x if w else None for x, w in zip(g, ctx.needs_input_grad)), None, None, None, None)

    return NormGateFunction


def _residual_function():
    import torch

    class ResidualNormFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, w, scale, post_norm, eps):
            ctx.number = None if isinstance(scale, torch.Tensor) else scale
            ctx.how = post_norm, eps
            ctx.set_materialize_grads(False)
            ctx.save_for_backward(x, residual, w, scale if ctx.number is None else None)
            return _b.residual_norm_forward(x, residual, w, scale, post_norm, eps)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dh, dy):
            x, residual, w, scale = ctx.saved_tensors
            if dh is None and dy is None:
                return (None,) * 6
            placed = lambda g: None if g is None else _placed(g)  # noqa: E731
            want = ctx.needs_input_grad
            g = _b.residual_norm_backward(x, residual, w, scale if ctx.number is None else ctx.number, placed(dh),
                                          placed(dy), *ctx.how, want_dx=want[0], want_dres=want[1])
            return (*(x if w else None for x, w in zip(g, want)), None, None)

    return ResidualNormFunction


def _plain(*tensors):
    """Whether no derivative of any kind is asked of these inputs (some may be None). A dual tensor of forward
    mode need not require grad, and no_grad() does not switch forward mode off: with a dual level open the
    autograd function is called, which refuses what it has no derivative for."""
    import torch
    if torch.autograd.forward_ad._current_level >= 0:
        return False
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return False
    return True


_FN = None
_DELTA = None
_QK = None
_CONV = None
_SCAN = None
_GATE = None
_RESIDUAL = None


def gla_attention(q, k, v, log_g=None, S0=None, gate=None):
    """(O, S_T) of the forward pass, differentiable in q, k, v, log_g and S0. Shapes and gate
    modes as for binding.forward; the inputs must be contiguous device tensors."""
    global _FN
    if _FN is None:
        _FN = _function()
    return _FN.apply(q, k, v, log_g, S0, gate)


def delta_attention(q, k, v, log_g, beta, S0=None, scale=None, path=_b.GLA_PATH_AUTO):
    """(O, S_T) of the gated delta rule (binding.delta_forward), differentiable once in q, k, v, log_g, beta
    and S0, in reverse mode (forward mode is refused). The inputs must be contiguous device tensors. A step captured into a CUDA graph starts from
    leaves of which no eager graph is alive (fresh detached ones, say): autograd would wait on the stream
    of that graph, which a capture cannot."""
    if _plain(q, k, v, log_g, beta, S0):
        return _b.delta_forward(q, k, v, log_g, beta, S0, scale=scale, path=path)
    global _DELTA
    if _DELTA is None:
        _DELTA = _delta_function()
    return _DELTA.apply(q, k, v, log_g, beta, S0, scale, path)


def qk_norm_rope(q, k=None, norm="l2", w_q=None, w_k=None, eps=1e-6, inv_freq=None, positions=None, start=0,
                 interleaved=False):
    """binding.qk_norm_rope_forward, differentiable once in q, k and the weights, in reverse mode."""
    if _plain(q, k, w_q, w_k):
        return _b.qk_norm_rope_forward(q, k, norm, w_q, w_k, eps, inv_freq, positions, start, interleaved)
    global _QK
    if _QK is None:
        _QK = _qk_function()
    return _QK.apply(q, k, w_q, w_k, inv_freq, positions, norm, eps, start, interleaved)


def causal_conv(x, w, bias=None, S0=None, activation="silu", want_state=True):
    """(y, ST) of the short causal convolution (binding.causal_conv_forward), differentiable once in x, w, bias and S0, in
    reverse mode."""
    if _plain(x, w, bias, S0):
        return _b.causal_conv_forward(x, w, bias, S0, activation, want_state)
    global _CONV
    if _CONV is None:
        _CONV = _conv_function()
    return _CONV.apply(x, w, bias, S0, activation, want_state)


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, S0=None, softplus=True, want_state=True):
    """(y, ST) of the selective scan (binding.selective_scan_forward), differentiable once in every tensor, in reverse
    mode. What delta_attention says of captured steps holds here too, and for the other functions of this module."""
    if _plain(x, dt, A, B, C, D, z, dt_bias, S0):
        return _b.selective_scan_forward(x, dt, A, B, C, D, z, dt_bias, S0, softplus, want_state)
    global _SCAN
    if _SCAN is None:
        _SCAN = _scan_function()
    return _SCAN.apply(x, dt, A, B, C, D, z, dt_bias, S0, softplus, want_state)


def norm_gate(x, gate=None, w=None, norm="rms", eps=1e-6, activation="silu", gate_first=False):
    """binding.norm_gate_forward, differentiable once in x, gate and w, in reverse mode."""
    if _plain(x, gate, w):
        return _b.norm_gate_forward(x, gate, w, norm, eps, activation, gate_first)
    global _GATE
    if _GATE is None:
        _GATE = _gate_function()
    return _GATE.apply(x, gate, w, norm, eps, activation, gate_first)


def residual_norm(x, residual=None, w=None, scale=None, post_norm=False, eps=1e-6):
    """(h, y) of binding.residual_norm_forward, differentiable once in x, residual, w and a scale that is a tensor, in
    reverse mode."""
    if _plain(x, residual, w, scale if hasattr(scale, "requires_grad") else None):
        return _b.residual_norm_forward(x, residual, w, scale, post_norm, eps)
    global _RESIDUAL
    if _RESIDUAL is None:
        _RESIDUAL = _residual_function()
    return _RESIDUAL.apply(x, residual, w, scale, post_norm, eps)
