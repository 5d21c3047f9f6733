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
keep their inputs only.
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
