"""The gated delta rule and the query/key norms in fp64 on the CPU, token by token and value by
value from their definitions, differentiable by autograd."""
import math

import torch


def delta(q, k, v, log_g, beta, S0, scale):
    """(O, S_T) of the recurrence; q, k [B,Hk,T,dk], v [B,H,T,dv]; everything in fp64."""
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    q, k = q.repeat_interleave(H // Hk, 1), k.repeat_interleave(H // Hk, 1)
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64) if S0 is None else S0
    o = []
    for t in range(T):
        Sd = S if log_g is None else S * log_g[:, :, t, None, None].exp()
        kt = k[:, :, t].unsqueeze(3)
        u = beta[:, :, t, None] * (v[:, :, t] - (kt * Sd).sum(2))
        S = Sd + kt * u.unsqueeze(2)
        o.append(scale * (q[:, :, t].unsqueeze(3) * S).sum(2))
    return torch.stack(o, 2) if o else torch.zeros(B, H, 0, dv, dtype=torch.float64), S


def make(B, H, Hk, T, dk, dv, dtype, seed=0, gate="sigmoid", s0=True, keys="unit", beta="sigmoid"):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    q, k, v = unit(rnd(B, Hk, T, dk)), unit(rnd(B, Hk, T, dk)), rnd(B, H, T, dv)
    if keys == "same":            # every token writes to one key: the triangular system is full
        k = k[:, :, :1].expand(B, Hk, T, dk).contiguous()
    b = torch.sigmoid(rnd(B, H, T))
    if beta == "one":
        b = torch.ones(B, H, T)
    if beta == "holes":           # tokens that must leave the state alone
        b = b * (torch.rand(B, H, T, generator=g) < 0.5)
    lg = torch.nn.functional.logsigmoid(rnd(B, H, T)) / 16
    if gate == "none":
        lg = None
    elif gate == "steep":
        lg = -8 * torch.rand(B, H, T, generator=g)
    elif gate == "resets":        # exp(log_g) = 0 now and then
        lg = torch.where(torch.rand(B, H, T, generator=g) < 0.05, torch.tensor(-math.inf), lg)
    S0 = rnd(B, H, dk, dv) * 0.3 if s0 else None
    x = [q.to(dtype), k.to(dtype), v.to(dtype), lg, b.to(dtype), S0]
    return x, g


def f64(xs):
    return [None if x is None else x.double() for x in xs]


def cuda(xs):
    return [None if x is None else x.cuda() for x in xs]


def norm_rope(x, norm, w, eps, inv_freq, positions, interleaved):
    """One of q, k in fp64: [B,H,T,d]."""
    d = x.shape[-1]
    if norm is not None:
        x = x / (x.square().sum(-1, keepdim=True) / (d if norm == "rms" else 1) + eps).sqrt()
    if w is not None:
        x = x * w
    if inv_freq is None:
        return x
    th = positions[:, None, :, None].double() * inv_freq
    r = 2 * inv_freq.numel()
    out = list(x.unbind(-1))
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = th[..., i].cos(), th[..., i].sin()
        out[a], out[b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return torch.stack(out, -1)
