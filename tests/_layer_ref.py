"""The short convolution, the selective scan, the gated norm and the residual norm in fp64 on the CPU, from their
definitions token by token, differentiable by autograd; and how far a result may be from them."""
import torch


def silu(a):
    return a / (1 + torch.exp(-a))


def conv(x, w, bias, S0, act):
    """x [B,T,D] (y, ST)."""
    B, T, D = x.shape
    W = w.shape[1]
    rows = torch.cat((torch.zeros(B, W - 1, D, dtype=x.dtype) if S0 is None else S0, x), 1)
    y = []
    for t in range(T):
        a = (rows[:, t:t + W] * w.t()).sum(1)
        y.append(a if bias is None else a + bias)
    y = torch.stack(y, 1) if y else x
    return silu(y) if act == "silu" else y, rows[:, T:]


def scan(x, dt, A, B, C, D, z, dt_bias, S0, softplus):
    """(y, ST) of the recurrence; x [B,T,D], B, C [B,T,G,N]."""
    nb, T, nd = x.shape
    G, N = B.shape[2:]
    v = dt if dt_bias is None else dt + dt_bias
    delta = torch.logaddexp(v, torch.zeros_like(v)) if softplus else v
    h = torch.zeros(nb, nd, N, dtype=x.dtype) if S0 is None else S0
    y = []
    for t in range(T):
        d = delta[:, t, :, None]
        h = torch.exp(d * A) * h + d * x[:, t, :, None] * B[:, t].repeat_interleave(nd // G, 1)
        y.append((h * C[:, t].repeat_interleave(nd // G, 1)).sum(2))
    y = torch.stack(y, 1) if y else x
    if D is not None:
        y = y + D * x
    return (y if z is None else y * silu(z)), h


def norm(x, how, eps):
    if how is None:
        return x
    return x / (x.square().sum(-1, keepdim=True) / (x.shape[-1] if how == "rms" else 1) + eps).sqrt()


def gate(x, g, w, how, eps, act, first):
    a = 1 if g is None else silu(g) if act == "silu" else 1 / (1 + torch.exp(-g))
    y = norm(x * a, how, eps) if first else norm(x, how, eps)
    if w is not None:
        y = y * w
    return (y if first else y * a).transpose(1, 2)


def residual(x, r, w, scale, post, eps):
    u = norm(x, "rms", eps) if post else x
    h = u if scale is None else u * scale
    if r is not None:
        h = h + r
    y = norm(h, "rms", eps)
    return h, y if w is None else y * w


def double(ts, grad=True):
    return [None if t is None else t.detach().double().cpu().requires_grad_(grad) for t in ts]


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def near(got, want, what, slack=2e-5):
    """One rounding to the result's type (bf16: 2^-8 of the value) and `slack` of the tensor's root mean square for the
    fp32 arithmetic before it: 30 roundings of 2^-24 of terms up to ten times that."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    got, want = got.detach().double().cpu(), want.detach().double()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)}"
    assert torch.isfinite(got).all(), f"{what} is not finite"
    if want.numel():
        tol = half * want.abs() + slack * want.square().mean().sqrt()
        worst = float(((got - want).abs() / (tol + 1e-30)).max())
        assert worst <= 1, f"{what}: {worst:.2f} of its bound"


def along(f, args, grads, seed=0, step=2.0 ** -7):
    """Each gradient of the scalar f(*args) (fp32 tensors) along a random direction against the difference of f's own values a step
    either way: off by the step's square times the third derivative (6e-5 of values of order one) and by the results' 2^-24
    over the step (1e-5 of the terms); held to 2e-2 of the root of the direction's summed squares."""
    g = torch.Generator().manual_seed(seed)
    for i, (x, d) in enumerate(zip(args, grads)):
        way = torch.randn(x.shape, generator=g).to(x.device)
        at = lambda s: f(*args[:i], x + s * way, *args[i + 1:])  # noqa: E731
        diff = (at(step) - at(-step)) / (2 * step)
        each = d.double() * way.double()
        want, size = float(each.sum()), float(each.square().sum().sqrt())
        assert abs(diff - want) <= 2e-2 * size + 1e-4, f"argument {i}: {diff} {want}"
