"""What stands around the recurrences of a layer, as measured work: the short causal convolution, the selective scan, the
heads' norm with its gate, and the residual with its norm.

causal_conv, a filter of W taps for every channel, over the tokens up to and with its own:
    y_t = silu(bias + sum_j w_j x_{t-W+1+j}),
x in [B,T,D] or, head by head, [B,H,T,d] (strided slices of a projection), the tokens before the first from a carried state
[B,W-1,D]; y is dense in x's shape, and the state after the call is returned.

selective_scan, N states h for every channel, whose decay differs per channel and state:
    delta_t = softplus(dt_t + dt_bias),   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,   y_t = (C_t . h_t + D x_t) silu(z_t),
x, dt, z in [B,T,D], A in [D,N], B and C in [B,T,G,N] (every D / G channels share one), h in [B,D,N].

norm_gate, the heads' outputs [B,H,T,d] on their way to the output projection [B,T,H,d]:
    y = w x / rms(x) silu(g),   or, with the gate first,   y = w u / rms(u), u = x silu(g).

residual_norm, a block's output into the residual and the next block's input out of it:
    h = residual + scale u,   u = x or x / rms(x),   y = w h / rms(h).
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def _conv(name, B, H, T, d, W, dtype="bf16", train=False):
    return {"name": name, "op": "conv_train" if train else "conv", "B": B, "H": H, "T": T, "d": d, "W": W, "dtype": dtype}


def _scan(name, B, T, D, N, G=1, dtype="bf16", train=False):
    return {"name": name, "op": "scan_train" if train else "scan", "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype}


def _gate(name, B, H, T, d, gate_first, dtype="bf16", train=False):
    return {"name": name, "op": "gate_train" if train else "gate", "B": B, "H": H, "T": T, "d": d,
            "gate_first": gate_first, "dtype": dtype}


def _res(name, rows, D, post_norm, scaled, dtype="bf16", res_dtype="bf16", train=False):
    return {"name": name, "op": "res_train" if train else "res", "rows": rows, "D": D, "post_norm": post_norm,
            "scaled": scaled, "dtype": dtype, "res_dtype": res_dtype}


def listed():
    return [
        # one user's next token: launch latency
        _scan("scan_single", 1, 1, 4096, 16),
        # the next token of a full serving batch: the states' bytes
        _scan("scan_step_batch", 128, 1, 4096, 16),
        # a layer's pass over a prompt batch, inner width twice the model's 2048
        _scan("scan_prefill_layer", 8, 2048, 4096, 16),
        # one long prompt of odd length: few channels for the chip, a long serial axis
        _scan("scan_prefill_long", 1, 16421, 4096, 16),
        # a layer's training step, forward and backward
        _scan("scan_train_layer", 4, 2048, 4096, 16, train=True),
        # a ragged fp32 training batch with two groups of B and C and wider states
        _scan("scan_train_ragged", 3, 777, 1040, 32, 2, "fp32", train=True),
        # the convolution of the same serving batch's next token
        _conv("conv_step_batch", 128, 1, 1, 4096, 4),
        # the values of the linear-attention layer (16 heads of 128), projection to head-major, with gradients
        _conv("conv_train_heads", 8, 16, 2048, 128, 4, train=True),
        # the outputs of that layer's heads, normed and gated into the projection's layout
        _gate("gate_layer", 8, 16, 2048, 128, False),
        # a ragged training batch of the 512-wide heads
        _gate("gate_train_wide", 3, 4, 1531, 512, False, train=True),
        # the next tokens of a serving batch into an fp32 residual
        _res("res_step", 64, 2048, False, False, res_dtype="fp32"),
        # the residual between two blocks of a training step at model width 2048, the block's output normed and scaled
        _res("res_train_layer", 8 * 2048, 2048, True, True, train=True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan_step", "scan_train", "conv", "conv_train", "gate", "gate_train", "res", "res_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind.startswith("scan"):
        N = rng.choice([8, 16, 16, 32, 64])
        G = rng.choice([1, 1, 2, 4])
        D = 16 * G * _spread(rng, 1, 8192 // (16 * G))
        T = rng.randint(1, 4) if kind == "scan_step" else _spread(rng, 5, 16421 if kind == "scan" else 2048)
        most = 8 * 2048 * 4096 * 16 // (2 if kind == "scan_train" else 1)
        if T * D * N > most:
            T = most // (D * N)
        B = _spread(rng, 1, max(1, min(256, most // (T * D * N))))
        c = _scan("", B, T, D, N, G, dtype, kind == "scan_train")
    elif kind.startswith("conv"):
        H = rng.choice([1, 1, 2, 4, 16])
        d = 16 * _spread(rng, 1, 512 // H)
        T = _spread(rng, 1, 4096)
        B = _spread(rng, 1, max(1, min(256, 8 * 2048 * 2048 // (H * d * T))))
        c = _conv("", B, H, T, d, rng.choice([2, 3, 4, 4]), dtype, kind == "conv_train")
    elif kind.startswith("gate"):
        d = rng.choice([64, 128, 128, 256, 512, 16 * rng.randint(1, 64)])
        H = _spread(rng, 1, 32)
        T = _spread(rng, 1, 4096)
        B = _spread(rng, 1, max(1, min(256, 8 * 2048 * 2048 // (H * d * T))))
        c = _gate("", B, H, T, d, rng.random() < 0.4, dtype, kind == "gate_train")
    else:
        D = 16 * _spread(rng, 8, 512)
        rows = _spread(rng, 1, 8 * 2048 * 2048 // D)
        c = _res("", rows, D, rng.random() < 0.5, rng.random() < 0.5, dtype,
                 rng.choice([dtype, "fp32"]), kind == "res_train")
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t, op = _dtype(case["dtype"]), case["op"]
    x = {"case": dict(case)}
    if op.startswith("conv"):
        B, H, T, d, W = case["B"], case["H"], case["T"], case["d"], case["W"]
        D = H * d
        # the first half of a projection's output
        proj = rnd(B, T, 2 * D).to(t)[:, :, :D]
        x["x"] = proj.unflatten(2, (H, d)).transpose(1, 2) if H > 1 else proj
        x["w"], x["bias"] = rnd(D, W) * W ** -0.5, rnd(D) * 0.1
        x["S0"] = rnd(B, W - 1, D).to(t)
        if op == "conv_train":
            x["dy"], x["dST"] = rnd(*x["x"].shape).to(t), (rnd(B, W - 1, D) * 0.1).to(t)
            x["grads"] = ("x", "w", "bias", "S0")
    elif op.startswith("scan"):
        B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
        R = 8 * max(1, D // 256)
        # z beside x's projection; B and C beside the low-rank delta in one projection's output
        x["z"] = rnd(B, T, 2 * D).to(t)[:, :, D:]
        low = rnd(B, T, R + 2 * G * N).to(t)
        x["B"], x["C"] = low[:, :, R:R + G * N].unflatten(2, (G, N)), low[:, :, R + G * N:].unflatten(2, (G, N))
        a = torch.nn.functional.silu(rnd(B, T, D))
        x["x"], x["dt"] = a.to(t), (rnd(B, T, D) * 0.5).to(t)
        x["A"] = -(1 + torch.arange(N, device="cuda")) * torch.exp(0.1 * rnd(D, N))
        # steps between 0.001 and 0.1 at dt = 0: the inverse of softplus
        step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        x["dt_bias"] = step + torch.log(-torch.expm1(-step))
        x["D"] = 1 + 0.1 * rnd(D)
        x["S0"] = rnd(B, D, N) * 0.1
        if op == "scan_train":
            x["dy"], x["dST"] = rnd(B, T, D).to(t), rnd(B, D, N) * 0.1
            x["grads"] = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0")
    elif op.startswith("gate"):
        B, H, T, d = case["B"], case["H"], case["T"], case["d"]
        # the attention's dense output, and the gate as a slice of a projection
        x["x"] = rnd(B, H, T, d).to(t)
        x["g"] = rnd(B, T, 2 * H * d).to(t)[:, :, H * d:].unflatten(2, (H, d)).transpose(1, 2)
        x["w"] = 1 + 0.1 * rnd(d)
        if op == "gate_train":
            x["dy"] = rnd(B, T, H, d).to(t)
            x["grads"] = ("x", "g", "w")
    else:
        n, D = case["rows"], case["D"]
        x["x"], x["r"] = rnd(n, D).to(t), (2 * rnd(n, D)).to(_dtype(case["res_dtype"]))
        x["w"] = 1 + 0.1 * rnd(D)
        if case["scaled"]:
            x["scale"] = 0.5 + 0.1 * rnd(D)
        if op == "res_train":
            x["dh"], x["dy"] = rnd(n, D).to(x["r"].dtype), rnd(n, D).to(t)
            x["grads"] = ("x", "r", "w", "scale") if case["scaled"] else ("x", "r", "w")
    for n in x.get("grads", ()):
        x[n] = x[n].detach().requires_grad_(True)
    return x


# ---------------------------------------------------------------- the plain forms

def _plain_conv(x, w, bias, S0):
    t = x.dtype
    heads = x.dim() == 4
    rows = (x.transpose(1, 2).flatten(2) if heads else x).float()
    B, T, D = rows.shape
    W = w.shape[1]
    rows = torch.cat((S0.float(), rows), 1)
    y = bias + sum(w[:, j] * rows[:, j:j + T] for j in range(W))
    y = y / (1 + torch.exp(-y))
    if heads:
        y = y.unflatten(2, x.shape[1::2]).transpose(1, 2).contiguous()
    return y.to(t), rows[:, T:].to(t)


def _plain_scan(x, dt, A, Bm, Cm, Dk, z, dt_bias, S0):
    """The tokens in pieces of about sqrt(T): every piece from a zero state, all pieces at once, token by token; then the
    states from piece to piece, and what each piece's entering state adds."""
    t, (B, T, D), G = x.dtype, x.shape, Bm.shape[2]
    L = max(1, math.isqrt(T))
    more = -T % L
    cut = lambda a: torch.nn.functional.pad(a, (0, 0, 0, more)).unflatten(1, (-1, L))  # noqa: E731  [B,n,L,.]
    xf, v = x.float(), dt.float() + dt_bias
    delta = v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))
    xd, dl, Bf, Cf = cut(delta * xf), cut(delta), cut(Bm.float().flatten(2)), cut(Cm.float().flatten(2))
    total = dl.double().cumsum(2)
    wide = lambda a, i: a[:, :, i].unflatten(2, (G, 1, -1)).expand(-1, -1, -1, D // G, -1).flatten(2, 3)  # noqa: E731  [B,n,D,N]
    h, y = torch.zeros((), device=x.device), []
    for i in range(L):
        h = torch.exp(dl[:, :, i, :, None] * A) * h + xd[:, :, i, :, None] * wide(Bf, i)
        y.append((h * wide(Cf, i)).sum(-1))
    S, enter = S0, []
    for n in range(h.shape[1]):
        enter.append(S)
        S = torch.exp(total[:, n, L - 1, :, None].float() * A) * S + h[:, n]
    enter = torch.stack(enter, 1)
    y = [a + (torch.exp(total[:, :, i, :, None].float() * A) * enter * wide(Cf, i)).sum(-1) for i, a in enumerate(y)]
    y = torch.stack(y, 2).flatten(1, 2)[:, :T] + Dk * xf
    zf = z.float()
    return (y * (zf / (1 + torch.exp(-zf)))).to(t), S


def _plain_gate(x, g, w, gate_first):
    t = x.dtype
    x, g = x.float(), g.float()
    s = g / (1 + torch.exp(-g))
    if gate_first:
        x = x * s
    x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    if not gate_first:
        x = x * s
    return x.transpose(1, 2).to(t).contiguous()


def _plain_res(x, r, w, scale, post_norm):
    u = x.float()
    if post_norm:
        u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt()
    h = r.float() + (u if scale is None else u * scale)
    y = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    return h.to(r.dtype), y.to(x.dtype)


# ---------------------------------------------------------------- one pass

def _outputs(x):
    case = x["case"]
    op = case["op"]
    if own:
        import chunkwise_gated_linear_gla_gb300 as gla
        if op.startswith("conv"):
            y, ST = gla.causal_conv(x["x"], x["w"], x["bias"], x["S0"])
            return {"y": y, "ST": ST}
        if op.startswith("scan"):
            y, ST = gla.selective_scan(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"], x["z"], x["dt_bias"], x["S0"])
            return {"y": y, "ST": ST}
        if op.startswith("gate"):
            return {"y": gla.norm_gate(x["x"], x["g"], x["w"], eps=EPS, gate_first=case["gate_first"])}
        h, y = gla.residual_norm(x["x"], x["r"], x["w"], scale=x.get("scale"), post_norm=case["post_norm"], eps=EPS)
        return {"h": h, "y": y}
    if op.startswith("conv"):
        return dict(zip(("y", "ST"), _plain_conv(x["x"], x["w"], x["bias"], x["S0"])))
    if op.startswith("scan"):
        return dict(zip(("y", "ST"), _plain_scan(x["x"], x["dt"], x["A"], x["B"], x["C"], x["D"], x["z"], x["dt_bias"], x["S0"])))
    if op.startswith("gate"):
        return {"y": _plain_gate(x["x"], x["g"], x["w"], case["gate_first"])}
    return dict(zip(("h", "y"), _plain_res(x["x"], x["r"], x["w"], x.get("scale"), case["post_norm"])))


def run(state):
    x = state
    out = _outputs(x)
    if "grads" not in x:
        return out
    got = torch.autograd.grad(list(out.values()), [x[n] for n in x["grads"]], [x["d" + n] for n in out])
    return {**{n: a.detach() for n, a in out.items()}, **{"d" + n: a for n, a in zip(x["grads"], got)}}


def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    train = op.endswith("train")
    if op.startswith("conv"):
        B, T, D, W = case["B"], case["T"], case["H"] * case["d"], case["W"]
        v, s, p = B * T * D, 2 * B * (W - 1) * D * e, (W + 1) * D * 4
        if train:   # x and dy read; y and dx written; states and their gradients
            return {"bytes": 4 * v * e + 2 * s + 2 * p, "flops": v * (6 * W + 20)}
        return {"bytes": 2 * v * e + s + p, "flops": v * (2 * W + 4)}
    if op.startswith("scan"):
        B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
        v, bc, s, p = B * T * D, 2 * B * T * G * N * e, 2 * B * D * N * 4, (D * N + 2 * D) * 4
        if train:   # x, dt, z, dy read; y, dx, ddt, dz written
            return {"bytes": 8 * v * e + 2 * bc + 2 * s + 2 * p, "flops": v * (20 * N + 30)}
        return {"bytes": 4 * v * e + bc + s + p, "flops": v * (7 * N + 14)}
    if op.startswith("gate"):
        v, p = case["B"] * case["H"] * case["T"] * case["d"], 4 * case["d"]
        return {"bytes": 6 * v * e + 2 * p, "flops": 30 * v} if train else {"bytes": 3 * v * e + p, "flops": 10 * v}
    v, er, p = case["rows"] * case["D"], 2 if case["res_dtype"] == "bf16" else 4, 8 * case["D"]
    if train:       # x, r, dh, dy read; h, y, dx, dr written
        return {"bytes": v * (4 * e + 4 * er) + 2 * p, "flops": 24 * v}
    return {"bytes": v * (2 * e + 2 * er) + p, "flops": 8 * v}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _sig(a):
    return 1 / (1 + torch.exp(-a))


def _exact_conv(x, train):
    heads = x["x"].dim() == 4
    z, w, b, S0 = (x[n].detach().double() for n in ("x", "w", "bias", "S0"))
    flat = lambda a: a.permute(0, 2, 1, 3).reshape(a.shape[0], a.shape[2], -1) if heads else a  # noqa: E731
    shaped = lambda a: a.reshape(a.shape[0], a.shape[1], x["x"].shape[1], -1).permute(0, 2, 1, 3).contiguous() if heads else a  # noqa: E731
    z = torch.cat((S0, flat(z)), 1)
    W = w.shape[1]
    T = z.shape[1] - W + 1
    a = b.expand(z.shape[0], T, -1).clone()
    for t0 in range(W):
        a += z[:, t0:t0 + T] * w[:, t0]
    s = _sig(a)
    out = {"y": shaped(a * s), "ST": z[:, T:]}
    if train:
        da = flat(x["dy"].double()) * (s + a * s * (1 - s))
        dz = torch.zeros_like(z)
        dz[:, T:] += x["dST"].double()
        dw = torch.empty_like(w)
        for t0 in range(W):
            dz[:, t0:t0 + T] += da * w[:, t0]
            dw[:, t0] = (da * z[:, t0:t0 + T]).sum((0, 1))
        out.update(dx=shaped(dz[:, W - 1:]), dw=dw, dbias=da.sum((0, 1)), dS0=dz[:, :W - 1])
    return out


def _exact_scan(x, train):
    u, dt, A, Bm, Cm, Dk, z, bias, h = (x[n].detach().double() for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "S0"))
    B, T, D = u.shape
    G = Bm.shape[2]
    v = dt + bias
    delta = torch.logaddexp(v, torch.zeros_like(v))
    per = lambda a, t: a[:, t].repeat_interleave(D // G, 1)  # noqa: E731  [B,D,N]
    every = max(1, int(T ** 0.5))
    kept, y = {}, torch.empty_like(u)
    for t in range(T):
        if t % every == 0:
            kept[t] = h
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * u[:, t]).unsqueeze(2) * per(Bm, t)
        y[:, t] = torch.einsum("bdn,bdn->bd", per(Cm, t), h)
    y += Dk * u
    s = _sig(z)
    out = {"y": y * z * s, "ST": h}
    if not train:
        return out
    dout = x["dy"].double()
    dyy = dout * z * s
    out_z = dout * y * (s + z * s * (1 - s))
    du, dd = dyy * Dk, torch.empty_like(u)
    dA, dB, dC, g = torch.zeros_like(A), torch.empty_like(Bm), torch.empty_like(Cm), x["dST"].double()
    fold = lambda a: a.reshape(B, G, D // G, -1).sum(2)  # noqa: E731
    for first in sorted(kept, reverse=True):
        h, seen, last = kept[first], [], min(T, first + every)
        for t in range(first, last):
            a = torch.exp(delta[:, t, :, None] * A)
            old, h = h, a * h + (delta[:, t] * u[:, t]).unsqueeze(2) * per(Bm, t)
            seen.append((a, old, h))
        for t in range(last - 1, first - 1, -1):
            a, old, new = seen.pop()
            g = g + dyy[:, t].unsqueeze(2) * per(Cm, t)
            dC[:, t] = fold(dyy[:, t].unsqueeze(2) * new)
            dB[:, t] = fold(g * (delta[:, t] * u[:, t]).unsqueeze(2))
            through = (g * per(Bm, t)).sum(2)
            du[:, t] += through * delta[:, t]
            g_a = g * old * a
            dd[:, t] = through * u[:, t] + (g_a * A).sum(2)
            dA += (g_a * delta[:, t, :, None]).sum(0)
            g = g * a
    ddt = dd * _sig(v)
    return {**out, "dx": du, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (dyy * u).sum((0, 1)), "dz": out_z,
            "ddt_bias": ddt.sum((0, 1)), "dS0": g}


def _exact_norm(a):
    return (a.square().sum(-1, keepdim=True) / a.shape[-1] + EPS).rsqrt()


def _exact_norm_grad(a, da_hat):
    """The gradient of a from that of a / rms(a)."""
    inv = _exact_norm(a)
    return inv * (da_hat - a * inv.square() * (a * da_hat).sum(-1, keepdim=True) / a.shape[-1])


def _exact_gate(x, train):
    z, g, w = (x[n].detach().double() for n in ("x", "g", "w"))
    s = _sig(g)
    act, slope = g * s, s + g * s * (1 - s)
    first = x["case"]["gate_first"]
    u = z * act if first else z
    n = u * _exact_norm(u)
    y = n * w if first else n * w * act
    out = {"y": y.transpose(1, 2).contiguous()}
    if train:
        dy = x["dy"].double().transpose(1, 2)
        if first:
            du = _exact_norm_grad(u, dy * w)
            out.update(dx=du * act, dg=du * z * slope, dw=(dy * n).sum((0, 1, 2)))
        else:
            out.update(dx=_exact_norm_grad(u, dy * w * act), dg=dy * n * w * slope, dw=(dy * n * act).sum((0, 1, 2)))
    return out


def _exact_res(x, train):
    z, r, w = (x[n].detach().double() for n in ("x", "r", "w"))
    scaled, post = x["case"]["scaled"], x["case"]["post_norm"]
    scale = x["scale"].detach().double() if scaled else 1.0
    u = z * _exact_norm(z) if post else z
    h = r + scale * u
    out = {"h": h, "y": h * _exact_norm(h) * w}
    if train:
        dy = x["dy"].double()
        dh = x["dh"].double() + _exact_norm_grad(h, dy * w)
        out.update(dx=_exact_norm_grad(z, dh * scale) if post else dh * scale, dr=dh, dw=(dy * h * _exact_norm(h)).sum(0))
        if scaled:
            out["dscale"] = (dh * u).sum(0)
    return out


def exact(case, seed):
    x = prepare(case, seed)
    op = case["op"]
    of = {"conv": _exact_conv, "scan": _exact_scan, "gate": _exact_gate, "res": _exact_res}[op.split("_")[0]]
    with torch.no_grad():
        return of(x, op.endswith("train"))
