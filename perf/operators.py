"""The gated delta rule and the query/key norms with the position rotation, as measured work.

The gated delta rule keeps one state S (dk x dv, fp32) for each batch row and head:

    S~_t = exp(log_g_t) S_{t-1},   u_t = beta_t (v_t - k_t S~_t),
    S_t  = S~_t + k_t^T u_t,       o_t = scale q_t S_t,

with q, k in [B,Hk,T,dk] (every H / Hk value heads share one), v in [B,H,T,dv], log_g fp32 and
beta in the inputs' type, both [B,H,T]. The norms take each row of q and k (read through
strides, as a slice of a fused projection's output), divide it by its 2-norm or its root mean
square, multiply by a weight where there is one, and turn its first `rot` values by the row's
position; the result is dense [B,H,T,dk], the layout that the attention calls take.
"""
import math

import torch

own = False

CHUNK = 64


# ---------------------------------------------------------------- cases

def _step(name, B, H, Hk, T, dk, dv, dtype="bf16"):
    return {"name": name, "op": "delta", "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv, "dtype": dtype}


def _qk(name, op, B, H, Hk, T, d, norm, rot, interleaved, weights, positions, dtype="bf16"):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "T": T, "d": d, "norm": norm, "rot": rot,
            "interleaved": interleaved, "weights": weights, "positions": positions, "dtype": dtype}


def listed():
    return [
        # one user's next token: launch latency
        _step("step_single", 1, 16, 16, 1, 128, 128),
        # the next token of a full serving batch: the state's bytes
        _step("step_batch", 128, 16, 8, 1, 128, 128),
        # a few drafted tokens for each of a batch, taken in one call, from a carried state
        _step("step_draft", 16, 32, 16, 5, 128, 128),
        # a layer's pass over a prompt batch: the causal linear-attention layer's shape
        _step("prefill_layer", 8, 16, 16, 2048, 128, 128),
        # one long prompt of odd length: few heads, a long serial axis
        _step("prefill_long", 1, 16, 16, 16421, 128, 128),
        # short ragged prompts, shared key heads, narrow keys
        _step("prefill_ragged", 3, 12, 6, 777, 64, 128),
        # the fp32 parity shape
        _step("fp32_small", 1, 2, 2, 256, 64, 64, "fp32"),
        # a layer's training step, forward and backward
        dict(_step("train_layer", 8, 16, 16, 2048, 128, 128), op="delta_train"),
        # a ragged training batch with shared key heads and a carried state
        dict(_step("train_ragged", 2, 8, 4, 1001, 128, 256), op="delta_train"),
        # the rows of the same layer on their way to it: unit queries and keys, half of each row turned
        _qk("qk_layer", "qk", 8, 16, 16, 2048, 128, "l2", 64, False, False, False),
        # the next token of a serving batch: learned weights, each row at a position of its own
        _qk("qk_step", "qk", 64, 16, 8, 1, 128, "rms", 128, False, True, True),
        # a ragged training step of them, neighbouring pairs turned
        _qk("qk_train", "qk_train", 4, 16, 4, 1531, 128, "rms", 128, True, True, True),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["step", "prefill", "fp32", "train", "qk", "qk_train"])
    Hk = _spread(rng, 1, 16)
    H = Hk * rng.choice([1, 1, 2, 3] if Hk <= 8 else [1, 1, 2])
    dk, dv = rng.choice([64, 128]), rng.choice([64, 128, 256])
    if kind == "step":
        T = rng.choice([1, 1, 1, 2, 3, 4, 5, 7, 8])
        B = _spread(rng, 1, max(1, 128 * 16 * 128 * 128 // (H * dk * dv)))
        return {k: v for k, v in _step("", B, H, Hk, T, dk, dv, rng.choice(["bf16", "bf16", "fp32"])).items() if k != "name"}
    if kind in ("prefill", "train"):
        T = _spread(rng, 9, 16421 if kind == "prefill" else 2048)
        B = _spread(rng, 1, max(1, min(64, int(8 * 16 * 2048 * 128 * 128 / (H * T * max(dk, 128) * max(dv, 128))))))
        c = _step("", B, H, Hk, T, dk, dv)
        if kind == "train":
            c["op"] = "delta_train"
        return {k: v for k, v in c.items() if k != "name"}
    if kind == "fp32":
        T = _spread(rng, 9, 512)
        B = _spread(rng, 1, 4)
        return {k: v for k, v in _step("", B, H, Hk, T, dk, dv, "fp32").items() if k != "name"}
    d = rng.choice([64, 128, 256])
    T = _spread(rng, 1, 4096)
    B = _spread(rng, 1, max(1, min(256, 8 * 32 * 2048 * 128 // ((H + Hk) * T * d) // (1 if kind == "qk" else 2))))
    norm = rng.choice(["l2", "rms", "rms", "none"])
    c = _qk("", kind, B, H, Hk, T, d, norm, rng.choice([d, d, d // 2, 32, 0] if norm != "none" else [d, d // 2]),
            rng.random() < 0.5, norm == "rms", rng.random() < 0.5, rng.choice(["bf16", "bf16", "fp32"]))
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------- inputs

EPS = 1e-6
BASE = 10000.0


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _delta_inputs(case, seed):
    """q, k of unit rows (what the norms leave), values of unit variance, beta = sigmoid(N(0,1)), the data-dependent
    decay log sigmoid(N(0,1)) / 16, and a carried state."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Hk, T, dk, dv, t = case["B"], case["H"], case["Hk"], case["T"], case["dk"], case["dv"], _dtype(case)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    return {
        "q": unit(rnd(B, Hk, T, dk)).to(t), "k": unit(rnd(B, Hk, T, dk)).to(t), "v": rnd(B, H, T, dv).to(t),
        "log_g": torch.nn.functional.logsigmoid(rnd(B, H, T)) / 16, "beta": torch.sigmoid(rnd(B, H, T)).to(t),
        "S0": rnd(B, H, dk, dv) * 0.1,
    }, g


def _qk_inputs(case, seed):
    """A fused projection's output [B,T,(H+2Hk)d], of which q and k are strided slices; positions anywhere in a long
    context."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, Hk, T, d, t = case["B"], case["H"], case["Hk"], case["T"], case["d"], _dtype(case)
    proj = torch.randn((B, T, (H + 2 * Hk) * d), generator=g, device="cuda").to(t)
    x = {"proj": proj, "q": proj[:, :, :H * d].unflatten(2, (H, d)).transpose(1, 2),
         "k": proj[:, :, H * d:(H + Hk) * d].unflatten(2, (Hk, d)).transpose(1, 2)}
    if case["weights"]:
        x["w_q"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
        x["w_k"] = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    if case["rot"]:
        x["inv_freq"] = BASE ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    if case["positions"]:
        start = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
        x["positions"] = start + torch.arange(T, device="cuda")
    return x, g


def prepare(case, seed):
    if case["op"].startswith("delta"):
        x, g = _delta_inputs(case, seed)
        if case["op"] == "delta_train":
            x["dO"] = torch.randn(x["v"].shape, generator=g, device="cuda").to(x["v"].dtype)
            x["dST"] = torch.randn(x["S0"].shape, generator=g, device="cuda") * 0.1
            for n in ("q", "k", "v", "log_g", "beta", "S0"):
                x[n].requires_grad_(True)
    else:
        x, g = _qk_inputs(case, seed)
        if case["op"] == "qk_train":
            x["dq"] = torch.randn(x["q"].shape, generator=g, device="cuda").to(x["q"].dtype)
            x["dk"] = torch.randn(x["k"].shape, generator=g, device="cuda").to(x["k"].dtype)
            for n in ("q", "k", "w_q", "w_k"):
                if n in x:
                    x[n] = x[n].detach().requires_grad_(True)
    x["case"] = dict(case)
    return x


# ---------------------------------------------------------------- the plain forms

def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower A [..., 64, 64], by doubling blocks: the inverse of [[X, 0], [C, Y]] is
    [[X^-1, 0], [-Y^-1 C X^-1, Y^-1]]."""
    n = A.shape[-1]
    T = torch.eye(n, dtype=A.dtype, device=A.device).expand_as(A)
    at = torch.arange(n, device=A.device)
    w = 1
    while w < n:
        # the lower-left block of every 2w x 2w diagonal block
        C = A * ((at[:, None] // (2 * w) == at // (2 * w)) & (at[:, None] // w % 2 == 1) & (at // w % 2 == 0))
        T = T - T @ (C @ T)
        w *= 2
    return T


def _plain_delta(q, k, v, log_g, beta, S0):
    """The chunkwise form: within chunks of 64 tokens the corrections u solve a unit lower triangular system, one product
    for all chunks at once; the state then runs over the chunks."""
    t, T, dk = q.dtype, q.shape[2], q.shape[3]
    share = v.shape[1] // q.shape[1]
    q, k, v, beta = q.float(), k.float(), v.float(), beta.float()
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    more = -T % CHUNK
    rows = lambda x: torch.nn.functional.pad(x, (0, 0, 0, more)).unflatten(2, (-1, CHUNK))  # noqa: E731
    q, k, v, beta = rows(q) * dk ** -0.5, rows(k), rows(v), rows(beta.unsqueeze(-1))
    G = rows(log_g.unsqueeze(-1)).double().cumsum(3)
    at = torch.arange(CHUNK, device=q.device)
    D = (G - G.transpose(3, 4)).masked_fill(at[:, None] < at, -math.inf).exp().float()
    eG, eL, e1 = G.exp().float(), (G[..., -1:, :] - G).exp().float(), G[..., -1:, :].exp().float()
    Tm = _unit_lower_inverse(beta * (k @ k.transpose(3, 4)) * D * (at[:, None] > at))
    U, W = Tm @ (beta * v), Tm @ (beta * eG * k)
    P, qg, kl = (q @ k.transpose(3, 4)) * D, q * eG, (k * eL).transpose(3, 4)
    S, o = S0, []
    for n in range(q.shape[2]):
        u = U[:, :, n] - W[:, :, n] @ S
        o.append(qg[:, :, n] @ S + P[:, :, n] @ u)
        S = e1[:, :, n] * S + kl[:, :, n] @ u
    return torch.cat(o, 2)[:, :, :T].to(t), S


def _plain_qk_one(x, w, cs, case):
    t, n = x.dtype, x.shape[-1]
    x = x.float()
    if case["norm"] != "none":
        x = x / (x.square().sum(-1, keepdim=True) / (n if case["norm"] == "rms" else 1) + EPS).sqrt()
    if w is not None:
        x = x * w
    r = case["rot"]
    if r:
        c, s = cs
        y, rest = x[..., :r], x[..., r:]
        a, b = (y[..., 0::2], y[..., 1::2]) if case["interleaved"] else (y[..., :r // 2], y[..., r // 2:])
        a, b = a * c - b * s, b * c + a * s
        y = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
        x = torch.cat((y, rest), -1)
    return x.to(t).contiguous()


def _plain_qk(x):
    case, cs = x["case"], None
    if case["rot"]:
        at = x["positions"] if case["positions"] else torch.arange(case["T"], device=x["q"].device).unsqueeze(0)
        angle = at[:, None, :, None].double() * x["inv_freq"]
        cs = angle.cos().float(), angle.sin().float()
    return _plain_qk_one(x["q"], x.get("w_q"), cs, case), _plain_qk_one(x["k"], x.get("w_k"), cs, case)


# ---------------------------------------------------------------- one pass

def _own_qk(x):
    import chunkwise_gated_linear_gla_gb300 as gla
    case = x["case"]
    return gla.qk_norm_rope(x["q"], x["k"], norm=None if case["norm"] == "none" else case["norm"], w_q=x.get("w_q"),
                            w_k=x.get("w_k"), eps=EPS, inv_freq=x.get("inv_freq"), positions=x.get("positions"),
                            interleaved=case["interleaved"])


def _own_delta(x):
    import chunkwise_gated_linear_gla_gb300 as gla
    if x["case"]["op"] == "delta_train":
        return gla.delta_attention(x["q"], x["k"], x["v"], x["log_g"], x["beta"], x["S0"])
    return gla.delta_forward(x["q"], x["k"], x["v"], x["log_g"], x["beta"], x["S0"])


def run(state):
    x = state
    op = x["case"]["op"]
    if op.startswith("delta"):
        if own:
            O, ST = _own_delta(x)
        else:
            O, ST = _plain_delta(x["q"], x["k"], x["v"], x["log_g"], x["beta"], x["S0"])
        out = {"O": O, "ST": ST}
        if op == "delta_train":
            names = ("q", "k", "v", "log_g", "beta", "S0")
            got = torch.autograd.grad((O, ST), [x[n] for n in names], (x["dO"], x["dST"]))
            out = {"O": O.detach(), "ST": ST.detach(), **{"d" + n: d for n, d in zip(names, got)}}
        return out
    y, z = _own_qk(x) if own else _plain_qk(x)
    if op == "qk":
        return {"q": y, "k": z}
    names = [n for n in ("q", "k", "w_q", "w_k") if n in x]
    got = torch.autograd.grad((y, z), [x[n] for n in names], (x["dq"], x["dk"]))
    return {"yq": y.detach(), "yk": z.detach(), **{"d" + n: d for n, d in zip(names, got)}}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, H, Hk, T = case["B"], case["H"], case["Hk"], case["T"]
    if case["op"].startswith("delta"):
        dk, dv = case["dk"], case["dv"]
        qk, v, gates, s = 2 * B * Hk * T * dk * e, B * H * T * dv * e, B * H * T * (4 + e), B * H * dk * dv * 4
        if case["op"] == "delta":
            # the recurrence itself: decay, k S, k^T u, q S
            return {"bytes": qk + 2 * v + gates + 2 * s, "flops": 7 * B * H * T * dk * dv}
        # inputs and dO, dST read once; O, ST and every gradient written once
        return {"bytes": 2 * qk + 4 * v + 2 * gates + 4 * s, "flops": 22 * B * H * T * dk * dv}
    d = case["d"]
    rows = B * (H + Hk) * T
    more = (B * T * 8 if case["positions"] else 0) + (8 * d if case["weights"] else 0) + case["rot"] * 4
    if case["op"] == "qk":
        return {"bytes": 2 * rows * d * e + more, "flops": 8 * rows * d}
    return {"bytes": 4 * rows * d * e + 2 * more, "flops": 24 * rows * d}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_delta(x, train):
    q, k, v, a, b, S0 = (x[n].detach().double() for n in ("q", "k", "v", "log_g", "beta", "S0"))
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    share, scale = H // Hk, dk ** -0.5
    a = a.exp()
    col = lambda y, t: y[:, :, t].repeat_interleave(share, 1).unsqueeze(3)  # noqa: E731  (B,H,dk,1)
    o = torch.empty((B, H, T, dv), dtype=torch.float64, device=q.device)
    every = max(1, int(T ** 0.5))
    kept, S = {}, S0

    def token(S, t):
        Sd = S * a[:, :, t, None, None]
        kt = col(k, t)
        r = v[:, :, t] - (kt * Sd).sum(2)
        return Sd, r, Sd + kt * (b[:, :, t, None] * r).unsqueeze(2)

    for t in range(T):
        if t % every == 0:
            kept[t] = S
        S = token(S, t)[2]
        o[:, :, t] = scale * (col(q, t) * S).sum(2)
    out = {"O": o, "ST": S}
    if not train:
        return out
    dO, dS = x["dO"].double(), x["dST"].double()
    dq, dk_, dv_ = torch.zeros((B, H, T, dk), dtype=torch.float64, device=q.device), None, torch.empty_like(v)
    dk_ = torch.zeros_like(dq)
    da, db = torch.empty_like(a), torch.empty_like(a)
    for first in sorted(kept, reverse=True):
        S, seen = kept[first], []
        for t in range(first, min(T, first + every)):
            Sd, r, Sn = token(S, t)
            seen.append((S, Sd, r, Sn))
            S = Sn
        for t in range(min(T, first + every) - 1, first - 1, -1):
            S, Sd, r, Sn = seen.pop()
            kt, bt, g = col(k, t), b[:, :, t, None], dO[:, :, t].unsqueeze(2)
            dq[:, :, t] = scale * (Sn * g).sum(3)
            dS = dS + scale * col(q, t) * g
            du = (kt * dS).sum(2)
            dr = bt * du
            db[:, :, t] = (du * r).sum(2)
            dv_[:, :, t] = dr
            dk_[:, :, t] = (dS * (bt * r).unsqueeze(2)).sum(3) - (Sd * dr.unsqueeze(2)).sum(3)
            dS = dS - kt * dr.unsqueeze(2)
            da[:, :, t] = (dS * Sd).sum((2, 3))
            dS = dS * a[:, :, t, None, None]
    fold = lambda y: y.unflatten(1, (Hk, share)).sum(2)  # noqa: E731
    return {**out, "dq": fold(dq), "dk": fold(dk_), "dv": dv_, "dlog_g": da, "dbeta": db, "dS0": dS}


def _exact_qk(x, train):
    case = x["case"]
    n, r = case["d"], case["rot"]
    i = torch.arange(n, device="cuda")
    turn = i < r
    if case["interleaved"]:
        pair, which, mate = i // 2, i % 2, i ^ 1
    else:
        pair, which, mate = i % max(1, r // 2), (i >= r // 2).long(), torch.where(i < r // 2, i + r // 2, i - r // 2)
    mate = torch.where(turn, mate, i)
    cos, sin = torch.ones((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64, device="cuda")
    if r:
        at = x["positions"] if case["positions"] else torch.arange(case["T"], device="cuda").unsqueeze(0)
        f = x["inv_freq"][torch.where(turn, pair, torch.zeros_like(pair))]
        th = at[:, None, :, None].double() * f
        cos = torch.where(turn, th.cos(), torch.ones_like(th))
        sin = torch.where(turn, th.sin(), torch.zeros_like(th)) * (2 * which - 1)
    N = {"l2": 1.0, "rms": float(n), "none": 0.0}[case["norm"]]
    out = {}
    for a in ("q", "k"):
        z = x[a].detach().double()
        w = x["w_" + a].detach().double() if case["weights"] else torch.ones(n, dtype=torch.float64, device="cuda")
        inv = (z.square().sum(-1, keepdim=True) / N + EPS).rsqrt() if N else torch.ones_like(z[..., :1])
        y = z * inv * w
        out[("y" if train else "") + a] = y * cos + y[..., mate] * sin
        if train:
            dy = x["d" + a].double()
            dz = dy * cos - dy[..., mate] * sin  # the rotation turned back
            if case["weights"]:
                out["dw_" + a] = (dz * z * inv).sum((0, 1, 2))
            dz = dz * w
            out["d" + a] = inv * (dz - z * inv.square() * (dz * z).sum(-1, keepdim=True) / N) if N else dz
    return out


def exact(case, seed):
    x = prepare(case, seed)
    with torch.no_grad():
        if case["op"].startswith("delta"):
            return _exact_delta(x, case["op"] == "delta_train")
        return _exact_qk(x, case["op"] == "qk_train")
