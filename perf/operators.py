"""Operators of the layers that stand next to the PD scan, as they are measured.

Two operators, each in its forward and its backward direction:

* ``qk`` / ``qk_bwd``: the norm of every query and key head, with the position rotation in the same pass.
* ``delta`` / ``delta_bwd``: the gated delta rule, whole sequences and single tokens.

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` by the calls of the package. ``exact`` goes by the
definitions, step by step in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # steps that the plain form of the delta rule takes at once


# --------------------------------------------------------------------- cases

def _qk(name, op, batch, seqlen, q_heads, k_heads, N, dtype, mode, weights, rot, interleaved, far):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "q_heads": q_heads, "k_heads": k_heads, "N": N, "dtype": dtype,
            "mode": mode, "weights": weights, "rot": rot, "interleaved": interleaved, "far": far}


def _delta(name, op, batch, seqlen, qk_heads, heads, N, P, dtype, gates, state, ragged):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "qk_heads": qk_heads, "heads": heads, "N": N, "P": P, "dtype": dtype,
            "gates": gates, "state": state, "ragged": ragged}


def listed():
    return [
        # one new token for each of 32 sequences, far into their texts: latency counts
        _qk("qk_decode", "qk", 32, 1, 32, 32, 64, "bf16", "rms", True, 64, False, True),
        # queries and keys of the language model layer (batch 8, 2048 tokens, 32 heads of 64)
        _qk("qk_layer", "qk", 8, 2048, 32, 32, 64, "bf16", "rms", True, 64, False, False),
        # the gradients of the same layer in a training step
        _qk("qk_bwd_layer", "qk_bwd", 8, 2048, 32, 32, 64, "bf16", "rms", True, 64, False, False),
        # odd sizes, fewer key heads than query heads, part of the head rotated in neighbouring pairs, unit norms for the delta rule
        _qk("qk_bwd_odd", "qk_bwd", 3, 517, 12, 4, 80, "f32", "l2", False, 36, True, True),
        # one new token of one sequence: the smallest serving step
        _delta("delta_token", "delta", 1, 1, 8, 8, 64, 64, "bf16", "f32", True, False),
        # one new token for each of 64 sequences: the states are read and written once
        _delta("delta_tokens", "delta", 64, 1, 32, 32, 128, 64, "bf16", "f32", True, False),
        # the language model layer in training, forward
        _delta("delta_layer", "delta", 8, 2048, 32, 32, 64, 64, "bf16", "f32", False, False),
        # long time series in 32 bits whose length is no multiple of a chunk
        _delta("delta_series", "delta", 4, 18000, 8, 8, 32, 32, "f32", "f32", False, False),
        # prompts of different lengths in one padded batch, continued from a state, two value heads to a key head
        _delta("delta_prompts", "delta", 4, 4096, 16, 32, 128, 128, "bf16", "f32", True, True),
        # the language model layer in training, backward
        _delta("delta_bwd_layer", "delta_bwd", 8, 2048, 32, 32, 64, 64, "bf16", "f32", False, False),
        # backward with shared key heads and 16-bit gates, a segment of a longer sequence (gradients of the state at both ends)
        _delta("delta_bwd_shared", "delta_bwd", 2, 2048, 16, 32, 128, 128, "bf16", "bf16", True, False),
        # small odd sizes in 32 bits, ragged
        _delta("delta_bwd_odd", "delta_bwd", 3, 333, 2, 6, 40, 24, "f32", "f32", True, True),
    ]


def _log(rng, low, high):
    return min(high, max(low, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["qk", "qk_bwd", "delta", "delta", "delta_bwd", "delta_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk", "qk_bwd"):
        N = rng.choice([32, 64, 64, 80, 96, 128, 128, rng.randint(3, 128)])
        q_heads = rng.randint(1, 32)
        k_heads = rng.choice([q_heads, rng.randint(1, q_heads)])
        rows = _log(rng, 1, max(1, min(32768, (1 << 26) // ((q_heads + k_heads) * N) // (2 if dtype == "f32" else 1))))
        batch = _log(rng, 1, min(rows, 64))
        rot = 2 * rng.choice([0, N // 4, N // 2, N // 2, rng.randint(0, N // 2)])
        return {"op": op, "batch": batch, "seqlen": max(1, rows // batch), "q_heads": q_heads, "k_heads": k_heads, "N": N, "dtype": dtype,
                "mode": rng.choice(["rms", "l2"]), "weights": rng.random() < 0.6, "rot": rot, "interleaved": rng.random() < 0.4,
                "far": rng.random() < 0.4}
    N = rng.choice([32, 64, 64, 128, 128, rng.randint(4, 128)])
    P = rng.choice([N, 64, 128, rng.randint(1, 128)])
    qk_heads = rng.randint(1, 12)
    heads = qk_heads * rng.choice([1, 1, 2, 3])
    L = _log(rng, 1, 8192 if op == "delta" else 4096)
    most = (1 << 32) if op == "delta" else (1 << 31)
    batch = _log(rng, 1, max(1, min(64, most // (L * heads * N * P))))
    return {"op": op, "batch": batch, "seqlen": L, "qk_heads": qk_heads, "heads": heads, "N": N, "P": P, "dtype": dtype,
            "gates": rng.choice(["f32", "f32", "bf16"]), "state": rng.random() < 0.6, "ragged": rng.random() < 0.35}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    c, dt = case, DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": dict(c)}
    B, L, N = c["batch"], c["seqlen"], c["N"]
    if c["op"] in ("qk", "qk_bwd"):
        # head outputs of a projection: a scale of its own for each head
        s["q"] = (normal(B, L, c["q_heads"], N) * torch.exp(0.5 * normal(c["q_heads"], 1))).to(dt)
        s["k"] = (normal(B, L, c["k_heads"], N) * torch.exp(0.5 * normal(c["k_heads"], 1))).to(dt)
        s["wq"] = 1 + 0.2 * normal(N) if c["weights"] else None
        s["wk"] = 1 + 0.2 * normal(N) if c["weights"] else None
        s["inv_freq"] = s["positions"] = None
        if c["rot"]:
            i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-2 * i / c["rot"])).float()
            first = torch.randint(0, 1000000 if c["far"] else 1, (B, 1), generator=gen, device="cuda")
            s["positions"] = (first + torch.arange(L, device="cuda")).to(torch.int32)
        if c["op"] == "qk_bwd":
            s["dq_out"] = normal(B, L, c["q_heads"], N).to(dt)
            s["dk_out"] = normal(B, L, c["k_heads"], N).to(dt)
        return s
    P, H, G = c["P"], c["heads"], DTYPES[c["gates"]]

    def unit(x):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)

    s["q"] = unit(normal(B, L, c["qk_heads"], N)).to(dt)
    s["k"] = unit(normal(B, L, c["qk_heads"], N)).to(dt)
    s["v"] = normal(B, L, H, P).to(dt)
    # decays from nearly none to a few tokens' memory, a bias of its own for each head
    s["g"] = -torch.log1p(torch.exp(normal(B, L, H) - 2.5 + normal(H))).to(G)
    s["beta"] = torch.sigmoid(normal(B, L, H)).to(G)
    s["h0"] = 0.3 * normal(B, H, N, P) if c["state"] else None
    s["lengths"] = None
    if c["ragged"]:
        lengths = torch.randint(0, L + 1, (B,), generator=gen, device="cuda")
        lengths[0] = L
        s["lengths"] = lengths.to(torch.int32)
    if c["op"] == "delta_bwd":
        s["dy"] = normal(B, L, H, P).to(dt)
        s["dh_final"] = 0.3 * normal(B, H, N, P) if c["state"] else None
    return s


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    B, L, N = c["batch"], c["seqlen"], c["N"]
    if c["op"] in ("qk", "qk_bwd"):
        values = B * L * (c["q_heads"] + c["k_heads"]) * N
        tensors = 2 if c["op"] == "qk" else 3  # x and the result; x, its result's gradient, its gradient
        extra = (8 * N * (2 if c["op"] == "qk_bwd" else 1) if c["weights"] else 0) + (4 * B * L + 2 * c["rot"] if c["rot"] else 0)
        return {"bytes": values * e * tensors + extra, "flops": values * (8 if c["op"] == "qk" else 16)}
    P, H, Hk, g = c["P"], c["heads"], c["qk_heads"], 2 if c["gates"] == "bf16" else 4
    rows, states = B * L, B * H * N * P * 4
    if c["op"] == "delta":
        byt = rows * (2 * Hk * N + 2 * H * P) * e + rows * H * 2 * g + states * (2 if c["state"] else 1)
        return {"bytes": byt, "flops": rows * H * 6 * N * P}
    byt = rows * (4 * Hk * N + 3 * H * P) * e + rows * H * 4 * g + states * (3 if c["state"] else 0)
    return {"bytes": byt, "flops": rows * H * 16 * N * P}


# --------------------------------------------------------------- plain forms

def _angles(s):
    a = s["positions"].double()[..., None] * s["inv_freq"].double()  # [B, L, rot / 2], in 64 bits: positions are far
    return torch.cos(a).float()[:, :, None], torch.sin(a).float()[:, :, None]


def _turn(x, cos, sin, rot, interleaved):
    """Rotates the first `rot` values of each head."""
    h = rot // 2
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _inverse_norm(x, mode):
    sq = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt((sq / x.shape[-1] if mode == "rms" else sq) + 1e-6)


def _plain_qk(s):
    c, out = s["case"], []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        f = x.float()
        y = f * _inverse_norm(f, c["mode"])
        if w is not None:
            y = y * w
        if c["rot"]:
            y = _turn(y, *_angles(s), c["rot"], c["interleaved"])
        out.append(y.to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _plain_qk_bwd(s):
    c, out = s["case"], {}
    for n, x, w, dy in (("q", s["q"], s["wq"], s["dq_out"]), ("k", s["k"], s["wk"], s["dk_out"])):
        f, d = x.float(), dy.float()
        r = _inverse_norm(f, c["mode"])
        if c["rot"]:
            cos, sin = _angles(s)
            d = _turn(d, cos, -sin, c["rot"], c["interleaved"])
        xhat = f * r
        if w is not None:
            out["dw" + n] = (d * xhat).double().sum((0, 1, 2)).float()
            d = d * w
        dot = (d * xhat).sum(-1, keepdim=True)
        out["d" + n] = (r * (d - xhat * (dot / f.shape[-1] if c["mode"] == "rms" else dot))).to(x.dtype)
    return out


def _chunked(q, k, v, g, beta, h0, lengths, scale):
    """The delta rule by chunks: within one, u solves a triangular system; only the state goes from one to the next."""
    B, L, H, P = v.shape
    N = k.shape[-1]
    q, k = (x.float().repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    v, g, beta = v.float(), g.double(), beta.float()
    if lengths is not None:
        live = torch.arange(L, device=v.device)[None, :, None] < lengths[:, None, None]
        q, k, v = (torch.where(live[..., None], x, 0.0) for x in (q, k, v))
        g, beta = torch.where(live, g, 0.0), torch.where(live, beta, 0.0)
    C = min(CHUNK, L)
    n = -(-L // C)

    def chunks(x):  # [B, L, H, ...] -> [n, B, H, C, ...], zeros behind the end
        pad = x.new_zeros((B, n * C - L) + x.shape[2:])
        x = torch.cat((x, pad), 1).reshape((B, n, C) + x.shape[2:])
        return x.movedim(3, 1).movedim(2, 0) if x.dim() == 4 else x.permute(1, 0, 3, 2, 4)

    q, k, v, g, beta = (chunks(x) for x in (q * scale, k, v, g, beta))
    G = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    kt = k.transpose(-1, -2)
    A = torch.matmul(q, kt) * D
    M = torch.matmul(k, kt) * D * beta[..., None] * low.tril(-1)
    rows = [torch.eye(C, device=v.device)[0].expand(M.shape[:-2] + (C,))]
    for i in range(1, C):  # the inverse of 1 + M, row by row
        T = torch.stack(rows, -2)
        rows.append(torch.eye(C, device=v.device)[i] - torch.matmul(M[..., i:i + 1, :i], T).squeeze(-2))
    T = torch.stack(rows, -2)
    grow, fade, last = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None], torch.exp(G[..., -1]).float()
    u0 = torch.matmul(T, beta[..., None] * v)
    w = torch.matmul(T, beta[..., None] * grow * k)
    qg, kf = q * grow, (k * fade).transpose(-1, -2)
    h = torch.zeros(B, H, N, P, device=v.device) if h0 is None else h0
    ys = []
    for i in range(n):
        u = u0[i] - torch.matmul(w[i], h)
        ys.append(torch.matmul(qg[i], h) + torch.matmul(A[i], u))
        h = last[i][..., None, None] * h + torch.matmul(kf[i], u)
    y = torch.stack(ys).permute(1, 0, 3, 2, 4).reshape(B, n * C, H, P)[:, :L]
    return y, h


def _plain_delta(s):
    y, h = _chunked(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], s["lengths"], s["case"]["N"] ** -0.5)
    return {"y": y.to(s["v"].dtype), "h_final": h}


def _plain_delta_bwd(s):
    names = ["q", "k", "v", "g", "beta"] + (["h0"] if s["h0"] is not None else [])
    x = {n: s[n].double().requires_grad_() if n == "g" else s[n].float().requires_grad_() for n in names}
    with torch.enable_grad():
        y, h = _chunked(x["q"], x["k"], x["v"], x["g"], x["beta"], x.get("h0"), s["lengths"], s["case"]["N"] ** -0.5)
        outs, grads = [y], [s["dy"].float()]
        if s["dh_final"] is not None:
            outs.append(h)
            grads.append(s["dh_final"])
        got = torch.autograd.grad(outs, [x[n] for n in names], grads)
    return {"d" + n: d.to(s[n].dtype) for n, d in zip(names, got)}


# ----------------------------------------------------------------------- run

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import structured_sparse_selective_b200 as pd
        c = s["case"]
        if op in ("qk", "qk_bwd"):
            how = dict(wq=s["wq"], wk=s["wk"], inv_freq=s["inv_freq"], positions=s["positions"], eps=1e-6, mode=c["mode"],
                       interleaved=c["interleaved"])
            if op == "qk":
                return pd.qk_norm(s["q"], s["k"], **how)
            return pd.qk_norm_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], **how)
        if op == "delta":
            return pd.delta_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], lengths=s["lengths"])
        return pd.delta_backward(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dy"], h0=s["h0"], dh_final=s["dh_final"],
                                 lengths=s["lengths"])
    return {"qk": _plain_qk, "qk_bwd": _plain_qk_bwd, "delta": _plain_delta, "delta_bwd": _plain_delta_bwd}[op](s)


# --------------------------------------------------------------------- exact

def _exact_qk(s):
    c, out = s["case"], {}
    rot, h = c["rot"], c["rot"] // 2
    back = c["op"] == "qk_bwd"
    if rot:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[..., None] * s["inv_freq"].double())[:, :, None]
        at = torch.arange(rot, device="cuda").reshape(h, 2) if c["interleaved"] else torch.arange(rot, device="cuda").reshape(2, h).T

    def rotated(x, t):
        if not rot:
            return x
        z = torch.complex(x[..., at[:, 0]], x[..., at[:, 1]]) * t
        x = x.clone()
        x[..., at[:, 0]], x[..., at[:, 1]] = z.real, z.imag
        return x

    for n, x, w in (("q", s["q"].double(), s["wq"]), ("k", s["k"].double(), s["wk"])):
        w = torch.ones(c["N"], device="cuda", dtype=torch.float64) if w is None else w.double()
        share = 1.0 / c["N"] if c["mode"] == "rms" else 1.0
        size = (share * (x ** 2).sum(-1, keepdim=True) + 1e-6).sqrt()
        if not back:
            out[n] = rotated(x / size * w, turn if rot else None)
            continue
        d = rotated(s["d%s_out" % n].double(), turn.conj() if rot else None)
        if c["weights"]:
            out["dw" + n] = (d * x / size).sum((0, 1, 2))
        out["d" + n] = d * w / size - x * share * (d * w * x).sum(-1, keepdim=True) / size ** 3
    return out


def _exact_delta(s, back):
    c = s["case"]
    B, L, H, N, P = c["batch"], c["seqlen"], c["heads"], c["N"], c["P"]
    r = H // c["qk_heads"]
    q, k = (s[n].double().repeat_interleave(r, 2) for n in ("q", "k"))
    q = q * N ** -0.5
    v, a, beta = s["v"].double(), s["g"].double().exp(), s["beta"].double()
    ends = torch.full((B,), L, device="cuda") if s["lengths"] is None else s["lengths"]
    live = (torch.arange(L, device="cuda")[:, None] < ends[None]).tolist()
    on = (torch.arange(L, device="cuda")[:, None] < ends[None])[:, :, None, None, None]
    h = torch.zeros(B, H, N, P, device="cuda", dtype=torch.float64) if s["h0"] is None else s["h0"].double()
    y = torch.zeros(B, L, H, P, device="cuda", dtype=torch.float64)

    def step(h, t):
        """(the faded state, what the value lacks, the new state)"""
        f = a[:, t, :, None, None] * h
        e = v[:, t] - torch.matmul(k[:, t, :, None, :], f).squeeze(-2)
        new = f + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None, :]
        return f, e, new if all(live[t]) else torch.where(on[t], new, h)

    every = 64
    kept = []
    for t in range(L):
        if back and t % every == 0:
            kept.append(h)
        h = step(h, t)[2]
        if not back:
            y[:, t] = torch.matmul(q[:, t, :, None, :], h).squeeze(-2)
    if not back:
        if s["lengths"] is not None:
            y = torch.where(on[:, :, :, 0].transpose(0, 1), y, 0.0)
        return {"y": y, "h_final": h}
    dy = s["dy"].double()
    dq, dk = (torch.zeros(B, L, H, N, device="cuda", dtype=torch.float64) for _ in range(2))
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(beta)
    dh = torch.zeros_like(h) if s["dh_final"] is None else s["dh_final"].double()
    for first in range((L - 1) // every * every, -1, -every):
        hs = [kept.pop()]
        for t in range(first, min(L, first + every)):
            hs.append(step(hs[-1], t)[2])
        for t in range(min(L, first + every) - 1, first - 1, -1):
            f, e, _ = step(hs[t - first], t)
            b = beta[:, t, :, None]
            d = dh + q[:, t, :, :, None] * dy[:, t, :, None, :]
            du = torch.matmul(k[:, t, :, None, :], d).squeeze(-2)
            w = b * du
            gk = torch.matmul(d, (b * e)[..., None]).squeeze(-1) - torch.matmul(f, w[..., None]).squeeze(-1)
            gq = torch.matmul(hs[t - first + 1], dy[:, t, :, :, None]).squeeze(-1)
            m = d - k[:, t, :, :, None] * w[:, :, None, :]
            some = not all(live[t])
            for to, x in ((dq, gq), (dk, gk), (dv, w), (db, (du * e).sum(-1)), (dg, (m * f).sum((-1, -2)))):
                to[:, t] = torch.where(on[t].reshape((B,) + (1,) * (x.dim() - 1)), x, 0.0) if some else x
            m = a[:, t, :, None, None] * m
            dh = torch.where(on[t], m, dh) if some else m
    dq, dk = (x.reshape(B, L, c["qk_heads"], r, N).sum(3) for x in (dq * N ** -0.5, dk))
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": db}
    if s["h0"] is not None:
        out["dh0"] = dh
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("qk", "qk_bwd"):
        return _exact_qk(s)
    return _exact_delta(s, case["op"] == "delta_bwd")
