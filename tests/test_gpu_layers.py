"""The layers beside the scan on the GPU against their oracles in 64 bits.

Tolerances. A result of 8, 11 or 24 bits is off by half a step of its type, eps / 2 relative to the value, whatever computes
it. Before that rounding the kernels work in fp32: a result that went through n roundings of independent sign, none of whose
operands is larger than S, is off by about sqrt(n) 2^-24 S; 8 standard deviations are allowed. For a head of N values n = N; for
the delta rule n = N L (each step's dot product of N terms enters the state once and is never enlarged: with |k| = 1 and
0 <= beta <= 1 a step's matrix has norm <= 1), and for a sum over P columns or r shared heads n = N P L r. S is the largest value
of the result's (sequence, head) slice, or 1 where that is less (the inputs are of that size).
"""
import numpy as np
import pytest
import torch

import structured_sparse_selective_b200 as pd
from oracle import layers

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.bfloat16]


def npy(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, want, n, unit=2.0 ** -24, axes=None, operands=1.0):
    """|got - want| <= half a step of got's type + 8 sqrt(n) unit S, S over `axes` (a slice's) at least `operands`."""
    g = npy(got)
    assert g.shape == want.shape, name
    S = np.maximum(operands, np.abs(want).max(axis=axes, keepdims=True)) if want.size else 1.0
    lim = HALF[got.dtype] * np.abs(want) + 8 * np.sqrt(n) * unit * S
    bad = ~(np.abs(g - want) <= lim)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.abs(g - want)[bad].max():.3g} at limit {np.broadcast_to(lim, g.shape)[bad].min():.3g}"


def randn(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).normal(size=shape)).float()


# ------------------------------------------------------------------- q / k norm

NORM = [  # batch, seqlen, q_heads, k_heads, N, rot, interleaved, mode
    (1, 1, 1, 1, 64, 64, False, "rms"), (2, 3, 5, 2, 64, 32, False, "l2"), (2, 37, 4, 4, 128, 128, True, "rms"),
    (1, 9, 3, 1, 80, 36, True, "l2"), (1, 9, 3, 1, 80, 40, False, "rms"), (2, 5, 2, 3, 7, 6, False, "rms"),
    (2, 5, 2, 3, 7, 4, True, "l2"), (1, 1300, 2, 1, 32, 16, False, "rms"), (3, 2, 1, 2, 1, 0, False, "rms"),
    (1, 4, 2, 2, 96, 6, False, "rms"), (1, 2, 33, 1, 128, 0, False, "l2"), (1, 3, 2, 2, 12, 12, True, "rms"),
    (2, 3, 0, 2, 16, 8, False, "rms"),
]


def norm_case(c, dt, seed=0, weights=True, far=True):
    Bt, L, Hq, Hk, N, rot, interleaved, mode = c
    q, k = randn(seed, Bt, L, Hq, N).to(dt).cuda(), (3 * randn(seed + 1, Bt, L, Hk, N)).to(dt).cuda()
    kw = dict(wq=1 + 0.2 * randn(seed + 2, N).cuda() if weights else None, wk=randn(seed + 3, N).cuda() if weights else None,
              inv_freq=(10000.0 ** (-torch.arange(0, rot, 2).double() / rot)).float().cuda() if rot else None,
              positions=torch.from_numpy(np.random.default_rng(seed).integers(0, 10 ** 6, (Bt, L))).int().cuda() if far else None,
              eps=1e-6, mode=mode, interleaved=interleaved)
    return q, k, kw


def norm_oracle(x, kw, w, dy=None):
    args = (npy(x), npy(kw[w]), npy(kw["inv_freq"]), None if kw["positions"] is None else kw["positions"].cpu().numpy(), kw["eps"],
            kw["mode"], kw["interleaved"])
    return layers.qk_norm(*args) if dy is None else layers.qk_norm_backward(*args, npy(dy))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", NORM)
@pytest.mark.parametrize("weights,far", [(True, True), (False, False)])
def test_qk_norm(c, dt, weights, far):
    q, k, kw = norm_case(c, dt, weights=weights, far=far)
    out = pd.qk_norm(q, k, **kw)
    for n, x in (("q", q), ("k", k)):
        assert out[n].dtype == dt
        close(n, out[n], norm_oracle(x, kw, "w" + n), c[4])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", NORM)
@pytest.mark.parametrize("weights,far", [(True, True), (False, False)])
def test_qk_norm_backward(c, dt, weights, far):
    q, k, kw = norm_case(c, dt, seed=7, weights=weights, far=far)
    dq, dk = randn(11, *q.shape).to(dt).cuda(), randn(12, *k.shape).to(dt).cuda()
    out = pd.qk_norm_backward(q, k, dq, dk, **kw)
    assert set(out) == ({"dq", "dk", "dwq", "dwk"} if weights else {"dq", "dk"})
    for n, x, d in (("q", q, dq), ("k", k, dk)):
        dx, dw = norm_oracle(x, kw, "w" + n, d)
        # dx = d w / s - x (sum of d w x) share / s^3: two terms of up to sqrt(2) |d| |w| / s (a turned pair is at most sqrt(2)
        # larger than its larger value), s = sqrt(share |x|^2 + eps), whose difference can be far smaller than their roundings
        # (a head of one value: it is 0 but for eps), so S is the terms' size
        xs = npy(x)
        s = np.sqrt((xs ** 2).sum(-1, keepdims=True) / (c[4] if c[7] == "rms" else 1) + kw["eps"])
        w = 1.0 if kw["w" + n] is None else np.abs(npy(kw["w" + n])).max()
        terms = np.sqrt(2) * np.abs(npy(d)).max(-1, keepdims=True) * w / s
        close("d" + n, out["d" + n], dx, c[4], axes=(-1,), operands=np.maximum(1.0, terms) if x.numel() else 1.0)
        if weights:  # a sum over all tokens and heads
            close("dw" + n, out["dw" + n], dw, max(1, x.numel()))


def test_qk_norm_at_unaligned_pointers_and_in_place():
    c = (2, 5, 4, 4, 64, 64, False, "rms")
    for dt in TYPES:
        q, k, kw = norm_case(c, dt)
        want = pd.qk_norm(q, k, **kw)
        room = torch.empty(q.numel() + 1, dtype=dt, device="cuda")[1:].view(q.shape)  # one value behind an aligned address
        room.copy_(q)
        got = pd.qk_norm(room, k, **kw)
        close("q", got["q"], npy(want["q"]), 64)
        pd.qk_norm(q, k, **kw, q_out=q, k_out=k)
        assert torch.equal(q, want["q"]) and torch.equal(k, want["k"])


def test_qk_norm_of_nothing():
    for shape in ((0, 3, 2, 8), (2, 0, 2, 8)):
        q, w = torch.empty(shape, device="cuda"), torch.ones(8, device="cuda")
        assert pd.qk_norm(q, q.clone(), wq=w)["q"].shape == shape
        out = pd.qk_norm_backward(q, q, q, q, wq=w, wk=w)
        assert not out["dwq"].any() and not out["dwk"].any()


def test_qk_norm_infinities_stay_in_their_heads():
    q = randn(1, 1, 4, 4, 64).cuda()
    want = pd.qk_norm(q, q)["q"]
    bad = q.clone()
    bad[0, 1, 2, 5] = float("inf")
    bad[0, 2, 0, 9] = float("nan")
    got = pd.qk_norm(bad, q)["q"]
    keep = torch.ones(4, 4, dtype=torch.bool, device="cuda")
    keep[1, 2] = keep[2, 0] = False
    assert torch.equal(got[0][keep], want[0][keep]) and not torch.isfinite(got[0, 2, 0]).any()


# ---------------------------------------------------------------- gated delta rule

DELTA = [  # batch, seqlen, qk_heads, heads, N, P
    (1, 1, 1, 1, 64, 64), (3, 1, 2, 4, 128, 64), (1, 2, 1, 1, 1, 1), (2, 15, 1, 2, 16, 16), (1, 16, 1, 1, 33, 17),
    (1, 17, 2, 2, 64, 64), (2, 31, 1, 3, 5, 7), (1, 32, 1, 1, 128, 128), (1, 33, 1, 2, 40, 24), (1, 63, 1, 1, 64, 128),
    (2, 64, 1, 1, 32, 32), (1, 65, 2, 2, 64, 64), (1, 127, 1, 1, 127, 125), (1, 128, 1, 1, 64, 64), (1, 129, 1, 2, 128, 128),
    (1, 200, 1, 2, 96, 80), (2, 257, 1, 1, 64, 3), (1, 300, 1, 1, 8, 128), (1, 333, 1, 1, 110, 64),
]


def delta_case(c, dt, gates=torch.float32, seed=0, state=True, bias=-2.5):
    Bt, L, Hk, H, N, P = c
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(q=unit(randn(seed, Bt, L, Hk, N)).to(dt), k=unit(randn(seed + 1, Bt, L, Hk, N)).to(dt), v=randn(seed + 2, Bt, L, H, P).to(dt),
             g=-torch.nn.functional.softplus(randn(seed + 3, Bt, L, H) + bias).to(gates), beta=torch.sigmoid(randn(seed + 4, Bt, L, H)).to(gates))
    a = {n: x.cuda() for n, x in a.items()}
    return a, randn(seed + 5, Bt, H, N, P).cuda() if state else None


def delta_oracle(a, h0, lengths=None, scale=None, dy=None, dh=None):
    x = [npy(a[n]) for n in ("q", "k", "v", "g", "beta")]
    scale = a["q"].shape[-1] ** -0.5 if scale is None else scale
    lengths = None if lengths is None else lengths.cpu().numpy()
    if dy is None:
        return layers.delta(*x, npy(h0), scale, lengths)
    return layers.delta_backward(*x, npy(h0), scale, lengths, npy(dy), npy(dh))


def check_forward(out, a, h0, lengths=None, scale=None):
    y, h = delta_oracle(a, h0, lengths, scale)
    L, N = a["q"].shape[1], a["q"].shape[3]
    close("y", out["y"], y, N * L, axes=(1, 3))
    close("h_final", out["h_final"], h, N * L, axes=(2, 3))


def check_backward(out, a, h0, dy, dh, lengths=None, scale=None):
    want = delta_oracle(a, h0, lengths, scale, dy, dh)
    L, Hk, N = a["q"].shape[1:]
    H, P = a["v"].shape[2:]
    n = N * P * L * (H // Hk)
    for name, d in out.items():
        close(name, d, want[name], n, axes=tuple(i for i in range(want[name].ndim) if i not in ((0, 1) if name == "dh0" else (0, 2))))


def gradients_in(a, state=True, seed=50):
    dy = randn(seed, *a["v"].shape).to(a["v"].dtype).cuda()
    Bt, _, H, P = a["v"].shape
    return dy, randn(seed + 1, Bt, H, a["q"].shape[-1], P).cuda() if state else None


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", DELTA)
def test_delta_forward(c, dt):
    a, h0 = delta_case(c, dt)
    check_forward(pd.delta_forward(**a, h0=h0), a, h0)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", DELTA)
def test_delta_backward(c, dt):
    a, h0 = delta_case(c, dt)
    dy, dh = gradients_in(a)
    check_backward(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh), a, h0, dy, dh)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("gates", TYPES)
@pytest.mark.parametrize("bias", [-30.0, 0.0, 30.0])
def test_delta_gates_from_no_decay_to_full_decay(dt, gates, bias):
    a, h0 = delta_case((1, 150, 1, 2, 64, 48), dt, gates, bias=bias)
    dy, dh = gradients_in(a)
    check_forward(pd.delta_forward(**a, h0=h0, scale=0.5), a, h0, scale=0.5)
    check_backward(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, scale=0.5), a, h0, dy, dh, scale=0.5)


@pytest.mark.parametrize("dt", TYPES)
def test_delta_without_states(dt):
    a, _ = delta_case((2, 70, 1, 2, 64, 64), dt)
    dy, _ = gradients_in(a)
    check_forward(pd.delta_forward(**a), a, None)
    assert set(pd.delta_forward(**a, want_h_final=False)) == {"y"}
    out = pd.delta_backward(**a, dy=dy)
    assert "dh0" not in out
    check_backward(pd.delta_backward(**a, dy=dy, want_dh0=True), a, None, dy, None)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("L", [1, 40, 200, 300])
def test_delta_lengths_leave_the_padding_out(dt, L):
    c = (5, L, 1, 2, 64, 40)
    a, h0 = delta_case(c, dt)
    dy, dh = gradients_in(a)
    lengths = torch.tensor([L, 0, (L + 1) // 2, -3, L + 7], dtype=torch.int32, device="cuda")
    want = delta_oracle(a, h0, lengths)
    dirty = {n: x.clone() for n, x in a.items()}
    dirty_dy = dy.clone()
    for b, n in enumerate(lengths.tolist()):
        for x in (*dirty.values(), dirty_dy):
            x[b, max(0, n):] = float("nan")
    out = pd.delta_forward(**dirty, h0=h0, lengths=lengths)
    close("y", out["y"], want[0], 64 * L, axes=(1, 3))
    close("h_final", out["h_final"], want[1], 64 * L, axes=(2, 3))
    assert torch.equal(out["h_final"][1], h0[1]) and torch.equal(out["h_final"][3], h0[3])
    got = pd.delta_backward(**dirty, dy=dirty_dy, h0=h0, dh_final=dh, lengths=lengths)
    check_backward(got, a, h0, dy, dh, lengths)
    assert torch.equal(got["dh0"][1], dh[1])
    for b, n in enumerate(lengths.tolist()):
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            assert not got[name][b, max(0, n):].any(), name


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("L", [3, 90, 150, 300])
def test_delta_gates_of_minus_infinity_drop_the_state(dt, L):
    a, h0 = delta_case((1, L, 1, 2, 64, 64), dt)
    a["g"][:, L // 2] = -float("inf")
    out = pd.delta_forward(**a, h0=h0)
    check_forward(out, a, h0)
    dy, dh = gradients_in(a)
    got = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    check_backward(got, a, h0, dy, dh)
    tail = {n: x[:, L // 2:].contiguous() for n, x in a.items()}
    y, h = delta_oracle(tail, None)
    close("y", out["y"][:, L // 2:], y, 64 * L, axes=(1, 3))


@pytest.mark.parametrize("dt", TYPES)
def test_delta_segments_and_tokens_make_the_whole(dt):
    a, h0 = delta_case((2, 100, 2, 2, 64, 64), dt)
    whole = pd.delta_forward(**a, h0=h0)
    y, h = delta_oracle(a, h0)
    for cuts in ([0, 37, 100], list(range(101))):
        state, ys = h0.clone(), []
        for i, j in zip(cuts, cuts[1:]):
            ys.append(pd.delta_forward(**{n: x[:, i:j].contiguous() for n, x in a.items()}, h0=state, h_final=state)["y"])
        close("y", torch.cat(ys, 1), y, 6400, axes=(1, 3))
        close("h_final", state, h, 6400, axes=(2, 3))
    close("h_final", whole["h_final"], h, 6400, axes=(2, 3))


def test_delta_of_nothing():
    for Bt, L in ((0, 4), (2, 0)):
        a, h0 = delta_case((Bt, L, 1, 2, 8, 8), torch.float32)
        out = pd.delta_forward(**a, h0=h0)
        assert out["y"].shape == a["v"].shape and torch.equal(out["h_final"], h0)
        assert not pd.delta_forward(**a)["h_final"].any()
        dy, dh = gradients_in(a)
        got = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
        assert torch.equal(got["dh0"], dh)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("L", [1, 150, 300])
def test_delta_in_graphs_on_streams_and_twice(dt, L):
    a, h0 = delta_case((2, L, 1, 2, 64, 64), dt)
    dy, dh = gradients_in(a)
    want, wantb = pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    again = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    for n in wantb:  # no order that changes: the same bits
        assert torch.equal(wantb[n], again[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, outb = pd.delta_forward(**a, h0=h0, stream=side), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, stream=side)
    side.synchronize()
    assert torch.equal(out["y"], want["y"]) and all(torch.equal(outb[n], wantb[n]) for n in wantb)
    # two captured graphs, replayed side by side: each has workspaces of its own
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append((pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)))
    for x in a.values():
        x.copy_(x.flip(0))
    new, newb = pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    for f, b in outs:
        assert torch.equal(f["y"], new["y"]) and torch.equal(f["h_final"], new["h_final"])
        assert all(torch.equal(b[n], newb[n]) for n in newb)


def test_delta_traced_launches_name_their_kernels():
    a, h0 = delta_case((1, 20, 1, 1, 64, 64), torch.float32)
    with pd.KernelTrace() as tr:
        pd.delta_forward(**a, h0=h0)
        pd.delta_backward(**a, dy=gradients_in(a)[0], h0=h0)
    torch.cuda.synchronize()
    assert [n for n, _ in tr.timings()] == ["delta_steps", "delta_steps_both", "delta_grad"] and all(ms > 0 for _, ms in tr.timings())


@pytest.mark.parametrize("dt", TYPES)
def test_a_layer_and_its_gradients_together(dt):
    """Projected queries and keys -> norm and rotation -> delta rule -> gradients back through both."""
    Bt, L, Hk, H, N, P = 2, 90, 2, 4, 64, 32
    q, k, kw = norm_case((Bt, L, Hk, Hk, N, 32, False, "l2"), dt, weights=False)
    a, h0 = delta_case((Bt, L, Hk, H, N, P), dt)
    qk = pd.qk_norm(q, k, **kw)
    a["q"], a["k"] = qk["q"], qk["k"]
    out = pd.delta_forward(**a, h0=h0)
    check_forward(out, a, h0)
    dy, dh = gradients_in(a)
    d = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    check_backward(d, a, h0, dy, dh)
    dx = pd.qk_norm_backward(q, k, d["dq"], d["dk"], **kw)
    for n, x in (("q", q), ("k", k)):
        close("d" + n, dx["d" + n], norm_oracle(x, kw, "w" + n, d["d" + n])[0], N, axes=(-1,))
    # the next token from the state that the segment left
    nxt = {n: x[:, :1].contiguous() for n, x in a.items()}
    check_forward(pd.delta_forward(**nxt, h0=out["h_final"].clone()), nxt, out["h_final"])


# ------------------------------------------------------- paths, pointers, sizes and failures

PATHS = [  # batch, seqlen, qk_heads, heads, N, P: short and long runs with few blocks and with more than the SMs
    (1, 9, 1, 1, 64, 64), (2, 12, 1, 2, 32, 16), (1, 41, 2, 2, 64, 64), (37, 13, 4, 16, 16, 8), (37, 12, 8, 16, 8, 4),
    (5, 70, 4, 16, 64, 64), (5, 66, 4, 16, 64, 72), (5, 64, 8, 16, 72, 64), (3, 130, 2, 26, 65, 66),
    (5, 100, 4, 16, 72, 64), (9, 100, 4, 16, 64, 64), (4, 260, 4, 16, 40, 128), (4, 260, 8, 16, 24, 100), (2, 260, 1, 1, 32, 33),
]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", PATHS)
def test_delta_on_every_path(c, dt):
    a, h0 = delta_case(c, dt, seed=21)
    check_forward(pd.delta_forward(**a, h0=h0), a, h0)
    dy, dh = gradients_in(a)
    check_backward(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh), a, h0, dy, dh)


@pytest.mark.parametrize("dt", TYPES)
def test_delta_by_the_reference_path(dt):
    a, h0 = delta_case((2, 150, 1, 2, 64, 40), dt)
    dy, dh = gradients_in(a)
    with pd.KernelTrace() as tr:
        check_forward(pd.delta_forward(**a, h0=h0, flags=pd.FLAG_REFERENCE_PATH), a, h0)
        check_backward(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=pd.FLAG_REFERENCE_PATH), a, h0, dy, dh)
    assert tr.names == ["delta_steps", "delta_steps_both", "delta_grad"]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("L", [1, 11, 150, 300])
def test_delta_at_unaligned_pointers(dt, L):
    a, h0 = delta_case((2, L, 1, 2, 64, 64), dt)
    dy, dh = gradients_in(a)

    def moved(x):  # one value behind an aligned address
        room = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
        return room.copy_(x)

    am, hm = {n: moved(x) for n, x in a.items()}, moved(h0)
    check_forward(pd.delta_forward(**am, h0=hm, h_final=hm), a, h0)
    hm = moved(h0)
    check_backward(pd.delta_backward(**am, dy=moved(dy), h0=hm, dh_final=moved(dh)), a, h0, dy, dh)
    # outputs too, through the entry points that take them
    pb = pd._delta_problem(*(a[n] for n in ("q", "k", "v", "g", "beta")), h0, None, None, 0)[0]
    ws = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    y, hf = moved(a["v"]), moved(h0)
    ins = [am[n] for n in ("q", "k", "v", "g", "beta")]
    pd.pdssm_delta_fwd(pb, *ins, None, h0, y, hf, ws(pd.pdssm_delta_workspace_size(pb)))
    check_forward({"y": y, "h_final": hf}, a, h0)
    out = {"d" + n: moved(a[n]) for n in ("q", "k", "v", "g", "beta")} | {"dh0": moved(h0)}
    pd.pdssm_delta_bwd(pb, *ins, None, h0, dy, dh, *out.values(), ws(pd.pdssm_delta_bwd_workspace_size(pb)))
    check_backward(out, a, h0, dy, dh)


@pytest.mark.parametrize("what", ["forward", "backward"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", [(2, 600, 1, 2, 64, 64), (2, 600, 1, 2, 128, 128), (5, 300, 2, 16, 128, 64), (1, 300, 1, 1, 8, 2)])
def test_delta_short_waits_report_a_timeout_and_the_next_call_is_clean(c, dt, what):
    """The chunk kernels' waits of one role on another are bounded: with waits of a microsecond some run out, which is
    reported, ends the call and leaves the device and the next call as they were."""
    a, h0 = delta_case(c, dt)
    dy, dh = gradients_in(a)
    pb = pd._delta_problem(*(a[n] for n in ("q", "k", "v", "g", "beta")), h0, None, None, 0)[0]
    size = pd.pdssm_delta_workspace_size(pb) if what == "forward" else pd.pdssm_delta_bwd_workspace_size(pb)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def call(flags):
        if what == "forward":
            return pd.delta_forward(**a, h0=h0, flags=flags, workspace=ws)
        return pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=flags, workspace=ws)

    clean = call(0)
    assert pd.pdssm_read_device_check(ws) == 0
    for _ in range(3):
        call(pd.FLAG_SHORT_WAITS)
        assert pd.pdssm_read_device_check(ws) == 6
    again = call(0)
    assert pd.pdssm_read_device_check(ws) == 0
    for n in clean:
        assert torch.equal(again[n], clean[n]), n


def test_delta_error_word_of_a_path_without_waits():
    a, h0 = delta_case((1, 20, 1, 1, 16, 16), torch.float32)
    pb = pd._delta_problem(*(a[n] for n in ("q", "k", "v", "g", "beta")), h0, None, None, 0)[0]
    ws = torch.full((pd.pdssm_delta_bwd_workspace_size(pb),), 255, dtype=torch.uint8, device="cuda")
    dy, dh = gradients_in(a)
    check_backward(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, workspace=ws, flags=pd.FLAG_SHORT_WAITS), a, h0, dy, dh)
    assert pd.pdssm_read_device_check(ws) == 0


@pytest.mark.parametrize("dt", TYPES)
def test_delta_values_that_are_not_finite_stay_in_their_sequences_and_heads(dt):
    a, h0 = delta_case((3, 300, 1, 2, 64, 32), dt)
    dy, dh = gradients_in(a)
    want, wantb = pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    a["v"][1, 70, 1, 3] = float("nan")
    a["k"][2, 3] = float("inf")
    got, gotb = pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    torch.cuda.synchronize()
    assert torch.equal(got["y"][0], want["y"][0]) and torch.equal(got["y"][1, :, 0], want["y"][1, :, 0])
    keep = torch.arange(32, device="cuda") != 3  # a value's column keeps to itself
    assert torch.equal(got["y"][1, :, 1][:, keep], want["y"][1, :, 1][:, keep]) and got["y"][1, 71:, 1, 3].isnan().all()
    assert torch.equal(got["h_final"][0], want["h_final"][0])
    for n in wantb:
        assert torch.equal(gotb[n][0], wantb[n][0]), n
    assert torch.equal(gotb["dv"][1, :, 0], wantb["dv"][1, :, 0])


@pytest.mark.parametrize("dt,N,flags", [(torch.bfloat16, 16, 0), (torch.float32, 16, pd.FLAG_REFERENCE_PATH), (torch.float32, 72, 0)])
def test_delta_offsets_beyond_32_bits(dt, N, flags):
    """More than 2^31 values: the last sequence is the same, bit for bit, as it is alone (each case takes one path at any size)."""
    Bt, L, Hk, H, P = 65, 2049, 1, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen, dtype=dt)  # noqa: E731
    a = dict(q=N ** -0.5 * rand(Bt, L, Hk, N), k=N ** -0.5 * rand(Bt, L, Hk, N), v=rand(Bt, L, H, P), g=-0.05 * rand(Bt, L, H).abs(),
             beta=torch.sigmoid(rand(Bt, L, H)))
    assert a["v"].numel() > 2 ** 31
    dy = rand(Bt, L, H, P)
    last = {n: x[-1:].contiguous() for n, x in a.items()}
    out, alone = pd.delta_forward(**a, flags=flags), pd.delta_forward(**last, flags=flags)
    assert torch.equal(out["y"][-1], alone["y"][0]) and torch.equal(out["h_final"][-1], alone["h_final"][0])
    del out
    out, alone = pd.delta_backward(**a, dy=dy, flags=flags), pd.delta_backward(**last, dy=dy[-1:].contiguous(), flags=flags)
    for n in alone:
        assert torch.equal(out[n][-1], alone[n][0]), n
    del out, a, dy
    torch.cuda.empty_cache()


def test_qk_norm_of_many_heads_and_offsets_beyond_32_bits():
    # more heads than a block goes through at once
    q, k, kw = norm_case((1, 2, 4500, 4099, 16, 8, False, "rms"), torch.float32)
    out, back = pd.qk_norm(q, k, **kw), pd.qk_norm_backward(q, k, q, k, **kw)
    for n, x in (("q", q), ("k", k)):
        close(n, out[n], norm_oracle(x, kw, "w" + n), 16)
        dx, dw = norm_oracle(x, kw, "w" + n, x)
        xs = npy(x)  # S: the size of dx's two terms, as above
        terms = np.sqrt(2) * np.abs(xs).max(-1, keepdims=True) * np.abs(npy(kw["w" + n])).max() / np.sqrt((xs ** 2).mean(-1, keepdims=True))
        close("d" + n, back["d" + n], dx, 16, axes=(-1,), operands=np.maximum(1.0, terms))
        close("dw" + n, back["dw" + n], dw, x.numel())
    big = torch.randn(1, 2 ** 20 + 1, 16, 128, device="cuda", dtype=torch.bfloat16)
    assert big.numel() > 2 ** 31
    k, w = big[:, :, :1].contiguous(), torch.rand(128, device="cuda") + 0.5
    freq, pos = torch.rand(32, device="cuda") * 0.1, torch.arange(2 ** 20 + 1, device="cuda", dtype=torch.int32)[None]
    kw = dict(inv_freq=freq, wq=w)
    out = pd.qk_norm(big, k, positions=pos, **kw)
    alone = pd.qk_norm(big[:, -1:].contiguous(), k[:, -1:].contiguous(), positions=pos[:, -1:].contiguous(), **kw)
    assert torch.equal(out["q"][:, -1:], alone["q"]) and torch.equal(out["k"][:, -1:], alone["k"])
    del out
    back = pd.qk_norm_backward(big, k, big, k, positions=pos, **kw)
    alone = pd.qk_norm_backward(big[:, -1:].contiguous(), k[:, -1:].contiguous(), big[:, -1:].contiguous(), k[:, -1:].contiguous(),
                                positions=pos[:, -1:].contiguous(), **kw)
    assert torch.equal(back["dq"][:, -1:], alone["dq"]) and torch.equal(back["dk"][:, -1:], alone["dk"])
    del back, big
    torch.cuda.empty_cache()
