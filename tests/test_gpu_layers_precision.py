"""The delta rule's fp32 results on the GPU at the precision that they are promised with.

Errors are norms over a (sequence, head)'s slice, relative, in units of 2^-24 (half a step of fp32, the largest relative error of one
rounding; of a norm over many values a rounding makes about 1 / sqrt(3) of it).
"""
import numpy as np
import pytest
import torch

import structured_sparse_selective_b200 as pd
from tests.layers_precision import BOUNDS, UNIT, backward_oracle, gate_terms, slices_off
from tests.test_gpu_layers import delta_case, gradients_in, npy

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def off(got, want):
    """The largest slice's error in units; slices are the leading two dimensions."""
    d, w = (got.double() - want).flatten(2), want.flatten(2)
    return float((d.norm(dim=-1) / w.norm(dim=-1)).max()) / UNIT


# --------------------------------------------------------------- slow decays over long sequences

LONG = 8192


def slow_case(dt, g, N, P, seed=3, L=LONG, H=2):
    """Decays so slow that the state remembers hundreds of chunks: exp(g) is a little off as a float, and is multiplied that often."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    g = torch.full((1, L, H), g, device="cuda") if g is not None else -1e-4 * rand(1, L, H).abs()
    a = dict(q=unit(rand(1, L, H, N)).to(dt), k=unit(rand(1, L, H, N)).to(dt), v=rand(1, L, H, P).to(dt), g=g,
             beta=torch.full((1, L, H), 0.002, device="cuda"))
    return a, rand(1, H, N, P), rand(1, L, H, P).to(dt), rand(1, H, N, P)


def last_state(a, h):
    k, v, f, b = a["k"].double(), a["v"].double(), a["g"].double().exp(), a["beta"].double()
    h = h.double()
    for t in range(v.shape[1]):
        h = f[:, t, :, None, None] * h
        e = v[:, t] - torch.matmul(k[:, t, :, None, :], h).squeeze(-2)
        h = h + k[:, t, :, :, None] * (b[:, t, :, None] * e)[:, :, None, :]
    return h


def first_adjoint(a, dy, x):
    q, k, f, b = a["q"].double() * a["q"].shape[-1] ** -0.5, a["k"].double(), a["g"].double().exp(), a["beta"].double()
    dy, x = dy.double(), x.double()
    for t in range(dy.shape[1] - 1, -1, -1):
        x = x + q[:, t, :, :, None] * dy[:, t, :, None, :]
        dv = b[:, t, :, None] * torch.matmul(k[:, t, :, None, :], x).squeeze(-2)
        x = f[:, t, :, None, None] * (x - k[:, t, :, :, None] * dv[:, :, None, :])
    return x


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,P", [(32, 32), (96, 80)])
@pytest.mark.parametrize("g", [-1e-4, -3e-4, None])
def test_slow_decays_by_chunks(dt, N, P, g):
    """A chunk multiplies the state once: with a factor that is off by a float's half step, 128 chunks would be off by up to 128 units.
    With an exact one there are two roundings a chunk, 0.6 sqrt(2 x 128) = 9 units, and those of one chunk's products, 5; three times
    that. (16 chunks or more are in memory.)"""
    a, h0, dy, dh = slow_case(dt, g, N, P)
    with pd.KernelTrace() as tr:
        got, back = pd.delta_forward(**a, h0=h0), pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)
    assert not any("steps" in n for n in tr.names)
    assert off(got["h_final"], last_state(a, h0)) <= 32
    assert off(back["dh0"], first_adjoint(a, dy, dh)) <= 32


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("N,P", [(32, 32), (96, 80)])
@pytest.mark.parametrize("g", [-1e-4, -3e-4, None])
def test_slow_decays_by_steps(dt, N, P, g):
    """A factor that is off by a float's half step would be off by up to 8,192 units. Two roundings a step are 0.6 sqrt(2 x 8,192) = 74
    units where they are independent; those of neighbouring steps are not, since the state changes little: eight times that."""
    a, h0, dy, dh = slow_case(dt, g, N, P)
    got = pd.delta_forward(**a, h0=h0, flags=pd.FLAG_REFERENCE_PATH)
    back = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=pd.FLAG_REFERENCE_PATH)
    assert off(got["h_final"], last_state(a, h0)) <= 592
    assert off(back["dh0"], first_adjoint(a, dy, dh)) <= 592


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("g", [-1e-4, -1.3e-4, -1.7e-4])
def test_slow_decays_by_short_segments(dt, g):
    """Four steps a call, 2,000 calls: eight times 0.6 sqrt(2 x 8,000) as by steps (a rounding that is the same in each call would be
    off by up to 8,000 units)."""
    a, h0, _, _ = slow_case(dt, g, 64, 64, L=8000, H=1)
    state = h0.clone()
    for t in range(0, 8000, 4):
        pd.delta_forward(**{n: x[:, t:t + 4].contiguous() for n, x in a.items()}, h0=state, h_final=state)
    assert off(state, last_state(a, h0)) <= 600


@pytest.mark.parametrize("dt", [BF16, F32])
def test_slow_decays_token_by_token(dt):
    """As by steps, 2,000 of them: eight times 0.6 sqrt(2 x 2,000)."""
    a, h0, _, _ = slow_case(dt, -1e-4, 64, 64, L=2000)
    state, tokens = h0.clone(), [{n: x[:, t:t + 1].contiguous() for n, x in a.items()} for t in range(2000)]
    for tok in tokens:
        pd.delta_forward(**tok, h0=state, h_final=state)
    assert off(state, last_state(a, h0)) <= 300


# --------------------------------------------------------------- gradients of the gates where decays are strong

PATHS = [(BF16, 300, 0), (BF16, 6, 0), (F32, 300, 0), (F32, 40, 0), (BF16, 150, pd.FLAG_REFERENCE_PATH)]


@pytest.mark.parametrize("gates", [F32, BF16])
@pytest.mark.parametrize("dt,L,flags", PATHS)
def test_a_dropped_states_gate_has_no_gradient(dt, L, flags, gates):
    a, h0 = delta_case((2, L, 2, 4, 64, 48), dt, gates)
    dy, dh = gradients_in(a)
    at = sorted({0, 1, L // 2, L - 1, min(63, L - 1), min(64, L - 1)})
    a["g"][:, at[::2]] = -float("inf")
    a["g"][:, at[1::2]] = -150.0
    got = pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=flags)
    assert not got["dg"][:, at].any()
    assert not got["dh0"].any()  # the first step drops it


@pytest.mark.parametrize("bias", [0.0, 3.0, 10.0, 30.0])
def test_gates_gradients_on_the_tensor_cores_against_their_terms(bias):
    a, h0 = delta_case((1, 300, 1, 2, 64, 64), BF16, bias=bias)
    dy, dh = gradients_in(a)
    y, h, want = backward_oracle(a, h0, dy, dh)
    got = npy(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)["dg"])
    M = gate_terms(a, h0, y, want, dy, dh, 64)
    for i in range(2):
        assert np.linalg.norm((got - want["dg"])[0, :, i]) <= BOUNDS["dg"] * UNIT * np.linalg.norm(M[0, :, i])


@pytest.mark.parametrize("bias", [3.0, 10.0, 30.0])
@pytest.mark.parametrize("dt,L,flags", [p for p in PATHS if p[:2] != (BF16, 300)])
def test_gates_gradients_where_every_term_decays_are_exact_relatively(dt, L, flags, bias):
    """The other paths sum terms that have the factor. An exponent of size |g| is off by |g| units and a term with it, its products by
    some 8; a step's sum has the later steps' of its chunk of 32 too, which cancel up to their rounding. A step's terms are up to three
    times their sum."""
    a, h0 = delta_case((1, L, 1, 2, 64, 64), dt, bias=bias)
    dy, dh = gradients_in(a)
    want = backward_oracle(a, h0, dy, dh)[2]["dg"]
    got = npy(pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=flags)["dg"])
    size = float(a["g"].abs().max())
    for i in range(2):
        w = np.abs(want[0, :, i])
        M = np.concatenate([w[t:t + 32][::-1].cumsum()[::-1] for t in range(0, L, 32)])
        assert np.linalg.norm((got - want)[0, :, i]) <= 3 * (8 + size) * UNIT * np.linalg.norm(M)


# --------------------------------------------------------------- states and gates' gradients on every path

CASES = [  # batch, seqlen, qk_heads, heads, N, P: the tensor cores' four kernels, with states and adjoints in one launch and in two
    (1, 600, 1, 2, 64, 64), (1, 300, 1, 2, 128, 128), (2, 200, 1, 2, 96, 48), (1, 200, 2, 2, 40, 100), (5, 130, 4, 16, 64, 64),
    (5, 130, 4, 16, 72, 80), (1, 40, 1, 2, 64, 64), (1, 8, 1, 2, 64, 64), (6, 100, 8, 16, 32, 32),
]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("bias", [-2.5, -8.0])
def test_fp32_results_are_exact_to_fp32(c, dt, bias):
    a, h0 = delta_case(c, dt, bias=bias)
    dy, dh = gradients_in(a)
    y, h, want = backward_oracle(a, h0, dy, dh)
    got = {n: npy(x) for n, x in (pd.delta_forward(**a, h0=h0) | pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh)).items()}
    for n, x in slices_off(got, h, want, gate_terms(a, h0, y, want, dy, dh, 64)).items():
        assert x <= BOUNDS[n], (n, x)
