"""The bounds on the delta rule's fp32 results hold for three bf16 parts of what is fp32, as the tensor-core path takes them, and do
not for two: by a model of that path on the CPU."""
import pytest
import torch

from tests import chunk_parts_ref
from tests.layers_precision import BOUNDS, backward_oracle, gate_terms, slices_off

CASES = [(200, 64, 64, -2.5), (200, 128, 48, -2.5), (300, 64, 64, -8.0), (130, 32, 100, 0.0)]


def case(L, N, P, bias, seed):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    a = dict(q=unit(rand(1, L, 1, N)).bfloat16(), k=unit(rand(1, L, 1, N)).bfloat16(), v=rand(1, L, 1, P).bfloat16(),
             g=-torch.nn.functional.softplus(rand(1, L, 1) + bias), beta=torch.sigmoid(rand(1, L, 1)))
    return a, rand(1, 1, N, P), rand(1, L, 1, P).bfloat16(), rand(1, 1, N, P)


@pytest.mark.parametrize("c", CASES)
def test_three_parts_are_within_the_bounds_and_two_are_not(c):
    largest = {2: {}, 3: {}}
    for seed in (1, 2, 3):
        a, h0, dy, dh = case(*c, seed)
        y, h, want = backward_oracle(a, h0, dy, dh)
        terms = gate_terms(a, h0, y, want, dy, dh, 64)
        one = {n: x[0, :, 0] for n, x in a.items()}
        for n in (2, 3):
            got = chunk_parts_ref.delta(**one, h0=h0[0, 0], scale=c[1] ** -0.5, dy=dy[0, :, 0], dh=dh[0, 0], n=n)
            got = {k: x.double().numpy()[(None, None) if x.dim() == 2 else (None, slice(None), None)] for k, x in got.items()}
            for k, x in slices_off(got, h, want, terms).items():
                largest[n][k] = max(x, largest[n].get(k, 0))
    for k, most in BOUNDS.items():
        assert largest[3][k] <= most < largest[2][k], (k, largest)
