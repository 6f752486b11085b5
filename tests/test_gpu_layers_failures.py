"""What the delta rule's calls leave behind when a wait of a kernel's role on another runs out.

PDSSM_FLAG_SHORT_WAITS lets the waits run out after a microsecond, on the host's wish and without a fault.
"""
import pytest
import torch

import structured_sparse_selective_b200 as pd
from tests.test_gpu_layers import delta_case, gradients_in

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 6
SEVEN = 7.0  # stands where nothing has been written
# batch, seqlen, qk_heads, heads, N, P: every chunk kernel; in fp32 with a warp for the copies and without one
CASES = [(2, 600, 1, 2, 64, 64), (5, 300, 2, 16, 128, 64), (1, 700, 1, 1, 96, 40)]


def setup(c, dt):
    a, h0 = delta_case(c, dt)
    dy, dh = gradients_in(a)
    names = ("q", "k", "v", "g", "beta")
    pb = pd._delta_problem(*(a[n] for n in names), h0, None, None, pd.FLAG_SHORT_WAITS)[0]
    return a, h0, dy, dh, [a[n] for n in names], pb


def forward(ins, pb, h0, lengths=None):
    out = {"y": torch.full_like(ins[2], SEVEN), "h_final": torch.full_like(h0, SEVEN)}
    ws = torch.zeros(pd.pdssm_delta_workspace_size(pb), dtype=torch.uint8, device="cuda")
    pd.pdssm_delta_fwd(pb, *ins, lengths, h0, out["y"], out["h_final"], ws)
    assert pd.pdssm_read_device_check(ws) == TIMEOUT
    return out


def backward(ins, pb, h0, dy, dh, lengths=None):
    out = {"d" + n: torch.full_like(x, SEVEN) for n, x in zip(("q", "k", "v", "g", "beta"), ins)}
    out["dh0"] = torch.full_like(h0, SEVEN)
    ws = torch.zeros(pd.pdssm_delta_bwd_workspace_size(pb), dtype=torch.uint8, device="cuda")
    pd.pdssm_delta_bwd(pb, *ins, lengths, h0, dy, dh, *out.values(), ws)
    assert pd.pdssm_read_device_check(ws) == TIMEOUT
    return out


@pytest.mark.parametrize("c", CASES)
def test_no_warp_computes_in_fp32_after_a_wait_has_run_out(c):
    """The waits run out before any record has been asked for, so no step's result can have been computed."""
    a, h0, dy, dh, ins, pb = setup(c, torch.float32)
    y, dv = forward(ins, pb, h0)["y"], backward(ins, pb, h0, dy, dh)["dv"]
    for x in (y, dv):
        assert ((x == SEVEN) | x.isnan()).all()
