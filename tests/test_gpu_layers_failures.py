"""What the delta rule's calls leave behind when a wait of a kernel's role on another runs out.

PDSSM_FLAG_SHORT_WAITS lets the waits run out after a microsecond, on the host's wish and without a fault.
"""
import pytest
import torch

import structured_sparse_selective_b200 as pd
from tests.test_gpu_layers import TYPES, delta_case, gradients_in

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


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("c", CASES)
def test_a_timeout_leaves_nan_where_values_are_not_finished(c, dt):
    a, h0, dy, dh, ins, pb = setup(c, dt)
    out = forward(ins, pb, h0) | backward(ins, pb, h0, dy, dh)
    for n, x in out.items():
        assert x.isnan().all(), n


@pytest.mark.parametrize("dt", TYPES)
def test_a_timeout_leaves_padding_and_sequences_without_steps_as_they_are(dt):
    L = 600
    a, h0, dy, dh, ins, pb = setup((4, L, 1, 2, 64, 64), dt)
    lengths = torch.tensor([L, 0, 450, 1], dtype=torch.int32, device="cuda")
    out, back = forward(ins, pb, h0, lengths), backward(ins, pb, h0, dy, dh, lengths)
    assert torch.equal(out["h_final"][1], h0[1]) and torch.equal(back["dh0"][1], dh[1])
    for b, n in enumerate(lengths.tolist()):
        for name, x in {"y": out["y"], **back}.items():
            if name != "dh0":
                assert x[b, :n].isnan().all() and not x[b, n:].any(), (name, b)
        if n:
            assert out["h_final"][b].isnan().all() and back["dh0"][b].isnan().all()


@pytest.mark.parametrize("dt", TYPES)
def test_a_timeout_shows_in_the_default_call(dt):
    """The wrapper keeps the workspace it allocates to itself: the outputs say that the call was not finished."""
    a, h0, dy, dh, _, _ = setup((1, 400, 1, 2, 72, 64), dt)
    out = pd.delta_forward(**a, h0=h0, flags=pd.FLAG_SHORT_WAITS)
    out |= pd.delta_backward(**a, dy=dy, h0=h0, dh_final=dh, flags=pd.FLAG_SHORT_WAITS)
    for n, x in out.items():
        assert x.isnan().all(), n


@pytest.mark.parametrize("dt", TYPES)
def test_the_error_word_is_that_of_the_last_call(dt):
    """One workspace for a prompt and the tokens behind it: what the prompt left in the word is not the token's."""
    a, h0, dy, dh, ins, pb = setup((2, 600, 1, 2, 64, 64), dt)
    ws = torch.full((pd.pdssm_delta_bwd_workspace_size(pb),), 255, dtype=torch.uint8, device="cuda")
    for L in (1, 5, 0):  # a token, steps, nothing
        pd.delta_forward(**a, h0=h0, flags=pd.FLAG_SHORT_WAITS, workspace=ws)
        assert pd.pdssm_read_device_check(ws) == TIMEOUT
        short = {n: x[:, :L].contiguous() for n, x in a.items()}
        pd.delta_forward(**short, h0=h0, workspace=ws)
        assert pd.pdssm_read_device_check(ws) == OK, L
    # no sequences at all, in either direction, on a buffer that nobody has cleared
    for L in (1, 600):
        none = {n: x[:0, :L].contiguous() for n, x in a.items()}
        ws.fill_(255)
        pd.delta_forward(**none, workspace=ws)
        assert pd.pdssm_read_device_check(ws) == OK
        ws.fill_(255)
        pd.delta_backward(**none, dy=none["v"], workspace=ws)
        assert pd.pdssm_read_device_check(ws) == OK


def test_a_workspace_where_none_is_needed_may_be_smaller_than_the_error_word():
    a, h0, *_ = setup((2, 1, 1, 2, 64, 64), torch.float32)
    room = torch.full((32,), 255, dtype=torch.uint8, device="cuda")
    want = pd.delta_forward(**a, h0=h0)
    got = pd.delta_forward(**a, h0=h0, workspace=room[:3])
    assert torch.equal(got["y"], want["y"]) and (room == 255).all()
    pd.delta_forward(**a, h0=h0, workspace=room)
    assert not room[:4].any() and (room[4:] == 255).all()
