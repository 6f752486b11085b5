"""Calls on a stream that is not the current one, while the current one still works: what a call allocates may be used by
nothing that is queued elsewhere, neither before the call nor after its results have been let go."""
import pytest
import torch

import structured_sparse_selective_b200 as pd
import workloads
from tests.test_gpu_layers import delta_case, gradients_in, norm_case

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000  # of a kernel that only waits: some 50 ms, in which the host queues everything below


def scan_inputs():
    sp = workloads.spec("lm", batch=1, seqlen=200, heads=2)
    inp = {k: v.cuda() for k, v in workloads.generate(sp, seed=3).items()}
    return sp, inp


def calls():
    """name -> (inputs by name, call(inputs, stream))"""
    sp, inp = scan_inputs()
    names = ("logits", "idx", "d", "B", "C", "x")
    out = pd.forward(*(inp[n] for n in names), want_s=True)
    a, h0 = delta_case((1, 200, 1, 2, 64, 64), torch.bfloat16)
    dy, dh = gradients_in(a)
    q, k, kw = norm_case((1, 50, 4, 4, 64, 64, False, "rms"), torch.float32)
    M = torch.randn(3, 16, 16, device="cuda")
    u, W = torch.randn(1, 128, 64, device="cuda").bfloat16(), torch.randn(64, 2 * 16, device="cuda").bfloat16()
    dense = torch.randn(sp.K, sp.N, sp.N, device="cuda")
    st = dict(idx_steps=pd.soft_select(inp["logits"], dense)["idx_steps"], **{n: inp[n] for n in ("d", "B", "C", "x")})
    first = {n: inp[n] for n in names}
    return {
        "forward": (first, lambda i, s: pd.forward(**i, stream=s)),
        "backward": ({**first, "s": out["s"], "dy": torch.randn_like(out["y"])}, lambda i, s: pd.backward(**i, stream=s)),
        "dict_hardmax": (dict(M=M), lambda i, s: {"idx": pd.dict_hardmax(**i, stream=s)}),
        "select_proj": (dict(u=u, W=W), lambda i, s: pd.select_proj(**i, heads=2, K=16, stream=s)),
        "soft_select": (dict(logits=inp["logits"], M=dense), lambda i, s: pd.soft_select(**i, stream=s)),
        "forward_steps": (st, lambda i, s: pd.forward_steps(**i, stream=s)),
        "qk_norm": (dict(q=q, k=k), lambda i, s: pd.qk_norm(**i, **kw, stream=s)),
        "qk_norm_backward": (dict(q=q, k=k, dq_out=q.flip(1), dk_out=k.flip(1)), lambda i, s: pd.qk_norm_backward(**i, **kw, stream=s)),
        "delta_forward": (dict(a, h0=h0), lambda i, s: pd.delta_forward(**i, stream=s)),
        "delta_backward": (dict(a, dy=dy, h0=h0, dh_final=dh), lambda i, s: pd.delta_backward(**i, stream=s)),
    }


NAMES = ("forward", "backward", "dict_hardmax", "select_proj", "soft_select", "forward_steps", "qk_norm", "qk_norm_backward",
         "delta_forward", "delta_backward")


def results(out):
    return {n: x for n, x in out.items() if n != "workspace"}


@pytest.mark.parametrize("given", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_lie_where_queued_work_still_writes(name, given):
    inputs, call = calls()[name]
    want = call(inputs, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    junk = [torch.empty_like(x) for x in want.values()]
    for x in junk:
        x.fill_(7)  # behind the wait; the memory is free for the current stream's next tensors
    del x, junk
    got = call(inputs, side if given == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    for n, x in results(want).items():
        assert torch.equal(got[n], x), n


@pytest.mark.parametrize("name", NAMES)
def test_results_that_are_let_go_stay_until_queued_work_has_read_them(name):
    inputs, call = calls()[name]
    side = torch.cuda.Stream()
    want = {n: x.clone() for n, x in results(call(inputs, None)).items()}
    other = {n: x.flip(0).contiguous() if x.dtype == torch.int32 else -x if x.is_floating_point() else x for n, x in inputs.items()}
    call(other, side)
    torch.cuda.synchronize()
    out = call(inputs, side)
    side.synchronize()
    torch.cuda._sleep(CYCLES)
    kept = {n: x.clone() for n, x in results(out).items()}  # behind the wait, on the current stream
    del out
    call(other, side)
    torch.cuda.synchronize()
    for n, x in want.items():
        assert torch.equal(kept[n], x), n


@pytest.mark.parametrize("stream", [None, 0])
def test_the_default_stream_by_its_handle(stream):
    inputs, call = calls()["delta_forward"]
    side = torch.cuda.Stream()
    want = call(inputs, None)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = call(inputs, stream)
    torch.cuda.synchronize()
    assert torch.equal(got["y"], want["y"]) and torch.equal(got["h_final"], want["h_final"])
