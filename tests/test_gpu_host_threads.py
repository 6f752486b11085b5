"""Calls of one kernel with different sizes of shared memory, made by two host threads at once: what one call allows its launch must
not take away what another needs."""
import threading

import pytest
import torch

import structured_sparse_selective_b200 as pd
import workloads
from tests.test_gpu_layers import delta_case, gradients_in

pytestmark = pytest.mark.gpu


def delta_forward(c):
    a, h0 = delta_case(c, torch.float32)
    ins = [a[n] for n in ("q", "k", "v", "g", "beta")]
    pb = pd._delta_problem(*ins, h0, None, None, 0)[0]
    out = {"y": torch.empty_like(a["v"]), "h_final": torch.empty_like(h0)}
    ws = torch.empty(pd.pdssm_delta_workspace_size(pb), dtype=torch.uint8, device="cuda")
    return lambda s: pd.pdssm_delta_fwd(pb, *ins, None, h0, *out.values(), ws, s), out


def delta_backward(c):
    a, h0 = delta_case(c, torch.float32)
    dy, dh = gradients_in(a)
    ins = [a[n] for n in ("q", "k", "v", "g", "beta")]
    pb = pd._delta_problem(*ins, h0, None, None, 0)[0]
    out = {"d" + n: torch.empty_like(x) for n, x in zip(("q", "k", "v", "g", "beta", "h0"), (*ins, h0))}
    ws = torch.empty(pd.pdssm_delta_bwd_workspace_size(pb), dtype=torch.uint8, device="cuda")
    return lambda s: pd.pdssm_delta_bwd(pb, *ins, None, h0, dy, dh, *out.values(), ws, s), out


def scan(K, backward):
    sp = workloads.spec("lm", batch=1, seqlen=40, heads=1)
    inp = {k: v.cuda() for k, v in workloads.generate(sp, seed=3).items()}
    logits, idx = inp["logits"][..., :K].contiguous(), inp["idx"][:K].contiguous()
    rest = [inp[n] for n in ("d", "B", "C", "x")]
    out = pd.forward(logits, idx, *rest, want_s=True)
    pb = pd.make_problem(logits, rest[0], rest[1], rest[3])
    ws = out.pop("workspace", None) or torch.empty(max(pd.pdssm_workspace_size(pb), pd.pdssm_bwd_workspace_size(pb)), dtype=torch.uint8,
                                                   device="cuda")
    if not backward:
        return lambda s: pd.pdssm_forward(pb, logits, idx, *rest, None, out["y"], out["h_final"], out["prod_idx"], out["prod_val"], out["s"],
                                          ws, s), out
    sel, dy = out["s"].clone(), out["y"].clone()
    grads = pd.backward(logits, sel, idx, *rest, dy=dy, want_dh0=False)
    return lambda s: pd.pdssm_scan_bwd(pb, logits, sel, idx, *rest, None, dy, None, 1.0, grads["dlogits"], grads["dd"], grads["dB"],
                                       grads["dC"], grads["dx"], None, ws, s), grads


def soft(K):
    sp = workloads.spec("lm", batch=1, seqlen=40, heads=1)
    logits = workloads.generate(sp, seed=3)["logits"].cuda()[..., :K].contiguous()
    M = torch.randn(K, sp.N, sp.N, device="cuda")
    pb = pd.Problem(batch=1, seqlen=40, heads=1, N=sp.N, P=1, K=K, chunk=0, logits_t=pd._DT[logits.dtype], in_t=0, d_t=0, state_t=0, out_t=0)
    ws = torch.empty(pd.pdssm_soft_select_workspace_size(pb), dtype=torch.uint8, device="cuda")
    out = {"idx_steps": torch.empty(1, 40, 1, sp.N, dtype=torch.uint8, device="cuda")}
    return lambda s: pd.pdssm_soft_select(pb, logits, M, 1.0, out["idx_steps"], ws, s), out


PAIRS = {  # two calls of the same kernels, the first with more shared memory than the second
    "delta_forward": lambda: (delta_forward((4, 300, 8, 8, 32, 32)), delta_forward((1, 300, 8, 8, 32, 32))),
    "delta_backward": lambda: (delta_backward((2, 100, 8, 8, 32, 32)), delta_backward((2, 100, 8, 8, 32, 8))),
    "scan_forward": lambda: (scan(16, False), scan(4, False)),
    "scan_backward": lambda: (scan(16, True), scan(4, True)),
    "soft_select": lambda: (soft(64), soft(4)),
}


@pytest.mark.parametrize("name", PAIRS)
def test_calls_of_different_sizes_by_two_threads(name):
    pair = PAIRS[name]()
    want = []
    for call, out in pair:
        call(None)
        torch.cuda.synchronize()
        want.append({n: x.clone() for n, x in out.items()})
    wrong, start = [], threading.Barrier(2)

    def work(call):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            for i in range(8000):
                call(stream)
                if i % 500 == 499:
                    stream.synchronize()
        except Exception as e:
            wrong.append(f"call {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in pair]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    for (_, out), w in zip(pair, want):
        for n, x in w.items():
            assert torch.equal(out[n], x), n
