"""The scan's entry points captured into a graph and replayed, on new inputs."""
import pytest
import torch

import structured_sparse_selective_b200 as pd
import workloads

pytestmark = pytest.mark.gpu


def inputs(name, seed):
    sp = workloads.spec(name, batch=1, seqlen=150, heads=2)
    return sp, {k: v.cuda() for k, v in workloads.generate(sp, seed=seed).items()}


def same(got, want):
    return all(torch.equal(got[n], want[n]) for n in want if n != "workspace")


@pytest.mark.parametrize("name", ["lm", "long", "complex"])
def test_forward_and_backward_in_a_graph(name):
    sp, inp = inputs(name, 3)
    names = ("logits", "idx", "d", "B", "C", "x")

    def run():
        f = pd.forward(*(inp[n] for n in names), want_s=True)
        return f, pd.backward(inp["logits"], f["s"], *(inp[n] for n in names[1:]), dy=f["y"])

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for n, x in inputs(name, 4)[1].items():
        inp[n].copy_(x)
    want = run()
    graph.replay()
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_selections_in_a_graph():
    sp, inp = inputs("lm", 3)
    M = torch.randn(sp.K, sp.N, sp.N, device="cuda")
    u, W = torch.randn(1, 128, 64, device="cuda").bfloat16(), torch.randn(64, 2 * 16, device="cuda").bfloat16()

    def run():
        steps = pd.soft_select(inp["logits"], M)
        return (steps, pd.forward_steps(steps["idx_steps"], *(inp[n] for n in ("d", "B", "C", "x"))), pd.select_proj(u, W, 2, 16),
                {"idx": pd.dict_hardmax(M)})

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for x in (M, u):
        x.copy_(-x)
    want = run()
    graph.replay()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert same(g, w)
