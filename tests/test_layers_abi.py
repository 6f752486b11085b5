"""The entry points of the layers beside the scan on a machine without a GPU: struct layouts, sizes and refusals.

No call here passes arguments that could reach a kernel launch.
"""
import ctypes
import os
import subprocess

import pytest
import torch

import structured_sparse_selective_b200 as pd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x1000  # stands for a pointer in calls that are refused for another reason
lib = pd._lib


@pytest.mark.parametrize("struct,name", [(pd.NormProblem, "pdssm_norm_problem"), (pd.DeltaProblem, "pdssm_delta_problem")])
def test_struct_layouts_match_c(tmp_path, struct, name):
    fields = [f for f, _ in struct._fields_]
    body = "".join(f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "pdssm.h"\n'
                   f'int main(void){{{body}printf("%zu\\n", sizeof({name}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


def norm(**kw):
    c = dict(batch=2, seqlen=5, q_heads=3, k_heads=1, N=8, io_t=pd.F32, mode=0, rot=4, interleaved=0, eps=1e-6, flags=0)
    c.update(kw)
    return pd.NormProblem(**c)


def delta(**kw):
    c = dict(batch=2, seqlen=5, heads=4, qk_heads=2, N=8, P=8, in_t=pd.F32, gate_t=pd.F32, scale=1.0, flags=0)
    c.update(kw)
    return pd.DeltaProblem(**c)


NORM_BAD = [(dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(q_heads=-1), INVALID), (dict(k_heads=-1), INVALID),
            (dict(N=0), INVALID), (dict(rot=3), INVALID), (dict(rot=10), INVALID), (dict(rot=-2), INVALID),
            (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
            (dict(flags=1), INVALID), (dict(interleaved=2), INVALID), (dict(mode=2), INVALID), (dict(N=129), UNSUPPORTED),
            (dict(io_t=pd.C64), UNSUPPORTED), (dict(q_heads=65536), UNSUPPORTED), (dict(seqlen=1 << 31), UNSUPPORTED),
            (dict(batch=1 << 40, seqlen=1 << 30), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", NORM_BAD)
def test_norm_problems_are_refused(kw, code):
    pb, n = norm(**kw), ctypes.c_size_t()
    assert lib.pdssm_qk_norm(pb, *[A] * 8, None) == code
    assert lib.pdssm_qk_norm_bwd(pb, *[A] * 13, 1 << 20, None) == code
    assert lib.pdssm_qk_norm_bwd_workspace_size(pb, n) == code


@pytest.mark.parametrize("missing", ["q", "k", "inv_freq", "q_out", "k_out"])
def test_norm_pointers_are_checked(missing):
    names = ["q", "k", "wq", "wk", "inv_freq", "positions", "q_out", "k_out"]
    assert lib.pdssm_qk_norm(norm(), *[None if n == missing else A for n in names], None) == INVALID
    assert lib.pdssm_qk_norm(norm(), *[A + 1 if n == missing else A for n in names], None) == INVALID


def test_norm_backward_pointers_are_checked():
    names = ["q", "k", "wq", "wk", "inv_freq", "positions", "dq_out", "dk_out", "dq", "dk", "dwq", "dwk", "workspace"]
    for n in ("q", "k", "wq", "wk", "inv_freq", "dq_out", "dk_out", "dq", "dk"):
        assert lib.pdssm_qk_norm_bwd(norm(), *[None if m == n else A for m in names], 1 << 20, None) == INVALID, n
    for n in names:
        assert lib.pdssm_qk_norm_bwd(norm(), *[A + 1 if m == n else A for m in names], 1 << 20, None) == INVALID, n
    assert lib.pdssm_qk_norm_bwd(norm(), *[None if m == "workspace" else A for m in names], 1 << 20, None) == WORKSPACE
    need = pd.pdssm_qk_norm_bwd_workspace_size(norm())
    assert need > 0
    assert lib.pdssm_qk_norm_bwd(norm(), *[A] * 13, need - 1, None) == WORKSPACE
    assert lib.pdssm_qk_norm(norm(batch=0), *[None] * 8, None) == OK


DELTA_BAD = [(dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(heads=0), INVALID), (dict(qk_heads=0), INVALID),
             (dict(heads=3), INVALID), (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(scale=float("inf")), INVALID),
             (dict(scale=float("nan")), INVALID), (dict(flags=pd.FLAG_HEAD_DICTS), INVALID), (dict(N=129), UNSUPPORTED),
             (dict(P=129), UNSUPPORTED), (dict(in_t=pd.C64), UNSUPPORTED), (dict(gate_t=pd.C64), UNSUPPORTED),
             (dict(batch=65536), UNSUPPORTED), (dict(heads=65536), UNSUPPORTED), (dict(seqlen=1 << 36), UNSUPPORTED),
             (dict(batch=65535, heads=65534, seqlen=1 << 34), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", DELTA_BAD)
def test_delta_problems_are_refused(kw, code):
    pb, n = delta(**kw), ctypes.c_size_t()
    assert lib.pdssm_delta_fwd(pb, *[A] * 10, 1 << 40, None) == code
    assert lib.pdssm_delta_bwd(pb, *[A] * 16, 1 << 40, None) == code
    assert lib.pdssm_delta_workspace_size(pb, n) == code
    assert lib.pdssm_delta_bwd_workspace_size(pb, n) == code


@pytest.mark.parametrize("in_t", [pd.F32, pd.BF16])
def test_delta_pointers_are_checked(in_t):
    pb = delta(in_t=in_t, seqlen=500)
    names = ["q", "k", "v", "g", "beta", "lengths", "h0", "y", "h_final", "workspace"]
    for n in ("q", "k", "v", "g", "beta", "y"):
        assert lib.pdssm_delta_fwd(pb, *[None if m == n else A for m in names], 1 << 40, None) == INVALID, n
    for n in names:
        assert lib.pdssm_delta_fwd(pb, *[A + 1 if m == n else A for m in names], 1 << 40, None) == INVALID, n
    need = pd.pdssm_delta_workspace_size(pb)
    if need:
        assert lib.pdssm_delta_fwd(pb, *[A] * 10, need - 1, None) == WORKSPACE
        assert lib.pdssm_delta_fwd(pb, *[None if m == "workspace" else A for m in names], need, None) == WORKSPACE
    names = ["q", "k", "v", "g", "beta", "lengths", "h0", "dy", "dh_final", "dq", "dk", "dv", "dg", "dbeta", "dh0", "workspace"]
    for n in ("q", "k", "v", "g", "beta", "dy", "dq", "dk", "dv", "dg", "dbeta"):
        assert lib.pdssm_delta_bwd(pb, *[None if m == n else A for m in names], 1 << 40, None) == INVALID, n
    for n in names:
        assert lib.pdssm_delta_bwd(pb, *[A + 1 if m == n else A for m in names], 1 << 40, None) == INVALID, n
    need = pd.pdssm_delta_bwd_workspace_size(pb)
    assert need > 0 and lib.pdssm_delta_bwd(pb, *[A] * 16, need - 1, None) == WORKSPACE
    assert lib.pdssm_delta_bwd(pb, *[None if m == "workspace" else A for m in names], need, None) == WORKSPACE


def test_null_problems_and_sizes():
    n = ctypes.c_size_t()
    assert lib.pdssm_delta_workspace_size(None, n) == INVALID and lib.pdssm_qk_norm_bwd_workspace_size(None, n) == INVALID
    assert lib.pdssm_delta_workspace_size(delta(), None) == INVALID
    assert pd.pdssm_delta_workspace_size(delta(seqlen=1, in_t=pd.BF16)) == 0  # a decoding step needs none
    # the backward pass's workspace grows with the tokens, not with their square
    one, two = (pd.pdssm_delta_bwd_workspace_size(delta(seqlen=s)) for s in (4096, 8192))
    assert two <= 2 * one + 4096


def test_binding_refuses_cpu_tensors_and_mismatches():
    q, v, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="device memory"):
        pd.delta_forward(q, q, v, g, g)
    with pytest.raises(ValueError, match="device memory"):
        pd.qk_norm(q, q)
    for kw, word in ((dict(k=torch.zeros(1, 4, 2, 7)), "k must be"), (dict(v=torch.zeros(1, 5, 2, 8)), "v must be"),
                     (dict(g=torch.zeros(1, 4, 3)), "g must be"), (dict(beta=g.bfloat16()), "beta must be"),
                     (dict(h0=torch.zeros(1, 2, 8, 7)), "h0 must be"), (dict(lengths=torch.zeros(1).long()), "lengths must be"),
                     (dict(q=q.double(), k=q.double()), "float32 or bfloat16"), (dict(v=v.bfloat16()), "v must be")):
        with pytest.raises(ValueError, match=word):
            pd.delta_forward(**{**dict(q=q, k=q, v=v, g=g, beta=g), **kw})
    with pytest.raises(ValueError, match="dy must be"):
        pd.delta_backward(q, q, v, g, g, v[:, :2])
    for kw, word in ((dict(wq=torch.zeros(7)), "wq must be"), (dict(positions=torch.zeros(1, 4)), "positions must be"),
                     (dict(mode="layer"), "mode must be"), (dict(q_out=q.bfloat16()), "q_out must be")):
        with pytest.raises(ValueError, match=word):
            pd.qk_norm(q, q, **kw)
