"""Which device and stream the binding hands to the library, on a machine without a GPU.

The tensors here lie on the CPU and say that they are on a card; the library's functions are replaced, so nothing is launched.
"""
import contextlib

import pytest
import torch

import structured_sparse_selective_b200 as pd


class OnCard(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 1."""
    index = 1
    device = property(lambda self: torch.device("cuda", self.index))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


class Stream:
    """Stands for a torch.cuda.Stream of a device."""

    def __init__(self, device_index, handle):
        self.device_index, self.cuda_stream = device_index, handle


def card(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnCard)


@pytest.fixture
def calls(monkeypatch):
    """What the replaced functions saw: (name, device current in the call, stream handle)."""
    seen, state = [], {"device": 0}

    def replace(name):
        def fake(*args):
            handle = args[-1]
            seen.append((name, state["device"], int(getattr(handle, "value", handle) or 0)))
            return 0
        monkeypatch.setattr(pd._lib, name, fake)

    @contextlib.contextmanager
    def device(index):
        before, state["device"] = state["device"], index
        yield
        state["device"] = before

    for name in ENTRIES:
        replace(name)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(pd, "_get_device", lambda: state["device"])
    monkeypatch.setattr(pd, "_current_handle", lambda index: 0)  # the default stream, on any device
    yield seen
    assert state["device"] == 0


def x(n):
    return [card(1, 2, 1, 4) for _ in range(n)]


ENTRIES = {
    "pdssm_select": lambda st: pd.pdssm_select(pd.Problem(), *x(2), stream=st),
    "pdssm_scan_fwd": lambda st: pd.pdssm_scan_fwd(pd.Problem(), *x(12), stream=st),
    "pdssm_forward": lambda st: pd.pdssm_forward(pd.Problem(), *x(13), stream=st),
    "pdssm_forward_noalloc": lambda st: pd.pdssm_forward_noalloc(pd.Problem(), *x(12), stream=st),
    "pdssm_scan_bwd": lambda st: pd.pdssm_scan_bwd(pd.Problem(), *x(10), 1.0, *x(7), stream=st),
    "pdssm_dict_hardmax": lambda st: pd.pdssm_dict_hardmax(1, 4, *x(2), stream=st),
    "pdssm_select_proj": lambda st: pd.pdssm_select_proj(pd.Problem(), 4, *x(5), stream=st),
    "pdssm_soft_select": lambda st: pd.pdssm_soft_select(pd.Problem(), *x(2), 1.0, *x(2), stream=st),
    "pdssm_scan_fwd_steps": lambda st: pd.pdssm_scan_fwd_steps(pd.Problem(), *x(11), stream=st),
    "pdssm_read_device_check": lambda st: pd.pdssm_read_device_check(card(4), stream=st),
    "pdssm_qk_norm": lambda st: pd.pdssm_qk_norm(pd.NormProblem(), *x(8), stream=st),
    "pdssm_qk_norm_bwd": lambda st: pd.pdssm_qk_norm_bwd(pd.NormProblem(), *x(13), stream=st),
    "pdssm_delta_fwd": lambda st: pd.pdssm_delta_fwd(pd.DeltaProblem(), *x(10), stream=st),
    "pdssm_delta_bwd": lambda st: pd.pdssm_delta_bwd(pd.DeltaProblem(), *x(16), stream=st),
}


@pytest.mark.parametrize("name", ENTRIES)
@pytest.mark.parametrize("stream,handle", [(None, 0), (0, 0), (77, 77), (Stream(1, 0), 0), (Stream(1, 99), 99)])
def test_a_call_runs_with_its_tensors_device_current(calls, name, stream, handle):
    """The default stream's handle is 0 on every device: the library takes it for the current one's."""
    ENTRIES[name](stream)
    assert calls == [(name, 1, handle)]


@pytest.mark.parametrize("name", ENTRIES)
def test_a_stream_of_another_device_is_refused(calls, name):
    with pytest.raises(ValueError, match="stream of cuda:0, tensors on cuda:1"):
        ENTRIES[name](Stream(0, 5))
    assert not calls


def test_a_call_on_the_current_device_leaves_it_alone(calls, monkeypatch):
    monkeypatch.setattr(OnCard, "index", 0)
    monkeypatch.setattr(torch.cuda, "device", None)  # not needed, and not used
    for name, call in ENTRIES.items():
        call(None)
        assert calls[-1] == (name, 0, 0)
