"""What the binding and the layer refuse before any launch, on the host alone: the
library's entry points that reach the GPU are replaced by ones that record the call,
and tensors of the CPU stand for the device's."""
import contextlib

import pytest
import torch

from combine_top_histogram_gb300 import MoeLayer
from combine_top_histogram_gb300 import binding as B

#: entry points that touch no GPU: the real ones run
HOST_ONLY = ("moe_workspace_bytes", "moe_recv_rows_max", "moe_fixed_slot_rows", "moe_error_string",
             "moe_expert_workspace_bytes")


class RecordingLibrary:
    """Every other entry point succeeds without doing anything; `calls` names them in order."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name in HOST_ONLY:
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append(name)
            if name == "moe_get_layout":  # every view at the workspace's start
                view = args[1]._obj
                for field, _ in view._fields_:
                    setattr(view, field, self.workspace)
            elif name == "moe_handle_create":
                self.workspace = args[1]
            return 0
        return call

    @contextlib.contextmanager
    def nothing_called(self):
        before = list(self.calls)
        yield
        assert self.calls == before


@pytest.fixture
def recorder(cuda_lib, monkeypatch):
    rec = RecordingLibrary(cuda_lib)
    monkeypatch.setattr(B, "load_library", lambda: rec)
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
    return rec


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def layer_for_training(P=2, Tr=8, E=8, k=2, H=64, F=32):
    layer = MoeLayer(P, Tr, E, k, H, device="cpu")
    layer.set_experts(bf16(E, 2 * F, H), bf16(E, H, F), train=True)
    x, w = bf16(layer.T, H), torch.zeros(layer.T, k)
    return layer, x, torch.zeros(layer.T, k, dtype=torch.int32), w


def test_experts_refuse_fixed_slots_before_the_dispatch(recorder):
    layer, x, ids, w = layer_for_training()
    with recorder.nothing_called(), pytest.raises(ValueError, match="fixed slots"):
        layer.forward(x, ids=ids, w=w, fixed_slots=True)
    assert not layer.fixed


def test_backward_refuses_the_fixed_slot_layout(recorder):
    """inv then names rows up to E T, past the T k rows of the layer's buffers."""
    layer, x, ids, w = layer_for_training()
    layer.forward(x, ids=ids, w=w)
    layer.layout(ids)
    layer.dispatch_fixed_slots(x, w)
    with recorder.nothing_called(), pytest.raises(ValueError, match="fixed slots"):
        layer.backward(x, w)
    layer.forward(x, ids=ids, w=w)
    layer.backward(x, w)
    assert "moe_expert_backward" in recorder.calls and recorder.calls[-1] == "moe_combine"


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("short", ["y", "dy"])
def test_combine_backward_wants_every_row_of_the_last_dispatch(recorder, fixed, short):
    layer, x, ids, w = layer_for_training()
    layer.layout(ids)
    (layer.dispatch_fixed_slots if fixed else layer.dispatch)(x, w)
    rows = B.moe_fixed_slot_rows(layer.cfg) if fixed else layer.rows
    t = {"y": bf16(rows, layer.H), "dy": bf16(rows, layer.H)}
    args = lambda: (layer.handle, x, t["y"], w, t["dy"], torch.zeros_like(w))  # noqa: E731
    B.moe_combine_backward(*args())
    t[short] = t[short][:-1]
    with recorder.nothing_called(), pytest.raises(ValueError, match=short):
        B.moe_combine_backward(*args())
    layer.layout(ids)
    layer.dispatch(x, w)  # the compact rows again, whatever came before
    t[short] = bf16(layer.rows, layer.H)
    B.moe_combine_backward(*args())
    assert recorder.calls[-1] == "moe_combine_backward"


def test_backward_allocates_nothing(recorder, monkeypatch):
    """Buffers made in a backward on another stream would be filled on the current one."""
    layer, x, ids, w = layer_for_training()
    layer.forward(x, ids=ids, w=w)
    for name in ("ones", "empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, lambda *a, **k: pytest.fail("allocated"))
    layer.backward(x, w, stream=1)
