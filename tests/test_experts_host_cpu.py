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


def test_backward_needs_a_forward_of_these_experts(recorder):
    """New experts have no hidden rows yet, whatever ran before them."""
    layer, x, ids, w = layer_for_training()
    for _ in range(2):
        layer.layout(ids)
        layer.dispatch(x, w)
        with recorder.nothing_called(), pytest.raises(ValueError, match="forward"):
            layer.backward(x, w)
        with recorder.nothing_called(), pytest.raises(ValueError, match="forward"):
            layer.experts.backward(ids, layer.recv_x, layer.y, layer.y)
        layer.forward(x, ids=ids, w=w)
        layer.backward(x, w)
        layer.set_experts(layer.experts.w13, layer.experts.w2, train=True)


E, H, F, ROWS = 2, 128, 128, 8
f32 = torch.zeros
SAME_SIZE = {torch.bfloat16: (torch.float16, torch.int16), torch.uint8: (torch.int8,
             torch.float8_e5m2, torch.bool), torch.float32: (torch.int32,),
             torch.int32: (torch.float32,)}


def call(op, fp8=False):
    """An operator's binding and its arguments by name, every one of the right type."""
    dt = torch.uint8 if fp8 else torch.bfloat16
    z = lambda *s, dtype=dt: torch.zeros(*s, dtype=dtype)  # noqa: E731
    if op == "combine_backward":
        layer, x, ids, w = layer_for_training()
        layer.forward(x, ids=ids, w=w)
        return B.moe_combine_backward, layer.handle, dict(
            dout=x, y=layer.y, w=w, dy=torch.zeros_like(layer.y), dw=torch.zeros_like(w))
    h = B.moe_expert_create(B.make_expert_config(E, H, F, ROWS, int(fp8), op == "backward"),
                            device="cpu")
    a = dict(expert_offset=z(E + 1, dtype=torch.int32))
    if op == "gated":
        a.update(inp=z(ROWS, H), inp_scale=f32(ROWS, 1) if fp8 else None, w13=z(E, 2 * F, H),
                 w13_scale=f32(E, 2, 1) if fp8 else None, hid=z(ROWS, F),
                 hid_scale=f32(ROWS, 1) if fp8 else None,
                 gate_up=None if fp8 else z(ROWS, 2 * F))
        return B.moe_expert_gated, h, a
    if op == "down":
        a.update(hid=z(ROWS, F), hid_scale=f32(ROWS, 1) if fp8 else None, w2=z(E, H, F),
                 w2_scale=f32(E, 1, 1) if fp8 else None, y=bf16(ROWS, H))
        return B.moe_expert_down, h, a
    a.update(inp=z(ROWS, H), gate_up=z(ROWS, 2 * F), hid=z(ROWS, F), dy=z(ROWS, H),
             w13=z(E, 2 * F, H), w2=z(E, H, F), dx=z(ROWS, H), dw13=z(E, 2 * F, H),
             dw2=z(E, H, F))
    return B.moe_expert_backward, h, a


@pytest.mark.parametrize("op, fp8", [("gated", False), ("gated", True), ("down", False),
                                     ("down", True), ("backward", False),
                                     ("combine_backward", False)])
def test_other_types_of_the_same_size_are_refused(recorder, op, fp8):
    fn, handle, args = call(op, fp8)
    fn(handle, **args)
    assert recorder.calls[-1] == fn.__name__
    for name, t in args.items():
        for other in SAME_SIZE[t.dtype] if t is not None else ():
            with recorder.nothing_called(), pytest.raises(ValueError, match=name):
                fn(handle, **{**args, name: t.view(other)})
        if t is not None and t.dtype == torch.uint8:  # codes by their own name
            fn(handle, **{**args, name: t.view(torch.float8_e4m3fn)})


@pytest.mark.parametrize("types", [(torch.float16, torch.float16), (torch.int8, torch.int8),
                                   (torch.float8_e5m2, torch.float8_e5m2),
                                   (torch.bfloat16, torch.float16), (torch.uint8, torch.int8),
                                   (torch.bfloat16, torch.uint8), (torch.float32, torch.float32)])
def test_experts_of_other_types_are_refused(recorder, types):
    one = torch.ones(2, 2, 1)
    for layer in (MoeLayer(1, 4, 2, 1, 128, device="cpu"),
                  MoeLayer(1, 4, 2, 1, 128, B.MOE_FP8_E4M3, device="cpu")):
        with recorder.nothing_called(), pytest.raises(ValueError):
            layer.set_experts(torch.zeros(2, 256, 128, dtype=types[0]),
                              torch.zeros(2, 128, 128, dtype=types[1]), one, one)
    assert layer.experts is None
