"""What the int8 path refuses on the host, without a GPU (see test_experts_host_cpu.py)."""
import ctypes

import pytest
import torch

from combine_top_histogram_gb300 import MoeError, MoeLayer
from combine_top_histogram_gb300 import binding as B
from test_experts_host_cpu import recorder  # noqa: F401


def test_sizes(cuda_lib):
    assert B.moe_workspace_bytes(B.make_config(2, 4, 8, 2, 48, B.MOE_INT8)) > 0
    assert B.moe_workspace_bytes(B.make_config(2, 4, 8, 2, 40, B.MOE_INT8)) == 0
    assert B.moe_workspace_bytes(B.make_config(2, 4, 8, 2, 48, 3)) == 0
    assert B.moe_expert_workspace_bytes(
        B.make_expert_config(4, 48, 80, 10, B.MOE_INT8)) == 256 + 10 * 80 * 4
    for bad in (B.make_expert_config(4, 40, 80, 10, B.MOE_INT8),
                B.make_expert_config(4, 48, 72, 10, B.MOE_INT8),
                B.make_expert_config(4, 48, 80, 10, B.MOE_INT8, train=True),
                B.make_expert_config(4, 48, 80, 10, 3)):
        assert B.moe_expert_workspace_bytes(bad) == 0
        out = ctypes.c_void_p()
        assert cuda_lib.moe_expert_create(ctypes.byref(bad), ctypes.c_void_p(256), 1 << 20,
                                          ctypes.byref(out)) in (-1, -2)


E, H, F, ROWS = 2, 48, 80, 8
OTHER = {torch.int8: (torch.uint8, torch.float8_e4m3fn, torch.bool), torch.float32: (torch.int32,),
         torch.int32: (torch.float32,), torch.bfloat16: (torch.float16,)}


def call(op):
    z = lambda *s, dtype=torch.int8: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f = torch.zeros
    h = B.moe_expert_create(B.make_expert_config(E, H, F, ROWS, B.MOE_INT8), device="cpu")
    off = z(E + 1, dtype=torch.int32)
    if op == "gated":
        return B.moe_expert_gated, h, dict(
            expert_offset=off, inp=z(ROWS, H), inp_scale=f(ROWS), w13=z(E, 2 * F, H),
            w13_scale=f(E, 2 * F), hid=z(ROWS, F), hid_scale=f(ROWS))
    return B.moe_expert_down, h, dict(
        expert_offset=off, hid=z(ROWS, F), hid_scale=f(ROWS), w2=z(E, H, F), w2_scale=f(E, H),
        y=z(ROWS, H, dtype=torch.bfloat16))


@pytest.mark.parametrize("op", ["gated", "down"])
def test_other_types_and_short_tensors_are_refused(recorder, op):  # noqa: F811
    fn, handle, args = call(op)
    fn(handle, **args)
    assert recorder.calls[-1] == fn.__name__
    for name, t in args.items():
        for other in (*(t.view(d) for d in OTHER[t.dtype]), t.flatten()[:-1]):
            with recorder.nothing_called(), pytest.raises(ValueError, match=name):
                fn(handle, **{**args, name: other})


def test_layer_and_experts_have_one_type(recorder):  # noqa: F811
    w13, w2 = torch.zeros(E, 2 * F, H, dtype=torch.int8), torch.zeros(E, H, F, dtype=torch.int8)
    s13, s2 = torch.zeros(E, 2 * F), torch.zeros(E, H)
    other = MoeLayer(1, 4, E, 1, H, device="cpu")
    layer = MoeLayer(1, 4, E, 1, H, B.MOE_INT8, device="cpu")
    assert layer.recv_x.dtype == torch.int8 and layer.recv_scale.shape == (layer.rows,)
    with recorder.nothing_called(), pytest.raises(ValueError, match="type"):
        layer.set_experts(w13.to(torch.bfloat16), w2.to(torch.bfloat16))
    with recorder.nothing_called(), pytest.raises(ValueError, match="type"):
        other.set_experts(w13, w2, s13, s2)
    with recorder.nothing_called(), pytest.raises(ValueError, match="scales"):
        layer.set_experts(w13, w2)
    with pytest.raises(MoeError):
        layer.set_experts(w13, w2, s13, s2, train=True)
    layer.set_experts(w13, w2, s13, s2)
    x, ids, w = torch.zeros(4, H), torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1)
    for mode in ("fused", "allgather"):
        with pytest.raises(ValueError, match="int8"):
            layer.forward(x, ids=ids, w=w, **{mode: True})
    layer.forward(x, ids=ids, w=w)
    assert recorder.calls[-3:] == ["moe_expert_gated", "moe_expert_down", "moe_combine"]
