"""Whole layers with real experts through MoeLayer: route or given ids, dispatch,
gated experts, combine, and for training the way back, against the plain layer
in 64 bits; padded slots, capacity drops, every dispatch form, single tokens."""
import importlib.util
import os

import pytest
import torch

import expert_reference as R
from test_experts_gpu import normal, quant_weights

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def routed(T, E, k, masked=0.1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
    ids[torch.rand(T, k, device="cuda", generator=g) < masked] = -1
    return ids, torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)


def plain(x, w13, w2, ids, w, kept):
    """sum_j w_j expert_{ids_j}(x) over the kept slots, in 64 bits."""
    F = w2.shape[2]
    out = torch.zeros(x.shape[0], w2.shape[1], dtype=torch.float64, device=x.device)
    for e in range(w13.shape[0]):
        t, j = ((ids == e) & kept).nonzero(as_tuple=True)
        both = x[t] @ w13[e].T
        h = both[:, :F] * torch.sigmoid(both[:, :F]) * both[:, F:]
        out = out.index_add(0, t, w[t, j, None] * (h @ w2[e].T))
    return out


def near(got, want, roundings):
    """Each rounding to bf16 changes its tensor by at most 2^-8 of its norm, and a random
    matrix carries a relative change of its input over to its output."""
    off = (got.double() - want).norm() / want.norm().clamp_min(1e-300)
    assert off <= roundings * R.BF16, float(off)


CASES = {"token": (1, 1, 16, 4, 128, 136, 0), "ragged": (2, 37, 8, 2, 264, 72, 0),
         "capacity": (4, 40, 8, 3, 136, 64, 45), "large": (2, 700, 4, 2, 256, 192, 0)}


@pytest.mark.parametrize("mode", ["separate", "fused", "two_stage", "allgather"])
@pytest.mark.parametrize("case", list(CASES))
def test_layer_bf16(gpu, case, mode):
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, F, cap = CASES[case]
    T = P * Tr
    layer = MoeLayer(P, Tr, E, k, H, cap=cap)
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    layer.set_experts(w13, w2)
    x, (ids, w) = normal(T, H), routed(T, E, k)
    out = layer.forward(x, ids=ids, w=w, **({} if mode == "separate" else {mode: True}))
    kept = layer.layout_view()["inv"].view(T, k) >= 0
    want = plain(x.double(), w13.double(), w2.double(), ids, w.double(), kept)
    near(out, want, 3)  # h, y, out
    assert layer.status() == 0 and layer.experts.status() == 0


@pytest.mark.parametrize("case", [(1, 1, 16, 4, 128, 128), (2, 37, 8, 2, 256, 384),
                                  (2, 700, 4, 2, 256, 128)])
def test_layer_fp8_routed(gpu, case):
    from combine_top_histogram_gb300 import MOE_FP8_E4M3, MoeLayer
    P, Tr, E, k, H, F = case
    T = P * Tr
    layer = MoeLayer(P, Tr, E, k, H, MOE_FP8_E4M3)
    q13, s13 = quant_weights(normal(E, 2 * F, H, std=H ** -0.5, seed=1))
    q2, s2 = quant_weights(normal(E, H, F, std=F ** -0.5, seed=2))
    layer.set_experts(q13, q2, s13, s2)
    x = normal(T, H)
    logits = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    out = layer.forward(x, logits=logits)
    want = plain(x.double(), R.dequant_weights(q13, s13), R.dequant_weights(q2, s2), layer.ids,
                 layer.w.double(), layer.ids >= 0)
    # e4m3 keeps four bits: x and h are each rounded to within 2^-4 of a value
    off = (out.double() - want).norm() / want.norm()
    assert off <= 2 * 2.0 ** -4 + 3 * R.BF16, float(off)
    assert layer.status() == 0 and layer.experts.status() == 0


@pytest.mark.parametrize("case", list(CASES))
def test_layer_backward(gpu, case):
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, F, cap = CASES[case]
    T = P * Tr
    layer = MoeLayer(P, Tr, E, k, H, cap=cap)
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    layer.set_experts(w13, w2, train=True)
    x, (ids, w), dout = normal(T, H), routed(T, E, k), normal(T, H, std=0.1, seed=4)
    layer.forward(x, ids=ids, w=w)
    grad = layer.backward(dout, w)
    kept = layer.layout_view()["inv"].view(T, k) >= 0
    leaf = [v.double().requires_grad_() for v in (x, w13, w2, w)]
    (plain(leaf[0], leaf[1], leaf[2], ids, leaf[3], kept) * dout.double()).sum().backward()
    # y, dy, gate_up, dg and du, each result; dx adds two sums of roundings
    for name, v, n in (("dx", leaf[0], 6), ("dw13", leaf[1], 5), ("dw2", leaf[2], 4),
                       ("dw", leaf[3], 3)):
        near(grad[name], v.grad, n)
    assert layer.status() == 0 and layer.experts.status() == 0


def test_layer_refusals(gpu):
    from combine_top_histogram_gb300 import MoeLayer
    layer = MoeLayer(2, 8, 4, 2, 64)
    w13, w2 = normal(4, 32, 64), normal(4, 64, 16)
    x, (ids, w) = normal(16, 64), routed(16, 4, 2)
    with pytest.raises(ValueError):
        layer.set_experts(w13, w2.transpose(1, 2).contiguous())
    with pytest.raises(ValueError):
        layer.set_experts(w13[:2], w2[:2])
    with pytest.raises(ValueError):
        layer.set_experts(torch.zeros(4, 256, 128, dtype=torch.uint8, device="cuda"),
                          torch.zeros(4, 128, 128, dtype=torch.uint8, device="cuda"))
    layer.set_experts(w13, w2)
    with pytest.raises(ValueError):
        layer.forward(x, ids=ids, w=w, fixed_slots=True)
    with pytest.raises(ValueError):
        layer.forward_pipelined(x, ids=ids, w=w)
    with pytest.raises(ValueError):
        layer.backward(x, w)
    with pytest.raises(ValueError):
        layer.forward(x, ids=ids, w=w, expert_scale=torch.ones(4, device="cuda"))
    layer.set_experts(None, None)  # the stand-in again
    layer.forward(x, ids=ids, w=w, fixed_slots=True)


def test_example_serves_and_trains(gpu):
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.serve()
    m.train()
