"""Layers of int8 experts over the other ways their rows can come: the two-stage dispatch and
token ranges leave the same receive rows as the plain one, so the layer's result is the same bit
for bit; masked slots, a capacity, a captured layer beside an eager one of the same weights."""
import pytest
import torch

import int8_reference as Q
from combine_top_histogram_gb300 import MoeLayer
from combine_top_histogram_gb300 import binding as B
from test_experts_layer_gpu import routed
from test_int8_gpu import gen

pytestmark = pytest.mark.gpu

#: P, Tr, E, k, H, F, capacity: few rows, tiles, rows cut at a capacity
LAYERS = {"few": (2, 3, 8, 2, 272, 80, 0), "tiles": (2, 150, 8, 3, 528, 144, 0),
          "capacity": (4, 40, 8, 3, 144, 64, 45)}


def weights(E, H, F):
    w13 = torch.randn(E, 2 * F, H, device="cuda", generator=gen(1)) / H ** 0.5
    w2 = torch.randn(E, H, F, device="cuda", generator=gen(2)) / F ** 0.5
    return (*Q.quantise(w13), *Q.quantise(w2))


def make(case):
    P, Tr, E, k, H, F, cap = LAYERS[case]
    w13, s13, w2, s2 = weights(E, H, F)
    layer = MoeLayer(P, Tr, E, k, H, B.MOE_INT8, cap)
    layer.set_experts(w13, w2, s13, s2)
    x = torch.randn(P * Tr, H, device="cuda", generator=gen(3)).to(torch.bfloat16)
    return layer, x, *routed(P * Tr, E, k)


def by_ranges(layer, x, ids, w):
    layer.layout(ids)
    for lo, hi in ((0, layer.T // 3), (layer.T // 3, layer.T)):
        B.moe_dispatch_tokens(layer.handle, lo, hi, x, w, layer.recv_x, layer.recv_scale,
                              layer.meta)
    layer.expert()
    layer.combine(w)


@pytest.mark.parametrize("case", list(LAYERS))
@pytest.mark.parametrize("way", ["two_stage", "ranges"])
def test_other_dispatches_give_the_same_layer(gpu, case, way):
    layer, x, ids, w = make(case)
    want = layer.forward(x, ids=ids, w=w).clone()
    assert want.isfinite().all() and (want != 0).any()
    layer.poison()
    if way == "two_stage":
        layer.forward(x, ids=ids, w=w, two_stage=True)
    else:
        by_ranges(layer, x, ids, w)
    assert torch.equal(layer.out, want)
    assert layer.status() == 0 and layer.experts.status() == 0


def test_a_batch_whose_every_slot_is_masked(gpu):
    layer, x, ids, w = make("tiles")
    layer.forward(x, ids=ids, w=w)
    out = layer.forward(x, ids=torch.full_like(ids, -1), w=w)
    assert (out == 0).all() and layer.status() == 0 and layer.experts.status() == 0


@pytest.mark.parametrize("case", list(LAYERS))
def test_a_captured_layer_beside_an_eager_one(gpu, case):
    """Two layers over the same weights, one replayed on its own stream while the other runs."""
    (a, x, ids, w), (b, *_) = make(case), make(case)
    want = a.forward(x, ids=ids, w=w).clone()
    b.forward(x, ids=ids, w=w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.forward(x, ids=ids, w=w)
    side = torch.cuda.Stream()
    for _ in range(10):
        a.out.fill_(float("nan"))
        b.out.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g.replay()
        a.forward(x, ids=ids, w=w)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want) and torch.equal(b.out, want)
