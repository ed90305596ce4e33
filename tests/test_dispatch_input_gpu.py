"""A dispatch whose tokens come from the launch right before it. Dispatch kernels load their
first rows before they wait for that launch, so a kernel of the library that writes such rows must
not let its dependents start while it still writes: combine's result of one layer is dispatched by
another whose layout was made earlier, and weights are routed between a layout and its dispatch."""
import pytest
import torch

from combine_top_histogram_gb300 import MoeLayer
from combine_top_histogram_gb300 import binding as B

pytestmark = pytest.mark.gpu

TYPES = {"bf16": B.MOE_BF16, "e4m3": B.MOE_FP8_E4M3, "int8": B.MOE_INT8}
H = 512


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ids_of(T, E, k, seed=0):
    return torch.rand(T, E, device="cuda", generator=gen(seed)).topk(k, 1).indices.to(
        torch.int32).contiguous()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T", [300, 40000])  # one wave of combine's CTAs, and many
@pytest.mark.parametrize("dtype", list(TYPES))
def test_combine_then_dispatch(gpu, dtype, T, graph):
    E, k = 8, 2
    first, second = MoeLayer(1, T, E, k, H), MoeLayer(1, T, E, k, H, TYPES[dtype])
    ids, w = ids_of(T, E, k), torch.rand(T, k, device="cuda", generator=gen(1))
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    first.forward(x.normal_(generator=gen(2)), ids=ids, w=w)
    second.forward(first.out, ids=ids, w=w)  # lays out once; the inputs below have other values

    def step():
        first.combine(w)
        second.dispatch(first.out, w)

    step()
    run = step
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    for seed in range(10):
        first.y.normal_(generator=gen(10 + seed))
        first.out.zero_()
        run()
        got = second.recv_x.clone(), None if second.recv_scale is None else second.recv_scale.clone()
        torch.cuda.synchronize()
        second.dispatch(first.out, w)  # the same rows, complete
        assert torch.equal(got[0].view(torch.uint8), second.recv_x.view(torch.uint8)), seed
        assert got[1] is None or torch.equal(got[1], second.recv_scale), seed


@pytest.mark.parametrize("graph", [False, True])
def test_route_between_layout_and_dispatch(gpu, graph):
    """The dispatched weights are those of the logits routed just before."""
    P, Tr, E, k = 4, 1500, 64, 4
    layer = MoeLayer(P, Tr, E, k, 64)
    T = P * Tr
    ids, x = ids_of(T, E, k), torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    routed, w = torch.empty_like(ids), torch.empty(T, k, device="cuda")

    def step():
        B.moe_route_topk(layer.handle, logits, routed, w)
        layer.dispatch(x, w)

    layer.layout(ids)
    logits.normal_(generator=gen(3))
    step()
    run = step
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    for seed in range(10):
        logits.normal_(generator=gen(20 + seed))
        w.zero_()
        run()
        inv = layer.layout_view()["inv"].long()
        assert torch.equal(layer.meta["weight"][inv], w.flatten()), seed
