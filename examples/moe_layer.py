"""A Mixture-of-Experts layer with real experts, served and trained.

    python examples/moe_layer.py

serve: FP8. Routes a decode batch and a single token, dispatches e4m3 rows,
runs the gated experts on e4m3 weights with 128 x 128 block scales and combines.
train: bf16. Fits a small layer to a fixed random target: forward, the gradients
of combine, experts and dispatch, the router's softmax in plain torch, and plain
SGD. Prints the loss, which falls.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_top_histogram_gb300 as moe  # noqa: E402


def quantise_weights(w):
    """e4m3 codes (uint8) and fp32 scales of each 128 x 128 block of w [E, n, m]."""
    E, n, m = w.shape
    b = w.float().view(E, n // 128, 128, m // 128, 128)
    scale = (b.abs().amax((2, 4)) / 448.0).clamp_min(1e-30)
    codes = (b / scale[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(E, n, m), scale.contiguous()


def init_experts(E, H, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    return (new(E, 2 * F, H).normal_(0, H ** -0.5, generator=g),
            new(E, H, F).normal_(0, F ** -0.5, generator=g))


def serve(P=8, E=64, k=8, H=2048, F=1024):
    w13, w2 = init_experts(E, H, F)
    (q13, s13), (q2, s2) = quantise_weights(w13), quantise_weights(w2)
    g = torch.Generator(device="cuda").manual_seed(1)
    for ranks, tokens in ((P, 16), (1, 1)):  # a batch over P ranks, then one token
        layer = moe.MoeLayer(ranks, tokens, E, k, H, moe.MOE_FP8_E4M3)
        layer.set_experts(q13, q2, s13, s2)
        x = torch.empty(layer.T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        logits = torch.randn(layer.T, E, device="cuda", generator=g)
        out = layer.forward(x, logits=logits)
        # the same layer from the unquantised weights
        want = torch.zeros(layer.T, H, device="cuda")
        for e in range(E):
            t, j = (layer.ids == e).nonzero(as_tuple=True)
            if len(t):
                gate, up = (x[t].float() @ w13[e].float().T).chunk(2, dim=1)
                h = torch.nn.functional.silu(gate) * up
                want.index_add_(0, t, layer.w[t, j, None] * (h @ w2[e].float().T))
        err = ((out.float() - want).norm() / want.norm()).item()
        print(f"serve {layer.T} tokens: relative distance from the bf16 layer {err:.4f}", flush=True)
        assert err < 0.1 and layer.status() == 0 and layer.experts.status() == 0


def train(P=4, Tr=64, E=8, k=2, H=256, F=128, steps=60, lr=0.05):
    w13, w2 = init_experts(E, H, F)
    layer = moe.MoeLayer(P, Tr, E, k, H)
    layer.set_experts(w13, w2, train=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(layer.T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    target = torch.randn(layer.T, H, device="cuda", generator=g)
    router = torch.randn(H, E, device="cuda", generator=g) * H ** -0.5
    master = [w13.float(), w2.float()]
    losses = []
    for _ in range(steps):
        logits = x.float() @ router
        diff = layer.forward(x, logits=logits).float() - target
        losses.append(diff.square().mean().item())
        dout = (diff * (2.0 / layer.T)).to(torch.bfloat16)
        grad = layer.backward(dout, layer.w)
        # the router: softmax over the k chosen logits
        w, ids = layer.w, layer.ids.long()
        dz = w * (grad["dw"] - (w * grad["dw"]).sum(1, keepdim=True))
        router -= lr * (x.float().T @ torch.zeros_like(logits).scatter_(1, ids, dz))
        for p, m, d in ((w13, master[0], grad["dw13"]), (w2, master[1], grad["dw2"])):
            m -= lr * d.float()
            p.copy_(m)
    print(f"train {steps} steps: loss {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    assert losses[-1] < 0.9 * losses[0] and layer.experts.status() == 0
    return losses


if __name__ == "__main__":
    serve()
    train()
