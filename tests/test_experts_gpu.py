"""The expert operators against their plain 64-bit forms (expert_reference.py):
gated projections, output product and backward pass over segments of every
kind -- empty, of one row, ending inside a tile, many tiles long -- with sizes
that no tile divides, in both dtypes; combine's backward pass; the arguments
they refuse; and what must not be touched."""
import ctypes

import pytest
import torch

import expert_reference as R
from combine_top_histogram_gb300 import binding as B

pytestmark = pytest.mark.gpu

# (counts of each expert, H, F): bf16 sizes are multiples of 8, FP8 of 128
BF16_CASES = {
    "one_row": ([1], 64, 64),
    "one_row_of_many": ([0, 0, 1, 0], 1024, 512),
    "token_top8": ([1 if e % 4 == 1 else 0 for e in range(32)], 256, 136),
    "token_pair": ([2, 0, 1, 1], 520, 264),
    "few_rows_one_expert": ([7, 0], 264, 72),
    "narrow": ([5, 3], 8, 8),
    "ragged": ([130, 1, 0, 257, 64], 200, 328),
    "tile_edges": ([128, 127, 129, 0, 256, 255], 192, 256),
    "long": ([1500, 3], 320, 136),
    "many_experts": ([(7 * e) % 23 for e in range(200)], 128, 96),
    "wide": ([33, 65], 2056, 1032),
    "none": ([0, 0, 0], 64, 64),
}
FP8_CASES = {
    "one_row": ([1], 128, 128),
    "token_top8": ([1 if e % 4 == 1 else 0 for e in range(32)], 1024, 256),
    "token_pair": ([2, 0, 1, 1], 640, 384),
    "ragged": ([130, 1, 0, 257, 64], 256, 384),
    "tile_edges": ([128, 127, 129, 0, 256, 255], 384, 128),
    "long": ([1500, 3], 128, 640),
    "many_experts": ([(7 * e) % 23 for e in range(200)], 128, 128),
    "wide": ([33, 65], 2176, 1152),
}


# Rows of the buffers past the segments, in multiples of 1 and of the experts:
# none, a few, and many per expert (the row count that a configuration allows
# chooses between the products' forms)
SPARE = {"exact": (0, 0), "spare": (37, 0), "roomy": (37, 1024)}


def with_spare(n, counts, spare):
    return max(1, n + SPARE[spare][0] + SPARE[spare][1] * len(counts))


def offsets(counts):
    c = torch.tensor([0] + list(counts), device="cuda").cumsum(0)
    return c.to(torch.int32)


def normal(*shape, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)


def quant_rows(v):
    b = v.float().view(v.shape[0], -1, 128)
    s = b.abs().amax(2) / 448
    q = torch.where(s[..., None] > 0, b / s[..., None], 0.0)
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(v.shape), s


def quant_weights(v):
    E, n, m = v.shape
    b = v.float().view(E, n // 128, 128, m // 128, 128)
    s = b.abs().amax((2, 4)) / 448
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(E, n, m), s.contiguous()


def poisoned(*shape, dtype=torch.bfloat16):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8 if dtype == torch.uint8 else torch.int16 if dtype == torch.bfloat16
           else torch.int32).fill_(-1 if dtype != torch.uint8 else 255)
    return t


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == 255).all())


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(BF16_CASES))
def test_gated_bf16(gpu, case, spare, keep):
    counts, H, F = BF16_CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    x, w13 = normal(rows, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1)
    x[n:] = float("nan")  # rows outside every segment
    hid, gu = poisoned(rows, F), poisoned(rows, 2 * F) if keep else None
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows))
    B.moe_expert_gated(h, offsets(counts), x, None, w13, None, hid, None, gu)
    assert B.moe_expert_read_status(h) == 0
    both, err = R.rows_times(x[:n].double(), w13.double(), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid[:n], *R.bf16_out(v, e))
    assert untouched(hid[n:])
    if keep:
        R.check("gate_up", gu[:n], *R.bf16_out(both, err))
        assert untouched(gu[n:])


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(FP8_CASES))
def test_gated_fp8(gpu, case, spare):
    counts, H, F = FP8_CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    x, xs = quant_rows(normal(rows, H))
    x[n:], xs[n:] = 0x7F, float("nan")
    w13, ws = quant_weights(normal(E, 2 * F, H, std=H ** -0.5, seed=1))
    hid, hs = poisoned(rows, F, dtype=torch.uint8), poisoned(rows, F // 128, dtype=torch.float32)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_FP8_E4M3))
    B.moe_expert_gated(h, offsets(counts), x, xs, w13, ws, hid, hs)
    assert B.moe_expert_read_status(h) == 0
    both, err = R.rows_times(R.dequant_rows(x[:n], xs[:n]), R.dequant_weights(w13, ws), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    amax = v.view(n, -1, 128).abs().amax(2)
    e_max = e.view(n, -1, 128).amax(2)
    R.check("hid_scale", hs[:n], amax / 448, (e_max + amax * 2.0 ** -22) / 448 + 2.0 ** -149)
    # a code is within half a step of h/s: 2^-4 of it, or 2^-10 near zero
    step = (amax + e_max).repeat_interleave(128, 1) / 448 * 2.0 ** -10
    R.check("hid", R.dequant_rows(hid[:n], hs[:n]), v, e + (v.abs() + e) * 2.0 ** -4 + step * 1.01)
    assert untouched(hid[n:]) and untouched(hs[n:])


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(BF16_CASES))
def test_down_bf16(gpu, case, spare):
    counts, H, F = BF16_CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    hid, w2 = normal(rows, F), normal(E, H, F, std=F ** -0.5, seed=1)
    hid[n:] = float("nan")
    y = poisoned(rows, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows))
    B.moe_expert_down(h, offsets(counts), hid, None, w2, None, y)
    assert B.moe_expert_read_status(h) == 0
    R.check("y", y[:n], *R.bf16_out(*R.rows_times(hid[:n].double(), w2.double(), counts)))
    assert untouched(y[n:])


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(FP8_CASES))
def test_down_fp8(gpu, case, spare):
    counts, H, F = FP8_CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    hid, hs = quant_rows(normal(rows, F))
    hid[n:], hs[n:] = 0x7F, float("nan")
    w2, ws = quant_weights(normal(E, H, F, std=F ** -0.5, seed=1))
    y = poisoned(rows, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_FP8_E4M3))
    B.moe_expert_down(h, offsets(counts), hid, hs, w2, ws, y)
    assert B.moe_expert_read_status(h) == 0
    v, e = R.rows_times(R.dequant_rows(hid[:n], hs[:n]), R.dequant_weights(w2, ws), counts)
    R.check("y", y[:n], *R.bf16_out(v, e))
    assert untouched(y[n:])


def backward_inputs(counts, H, F, rows):
    E = len(counts)
    return dict(x=normal(rows, H), gu=normal(rows, 2 * F, seed=1), hid=normal(rows, F, seed=2),
                dy=normal(rows, H, std=0.1, seed=3), w13=normal(E, 2 * F, H, std=H ** -0.5, seed=4),
                w2=normal(E, H, F, std=F ** -0.5, seed=5))


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(BF16_CASES))
def test_backward(gpu, case, spare):
    counts, H, F = BF16_CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    t = backward_inputs(counts, H, F, rows)
    for name in ("x", "gu", "hid", "dy"):
        t[name][n:] = float("nan")
    dx, dw13, dw2 = poisoned(rows, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, train=True))
    h.workspace[256:].fill_(255)  # the scratch gradient holds NaN past the segments
    B.moe_expert_backward(h, offsets(counts), t["x"], t["gu"], t["hid"], t["dy"], t["w13"],
                          t["w2"], dx, dw13, dw2)
    assert B.moe_expert_read_status(h) == 0
    d = {k: (v if k in ("w13", "w2") else v[:n]).double() for k, v in t.items()}
    want = R.backward(d["x"], d["gu"], d["hid"], d["dy"], d["w13"], d["w2"], counts)
    R.check("dx", dx[:n], *want[0])
    R.check("dw13", dw13, *want[1])
    R.check("dw2", dw2, *want[2])
    assert untouched(dx[n:])
    for e, c in enumerate(counts):
        if c == 0:
            assert not dw13[e].any() and not dw2[e].any()


def test_backward_parts(gpu):
    """dx alone and the weights' gradients alone are the whole call's, bit for bit."""
    counts, H, F = BF16_CASES["ragged"]
    E, rows = len(counts), sum(counts)
    t = backward_inputs(counts, H, F, rows)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, train=True))
    args = (h, offsets(counts), t["x"], t["gu"], t["hid"], t["dy"], t["w13"], t["w2"])
    whole = poisoned(rows, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(*args, *whole)
    dx, dw13, dw2 = poisoned(rows, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(*args, dx=dx)
    B.moe_expert_backward(*args, dw13=dw13, dw2=dw2)
    for a, b in zip(whole, (dx, dw13, dw2)):
        assert torch.equal(a, b)


def test_backward_against_differences(gpu):
    """The kernels' gradients along random directions against central differences of the
    block in 64 bits: L = <dy, h W2^T>, h = silu(x Wg^T) (x Wu^T)."""
    counts, H, F = [40, 0, 25, 1], 136, 72
    E, n = len(counts), sum(counts)
    x, w13, w2 = normal(n, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(
        E, H, F, std=F ** -0.5, seed=2)
    dy = normal(n, H, std=0.1, seed=3)
    off = offsets(counts)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, train=True))
    hid, gu = poisoned(n, F), poisoned(n, 2 * F)
    B.moe_expert_gated(h, off, x, None, w13, None, hid, None, gu)
    dx, dw13, dw2 = poisoned(n, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(h, off, x, gu, hid, dy, w13, w2, dx, dw13, dw2)

    def loss(x, w13, w2):
        both, _ = R.rows_times(x, w13, counts)
        y, _ = R.rows_times(both[:, :F] * torch.sigmoid(both[:, :F]) * both[:, F:], w2, counts)
        return (y * dy.double()).sum().item()

    at = [x.double(), w13.double(), w2.double()]
    for i, grad in enumerate((dx, dw13, dw2)):
        step = torch.randn(at[i].shape, dtype=torch.float64, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(i))
        eps = 1e-5
        hi = [v + eps * step if j == i else v for j, v in enumerate(at)]
        lo = [v - eps * step if j == i else v for j, v in enumerate(at)]
        want = (loss(*hi) - loss(*lo)) / (2 * eps)
        got = (grad.double() * step).sum().item()
        # gu, hid, dg, du and the result are each rounded to bf16: independent
        # errors of at most 2^-8 of terms whose root sum of squares is that of
        # the gradient's; five roundings, five standard deviations
        tol = 5 * 5 * R.BF16 * grad.double().norm().item()
        assert abs(got - want) <= tol, (i, got, want, tol)


@pytest.mark.parametrize("shape", [(1, 4, 8, 2, 64, 0), (2, 37, 16, 8, 264, 0),
                                   (4, 50, 8, 3, 1032, 0), (2, 64, 8, 4, 512, 20),
                                   (1, 1, 1, 1, 8, 0), (2, 33, 32, 12, 2056, 0),
                                   (8, 300, 64, 2, 136, 0)])
@pytest.mark.parametrize("fixed", [False, True])
def test_combine_backward(gpu, shape, fixed):
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, cap = shape
    if fixed and cap:
        pytest.skip("fixed slots have no capacity")
    T = P * Tr
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
    ids = torch.where(torch.rand(T, k, device="cuda", generator=g) < 0.1, -1, ids)
    ids[0] = -1  # a token without experts
    w = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)
    layer = MoeLayer(P, Tr, E, k, H, cap=cap)
    layer.layout(ids)
    (layer.dispatch_fixed_slots if fixed else layer.dispatch)(normal(T, H), w)
    rows = layer.slots["y"].shape[0] if fixed else layer.rows
    inv = layer.layout_view()["inv"].view(T, k).long()
    y, dout = normal(rows, H, seed=1), normal(T, H, seed=2)
    used = torch.zeros(rows, dtype=torch.bool, device="cuda")
    used[inv[inv >= 0]] = True
    y[~used] = float("nan")
    dy, dw = poisoned(rows, H), poisoned(T, k, dtype=torch.float32)
    B.moe_combine_backward(layer.handle, dout, y, w, dy, dw)
    assert layer.status() == 0
    kept = inv >= 0
    rowsel = inv.clamp_min(0)
    prod = torch.where(kept[..., None], y[rowsel].double(), 0.0) * dout.double()[:, None, :]
    R.check("dw", dw, prod.sum(2), prod.abs().sum(2) * (H + 8) * 2.0 ** -23)
    assert not dw[~kept].any()
    want = w.double()[:, :, None] * dout.double()[:, None, :]
    R.check("dy", dy[inv[kept]], *R.bf16_out(want[kept], want[kept].abs() * 2.0 ** -23))
    assert untouched(dy[~used])


@pytest.mark.parametrize("k", [1, 2, 4, 8])
@pytest.mark.parametrize("tokens,H", [(304, 1032), (305, 1032), (7, 4104), (304, 1024)])
def test_combine_backward_of_few_and_wide_tokens(gpu, k, tokens, H):
    test_combine_backward(gpu, (1, tokens, 16, k, H, 0), False)


def test_special_values_stay_in_their_rows(gpu):
    """An infinity or NaN of one row or one weight reaches only the results it enters."""
    counts, H, F = [3, 140, 2], 192, 136
    E, n = len(counts), sum(counts)
    x, w13 = normal(n, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1)
    x[2, 5], x[70, 0] = float("nan"), float("inf")
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n))
    hid = poisoned(n, F)
    B.moe_expert_gated(h, offsets(counts), x, None, w13, None, hid)
    fine = torch.isfinite(hid).all(1)
    assert not fine[2] and not fine[70]
    fine[2] = fine[70] = True
    assert fine.all()
    # a NaN in one expert's weights, next to a ragged reduction length
    t = backward_inputs(counts, H, F, n)
    t["w13"][1, 0, 0], t["w2"][1, 0, 0] = float("nan"), float("nan")
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, train=True))
    dx, dw13, dw2 = poisoned(n, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(h, offsets(counts), t["x"], t["gu"], t["hid"], t["dy"], t["w13"],
                          t["w2"], dx, dw13, dw2)
    assert torch.isfinite(dx[:3]).all() and torch.isfinite(dx[143:]).all()
    assert torch.isfinite(dw13[[0, 2]]).all() and torch.isfinite(dw2).all()
    # one row's NaN gradient stays in its expert's weights' gradients
    t = backward_inputs(counts, H, F, n)
    t["dy"][3, 0] = float("nan")
    B.moe_expert_backward(h, offsets(counts), t["x"], t["gu"], t["hid"], t["dy"], t["w13"],
                          t["w2"], dx, dw13, dw2)
    assert torch.isfinite(dw13[[0, 2]]).all() and torch.isfinite(dw2[[0, 2]]).all()
    assert not torch.isfinite(dw2[1]).all()


@pytest.mark.parametrize("counts", [[1, 0, 3, 2], [70, 0, 3, 200]])
def test_special_values_of_e4m3_rows(gpu, counts):
    """A NaN or an infinite scale of one row shows in that row's scales and results, and
    in no other's; few rows and many."""
    H, F, E, n = 256, 384, len(counts), sum(counts)
    x, xs = quant_rows(normal(n, H))
    xs[0, 1] = float("nan")  # the whole row's sums
    x[2, 3] = 0x7F           # one NaN code
    xs[n - 1, 0] = float("inf")
    w13, ws = quant_weights(normal(E, 2 * F, H, std=H ** -0.5, seed=1))
    w2, ws2 = quant_weights(normal(E, H, F, std=F ** -0.5, seed=2))
    hid, hs = poisoned(n, F, dtype=torch.uint8), poisoned(n, F // 128, dtype=torch.float32)
    y = poisoned(n, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, B.MOE_FP8_E4M3))
    B.moe_expert_gated(h, offsets(counts), x, xs, w13, ws, hid, hs)
    B.moe_expert_down(h, offsets(counts), hid, hs, w2, ws2, y)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[0, 2, n - 1]] = True
    assert torch.isfinite(hs[~bad]).all() and torch.isfinite(y[~bad]).all()
    assert not torch.isfinite(hs[bad]).any() and not torch.isfinite(y[bad]).any()


@pytest.mark.parametrize("counts", [[1, 0, 3, 2], [70, 0, 3, 200]])
def test_special_values_of_few_and_many_rows(gpu, counts):
    H, F, E, n = 264, 136, len(counts), sum(counts)
    x, w13 = normal(n, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1)
    w2 = normal(E, H, F, std=F ** -0.5, seed=2)
    x[1, 5], x[n - 1, 0] = float("nan"), float("-inf")
    hid, y = poisoned(n, F), poisoned(n, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n))
    B.moe_expert_gated(h, offsets(counts), x, None, w13, None, hid)
    B.moe_expert_down(h, offsets(counts), hid, None, w2, None, y)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[1, n - 1]] = True
    assert torch.isfinite(y[~bad]).all() and not torch.isfinite(y[bad]).any()


def test_large_gates_saturate(gpu):
    """Gates of +-200 and +-3e38: the sigmoid is 0 or 1, never NaN for finite products."""
    H, F = 8, 8
    x = torch.zeros(4, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([200.0, -200.0, 3e38, -3e38], device="cuda")
    w13 = torch.zeros(1, 2 * F, H, dtype=torch.bfloat16, device="cuda")
    w13[0, :F, 0] = 1.0
    w13[0, F:, 1] = 1.0
    x[:, 1] = 0.5
    hid = poisoned(4, F)
    h = B.moe_expert_create(B.make_expert_config(1, H, F, 4))
    B.moe_expert_gated(h, offsets([4]), x, None, w13, None, hid)
    want = torch.tensor([100.0, 0.0, 1.5e38, 0.0], device="cuda").bfloat16()
    assert torch.equal(hid, want[:, None].expand(4, F))


def test_fp8_zero_rows_and_blocks(gpu):
    counts, H, F = [3, 0, 2], 256, 256
    n = sum(counts)
    x, xs = quant_rows(normal(n, H))
    xs[1] = 0.0
    x[1] = 0
    w13, ws = quant_weights(normal(3, 2 * F, H, std=H ** -0.5, seed=1))
    hid, hs = poisoned(n, F, dtype=torch.uint8), poisoned(n, F // 128, dtype=torch.float32)
    h = B.moe_expert_create(B.make_expert_config(3, H, F, n, B.MOE_FP8_E4M3))
    B.moe_expert_gated(h, offsets(counts), x, xs, w13, ws, hid, hs)
    assert not hs[1].any() and not (hid[1] & 0x7F).any()
    assert torch.isfinite(hs).all()


def test_offsets_are_held_to_the_buffers(gpu):
    """Offsets past the buffers, negative or descending touch no row outside them."""
    H, F, rows = 64, 64, 40
    x, w13 = normal(rows + 8, H), normal(3, 2 * F, H, std=0.1, seed=1)
    w2 = normal(3, H, F, std=0.1, seed=2)
    for off in ([0, 10, 1 << 30, 7], [-5, 50, 20, 45], [0, 40, 40, 2147483647]):
        hid, y = poisoned(rows + 8, F), poisoned(rows + 8, H)
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        h = B.moe_expert_create(B.make_expert_config(3, H, F, rows))
        B.moe_expert_gated(h, o, x, None, w13, None, hid)
        B.moe_expert_down(h, o, hid, None, w2, None, y)
        assert B.moe_expert_read_status(h) == 0
        assert untouched(hid[rows:]) and untouched(y[rows:])


@pytest.mark.parametrize("spare", ["exact", "roomy"])
def test_rows_past_32_bit_offsets(gpu, spare):
    """Segments whose rows start more than 2^32 bytes (and 2^31 elements) into their buffers."""
    counts, H, F = [1, 130, 3], 4104, 16
    E, n = len(counts), sum(counts)
    first = (1 << 31) // H + 1
    rows = first + n + SPARE[spare][0]
    assert first * H * 2 > 1 << 32
    off = offsets(counts) + first
    big = lambda w: torch.zeros(rows, w, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    x, dy, dx = big(H), big(H), big(H)
    gu, hid = big(2 * F), big(F)
    tail = slice(first, first + n)
    x[tail], dy[tail] = normal(n, H), normal(n, H, std=0.1, seed=3)
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, train=True))
    B.moe_expert_gated(h, off, x, None, w13, None, hid, None, gu)
    both, err = R.rows_times(x[tail].double(), w13.double(), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid[tail], *R.bf16_out(v, e))
    R.check("gate_up", gu[tail], *R.bf16_out(both, err))
    B.moe_expert_down(h, off, hid, None, w2, None, dx)  # dx as y, for room
    R.check("y", dx[tail], *R.bf16_out(*R.rows_times(hid[tail].double(), w2.double(), counts)))
    dw13, dw2 = poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(h, off, x, gu, hid, dy, w13, w2, dx, dw13, dw2)
    want = R.backward(*(t[tail].double() for t in (x, gu, hid, dy)), w13.double(), w2.double(),
                      counts)
    for name, got, ref in (("dx", dx[tail], want[0]), ("dw13", dw13, want[1]),
                           ("dw2", dw2, want[2])):
        R.check(name, got, *ref)
    assert B.moe_expert_read_status(h) == 0 and not dx[:first].any() and not hid[:first].any()


@pytest.mark.parametrize("rows", [3, 140])
def test_weights_past_32_bit_offsets(gpu, rows):
    """The last expert's weights and gradients lie more than 2^32 bytes into theirs."""
    H, F = 4104, 1032
    E = (1 << 31) // (2 * F * H) + 2
    counts = [0] * (E - 1) + [rows]
    w13 = torch.zeros(E, 2 * F, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, F, dtype=torch.bfloat16, device="cuda")
    w13[-1], w2[-1] = normal(2 * F, H, std=H ** -0.5, seed=1), normal(H, F, std=F ** -0.5, seed=2)
    x, dy = normal(rows, H), normal(rows, H, std=0.1, seed=3)
    hid, gu, y, dx = poisoned(rows, F), poisoned(rows, 2 * F), poisoned(rows, H), poisoned(rows, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, train=True))
    off = offsets(counts)
    B.moe_expert_gated(h, off, x, None, w13, None, hid, None, gu)
    one = [rows]
    both, err = R.rows_times(x.double(), w13[-1:].double(), one)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid, *R.bf16_out(v, e))
    B.moe_expert_down(h, off, hid, None, w2, None, y)
    R.check("y", y, *R.bf16_out(*R.rows_times(hid.double(), w2[-1:].double(), one)))
    dw13, dw2 = poisoned(E, 2 * F, H), poisoned(E, H, F)
    B.moe_expert_backward(h, off, x, gu, hid, dy, w13, w2, dx, dw13, dw2)
    want = R.backward(*(t.double() for t in (x, gu, hid, dy, w13[-1:], w2[-1:])), one)
    R.check("dx", dx, *want[0])
    R.check("dw13", dw13[-1:], *want[1])
    R.check("dw2", dw2[-1:], *want[2])
    assert not dw13[:-1].any() and not dw2[:-1].any() and B.moe_expert_read_status(h) == 0


def test_waits_that_run_out_set_the_status(gpu):
    """With a wait limit of zero the kernel gives up, reports it and leaves; the next call
    with the usual limit is right."""
    counts, H, F = [300, 20], 512, 256
    n = sum(counts)
    x, w13 = normal(n, H), normal(2, 2 * F, H, std=H ** -0.5, seed=1)
    hid = poisoned(n, F)
    h = B.moe_expert_create(B.make_expert_config(2, H, F, n))
    off = offsets(counts)
    B.moe_expert_set_wait_limit(h, 0)
    B.moe_expert_gated(h, off, x, None, w13, None, hid)
    assert B.moe_expert_read_status(h) == B.MOE_STATUS_TIMEOUT
    assert B.moe_expert_read_status(h) == 0
    B.moe_expert_set_wait_limit(h, 1 << 32)
    B.moe_expert_gated(h, off, x, None, w13, None, hid)
    assert B.moe_expert_read_status(h) == 0
    both, err = R.rows_times(x.double(), w13.double(), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid, *R.bf16_out(v, e))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_few_rows_in_a_graph(gpu, dtype):
    """The single-token kernels (of e4m3 a cluster launch) in a captured graph."""
    counts, H, F = FP8_CASES["token_top8"]
    E, n = len(counts), sum(counts)
    off, x, fp8 = offsets(counts), normal(n, H), dtype == "fp8"
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    xs = s13 = s2 = hs = None
    hid = poisoned(n, F)
    if fp8:
        (x, xs), (w13, s13), (w2, s2) = quant_rows(x), quant_weights(w13), quant_weights(w2)
        hid, hs = poisoned(n, F, dtype=torch.uint8), poisoned(n, F // 128, dtype=torch.float32)
    y = poisoned(n, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, int(fp8)))

    def run():
        B.moe_expert_gated(h, off, x, xs, w13, s13, hid, hs)
        B.moe_expert_down(h, off, hid, hs, w2, s2, y)

    run()
    torch.cuda.synchronize()
    first = hid.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    hid.zero_(), y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(hid, first[0]) and torch.equal(y, first[1])


def test_same_inputs_same_bits_on_another_stream_and_in_a_graph(gpu):
    counts, H, F = BF16_CASES["ragged"]
    E, n = len(counts), sum(counts)
    t = backward_inputs(counts, H, F, n)
    off = offsets(counts)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, train=True))

    def run(stream=None):
        hid, gu, y = poisoned(n, F), poisoned(n, 2 * F), poisoned(n, H)
        dx, dw13, dw2 = poisoned(n, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
        torch.cuda.current_stream().synchronize()
        B.moe_expert_gated(h, off, t["x"], None, t["w13"], None, hid, None, gu, stream)
        B.moe_expert_down(h, off, hid, None, t["w2"], None, y, stream)
        B.moe_expert_backward(h, off, t["x"], gu, hid, t["dy"], t["w13"], t["w2"], dx, dw13, dw2,
                              stream)
        return hid, gu, y, dx, dw13, dw2

    first = run()
    side = torch.cuda.Stream()
    other = run(side)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    outs = [torch.empty_like(v) for v in first]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.moe_expert_gated(h, off, t["x"], None, t["w13"], None, outs[0], None, outs[1])
        B.moe_expert_down(h, off, outs[0], None, t["w2"], None, outs[2])
        B.moe_expert_backward(h, off, t["x"], outs[1], outs[0], t["dy"], t["w13"], t["w2"],
                              *outs[3:])
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_refusals(gpu):
    lib = B.load_library()
    n, H, F, E = 8, 64, 64, 2
    off = offsets([4, 4])
    x, w13, w2 = normal(n, H), normal(E, 2 * F, H), normal(E, H, F)
    hid, gu, y = poisoned(n, F), poisoned(n, 2 * F), poisoned(n, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n))

    def code(fn, *a):
        with pytest.raises(B.MoeError) as err:
            fn(*a)
        return err.value.code

    assert code(B.moe_expert_create, B.make_expert_config(E, H, F, n),
                torch.empty(64, dtype=torch.uint8, device="cuda")) == -3
    assert code(B.moe_expert_backward, h, off, x, gu, hid, y, w13, w2, y) == -5
    t = B.moe_expert_create(B.make_expert_config(E, H, F, n, train=True))
    assert code(B.moe_expert_backward, t, off, x, gu, hid, y, w13, w2) == -1
    assert code(B.moe_expert_backward, t, off, x, gu, hid, y, w13, w2, None, w13) == -1
    assert code(B.moe_expert_set_wait_limit, h, -1) == -1
    # bf16 rows take no scales, FP8 rows need them and keep no pre-activations
    s = torch.ones(64, device="cuda")
    assert code(B.moe_expert_gated, h, off, x, s, w13, None, hid) == -1
    q = B.moe_expert_create(B.make_expert_config(E, 128, 128, n, B.MOE_FP8_E4M3))
    x8, w8 = (torch.zeros(m, dtype=torch.uint8, device="cuda") for m in (n * 128, E * 256 * 128))
    with pytest.raises(ValueError):
        B.moe_expert_gated(q, off, x8, None, w8, s, x8, s)
    assert code(B.moe_expert_gated, q, off, x8, s, w8, s, x8.clone(), s, poisoned(n, 256)) == -1
    # tensors too small, strided, on the host, or misaligned
    with pytest.raises(ValueError):
        B.moe_expert_gated(h, off, x[:4], None, w13, None, hid)
    with pytest.raises(ValueError):
        B.moe_expert_gated(h, off, x, None, w13.transpose(1, 2), None, hid)
    with pytest.raises(ValueError):
        B.moe_expert_gated(h, off.cpu(), x, None, w13, None, hid)
    with pytest.raises(ValueError):
        B.moe_expert_gated(h, off, x.float(), None, w13, None, hid)
    odd = torch.empty(n * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(n, H)
    assert code(B.moe_expert_gated, h, off, odd, None, w13, None, hid) == -1
    assert lib.moe_expert_down(None, *[None] * 7) == -1
    shifted = torch.empty(1024, dtype=torch.uint8, device="cuda")[2:]  # 2 bytes past 4
    assert lib.moe_expert_gated(h.ptr, shifted.data_ptr(), x.data_ptr(), None, w13.data_ptr(),
                                None, hid.data_ptr(), None, None, None) == -1
    assert code(B.moe_combine_backward, B.moe_handle_create(B.make_config(1, n, E, 1, H)), y, y,
                torch.empty(n, device="cuda"), y, torch.empty(n, device="cuda")) == -5
    out = ctypes.c_void_p()
    assert lib.moe_expert_create(None, None, 0, ctypes.byref(out)) == -1


@pytest.mark.parametrize("counts", [[3, 900, 0, 40, 130, 5], [700, 0, 0, 0, 3, 900, 64, 1]])
def test_backward_of_uneven_experts(gpu, counts):
    """Weight gradients where few experts have most rows: their tiles are walked in another
    order."""
    H, F = 1032, 776
    E, n = len(counts), sum(counts)
    t = backward_inputs(counts, H, F, n)
    dx, dw13, dw2 = poisoned(n, H), poisoned(E, 2 * F, H), poisoned(E, H, F)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, n, train=True))
    B.moe_expert_backward(h, offsets(counts), t["x"], t["gu"], t["hid"], t["dy"], t["w13"],
                          t["w2"], dx, dw13, dw2)
    assert B.moe_expert_read_status(h) == 0
    want = R.backward(*(t[k].double() for k in ("x", "gu", "hid", "dy", "w13", "w2")), counts)
    for name, got, ref in (("dx", dx, want[0]), ("dw13", dw13, want[1]), ("dw2", dw2, want[2])):
        R.check(name, got, *ref)
