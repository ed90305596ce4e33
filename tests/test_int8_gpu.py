"""The int8 path on the GPU: the dispatch's codes and scales against the plain
quantiser, code for code, in every form it has; the experts' products and the
quantised h against 64 bits; whole layers, captured ones, other streams; what is
not touched and what is refused."""
import ctypes
import importlib.util
import os

import pytest
import torch

import expert_reference as R
import int8_reference as Q
from combine_top_histogram_gb300 import binding as B
from test_experts_gpu import offsets, poisoned, untouched, with_spare, SPARE
from test_experts_layer_gpu import plain, routed

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tokens(T, H, seed=0, offset=0):
    """bf16 rows of unlike size, with the rows a quantiser can stumble over."""
    buf = torch.empty(T * H + offset, dtype=torch.bfloat16, device="cuda")
    x = buf[offset:].view(T, H)
    x.copy_(torch.randn(T, H, device="cuda", generator=gen(seed))
            * torch.exp2(torch.randint(-40, 40, (T, 1), device="cuda", generator=gen(seed + 1))))
    special = [0.0, 1e-39, 2.0 ** -133, float("inf"), float("nan"), 2.0 ** -64, 3e38, -1.0]
    for i, v in enumerate(special):
        if 2 * i + 1 < T:
            if v in (0.0, 1e-39, 2.0 ** -133, 2.0 ** -64):
                x[2 * i + 1] = 0.0
            x[2 * i + 1, (7 * i) % H] = v
    if T > 20:
        x[19, 0], x[19, -1] = float("-inf"), float("nan")
    return x


def codes_of(*shape, seed=0, low=-128):
    return torch.randint(low, 128, shape, dtype=torch.int8, device="cuda", generator=gen(seed))


# P, Tr, E, k, H, capacity, x offset in elements: direct and scanned layouts, rows shorter than a
# warp's share, of 2048 and 8192 values and past them, x on a 16-byte boundary only
DISPATCH = {"one": (1, 1, 1, 1, 16, 0, 0), "small": (2, 5, 4, 2, 48, 0, 0),
            "decode": (8, 17, 16, 8, 7168, 0, 0), "unaligned": (2, 40, 8, 2, 2064, 0, 8),
            "capacity": (4, 60, 8, 3, 528, 70, 0), "scanned": (4, 1500, 16, 4, 512, 0, 0),
            "wide": (2, 9, 4, 2, 8208, 0, 8), "very_wide": (1, 30, 4, 4, 20480, 0, 0),
            "many": (2, 3000, 8, 2, 2048, 0, 0)}


def check_dispatch(layer, x, ids, w, recv, scale, meta):
    codes, s = Q.quantise(x)
    inv = layer.layout_view()["inv"].view(layer.T, layer.k)
    t, j = (inv >= 0).nonzero(as_tuple=True)
    r = inv[t, j].long()
    assert torch.equal(recv[r], codes[t])
    assert torch.equal(scale[r].isnan(), s[t].isnan())
    assert torch.equal(scale[r].nan_to_num(nan=-1.0, posinf=-2.0),
                       s[t].nan_to_num(nan=-1.0, posinf=-2.0))
    assert torch.equal(meta["weight"][r], w[t, j]) and torch.equal(meta["slot"][r].long(), j)
    assert torch.equal(meta["src_token"][r].long(), t % layer.Tr)
    rest = torch.ones(recv.shape[0], dtype=torch.bool, device="cuda")
    rest[r] = False
    assert untouched(recv[rest]) and untouched(scale[rest])
    assert layer.status() == 0


@pytest.mark.parametrize("case, form", [
    (case, form) for form in ("dispatch", "two_stage", "fixed_slots", "tokens") for case in DISPATCH
    if form != "fixed_slots" or not DISPATCH[case][5]])  # fixed slots have no capacity
def test_dispatch(gpu, case, form):
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, cap, at = DISPATCH[case]
    T = P * Tr
    layer = MoeLayer(P, Tr, E, k, H, B.MOE_INT8, cap)
    x, (ids, w) = tokens(T, H, offset=at), routed(T, E, k)
    layer.layout(ids)
    if form == "fixed_slots":
        layer.dispatch_fixed_slots(x, w)  # allocates
        layer.layout(ids)
    layer.poison()
    if form == "dispatch":
        layer.dispatch(x, w)
    elif form == "two_stage":
        layer.dispatch_two_stage(x, w)
    elif form == "fixed_slots":
        layer.dispatch_fixed_slots(x, w)
    else:
        for lo, hi in ((0, T // 3), (T // 3, T)):
            B.moe_dispatch_tokens(layer.handle, lo, hi, x, w, layer.recv_x, layer.recv_scale,
                                  layer.meta)
    bufs = ((layer.slots["x"], layer.slots["scale"], layer.slots["meta"])
            if form == "fixed_slots" else (layer.recv_x, layer.recv_scale, layer.meta))
    check_dispatch(layer, x, ids, w, *bufs)


@pytest.mark.parametrize("chunks", [0, 3])
def test_standin_reads_the_rows_back(gpu, chunks):
    """y = bf16(c * (code * s)), and the layer's sum of them."""
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H = 2, 33, 8, 2, 272
    layer = MoeLayer(P, Tr, E, k, H, B.MOE_INT8)
    x, (ids, w) = torch.randn(P * Tr, H, device="cuda").to(torch.bfloat16), routed(P * Tr, E, k)
    c = torch.rand(E, device="cuda") + 0.5
    if chunks:
        out = layer.forward_pipelined(x, ids=ids, w=w, expert_scale=c, chunks=chunks)
    else:
        out = layer.forward(x, ids=ids, w=w, expert_scale=c)
    codes, s = Q.quantise(x)
    y = ((codes.float() * s[:, None])[:, None] * c[ids.clamp_min(0).long()][..., None]).to(
        torch.bfloat16)
    acc = torch.zeros(P * Tr, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        acc += torch.where(ids[:, j, None] >= 0, w[:, j, None].double() * y[:, j].double(), 0.0)
    size = (w[..., None].double() * y.double().abs()).sum(1)
    R.check("out", out, *R.bf16_out(acc, size * k * 2.0 ** -23))


# (counts of each expert, H, F): multiples of 16
CASES = {
    "one_row": ([1], 64, 64),
    "narrow": ([5, 3], 16, 16),
    "token_top8": ([1 if e % 4 == 1 else 0 for e in range(32)], 1024, 272),
    "token_pair": ([2, 0, 1, 1], 528, 272),
    "few_rows_one_expert": ([7, 0], 272, 80),
    "ragged": ([130, 1, 0, 257, 64], 208, 336),
    "tile_edges": ([128, 127, 129, 0, 256, 255], 192, 256),
    "wide_tile_edges": ([192, 191, 193, 0, 384, 33, 32, 1, 97], 224, 400),
    "long": ([1500, 3], 320, 144),
    "many_experts": ([(7 * e) % 23 for e in range(200)], 128, 96),
    "wide": ([33, 65], 2064, 1040),
    "deep": ([40, 0, 70], 7168, 2048),
    "none": ([0, 0, 0], 64, 64),
}


def weights(E, n, m, seed):
    return codes_of(E, n, m, seed=seed), (torch.rand(E, n, device="cuda", generator=gen(seed + 50))
                                          + 0.5) / (74 * m ** 0.5)


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(CASES))
def test_gated(gpu, case, spare):
    counts, H, F = CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    x, xs = codes_of(rows, H, seed=1), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    xs[n:] = float("nan")  # rows outside every segment
    w13, ws = weights(E, 2 * F, H, 3)
    hid = poisoned(rows, F, dtype=torch.uint8).view(torch.int8)
    hs = poisoned(rows, dtype=torch.float32)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_INT8))
    B.moe_expert_gated(h, offsets(counts), x, xs, w13, ws, hid, hs)
    assert B.moe_expert_read_status(h) == 0
    if n:
        Q.check_quantised(hid[:n], hs[:n], *Q.gated(x[:n], xs[:n], w13, ws, counts))
    assert untouched(hid[n:]) and untouched(hs[n:])


@pytest.mark.parametrize("spare", SPARE)
@pytest.mark.parametrize("case", list(CASES))
def test_down(gpu, case, spare):
    counts, H, F = CASES[case]
    E, n = len(counts), sum(counts)
    rows = with_spare(n, counts, spare)
    hid, hs = codes_of(rows, F, seed=1), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    hs[n:] = float("nan")
    w2, ws = weights(E, H, F, 3)
    y = poisoned(rows, H)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_INT8))
    B.moe_expert_down(h, offsets(counts), hid, hs, w2, ws, y)
    assert B.moe_expert_read_status(h) == 0
    R.check("y", y[:n], *R.bf16_out(*Q.rows_times(hid[:n], hs[:n], w2, ws, counts)))
    assert untouched(y[n:])


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("value", [-128, 127])
def test_largest_codes(gpu, rows, value):
    """Sums far past 2^24, all of one sign: within the bound of an fp32 sum."""
    H, F = 4096, 2048
    x = torch.full((rows, H), value, dtype=torch.int8, device="cuda")
    w2 = torch.full((2, F, H), -128, dtype=torch.int8, device="cuda")
    xs, ws = torch.full((rows,), 2.0 ** -7, device="cuda"), torch.full((2, F), 2.0 ** -12,
                                                                      device="cuda")
    y = poisoned(rows, F)
    h = B.moe_expert_create(B.make_expert_config(2, F, H, rows, B.MOE_INT8))
    counts = [rows - 2, 2]
    B.moe_expert_down(h, offsets(counts), x, xs, w2, ws, y)
    R.check("y", y, *R.bf16_out(*Q.rows_times(x, xs, w2, ws, counts)))


@pytest.mark.parametrize("rows", [3, 300])
def test_special_scales(gpu, rows):
    """A scale that is not finite shows in its rows' results and in no other's; an all-zero h has
    scale 0 and zero codes."""
    H, F = 256, 144
    x, xs = codes_of(rows, H), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    xs[0], xs[1], x[2] = float("nan"), float("inf"), 0
    w13, ws = weights(1, 2 * F, H, 3)
    hid, hs = poisoned(rows, F, dtype=torch.uint8).view(torch.int8), poisoned(
        rows, dtype=torch.float32)
    h = B.moe_expert_create(B.make_expert_config(1, H, F, rows, B.MOE_INT8))
    B.moe_expert_gated(h, offsets([rows]), x, xs, w13, ws, hid, hs)
    assert hs[0].isnan() and not hs[1].isfinite() and hs[2] == 0
    assert (hid[:3] == 0).all()
    if rows > 3:
        Q.check_quantised(hid[3:], hs[3:], *Q.gated(x[3:], xs[3:], w13, ws, [rows - 3]))
    w2, w2s = weights(1, H, F, 5)
    y = poisoned(rows, H)
    B.moe_expert_down(h, offsets([rows]), hid, hs, w2, w2s, y)
    assert y[:2].isnan().all() and (y[2] == 0).all() and y[3:].isfinite().all()


@pytest.mark.parametrize("room", [1, 300])
def test_least_values_of_h(gpu, room):
    """s = amax/127 of a few times the least fp32 value rounds to whole multiples of that: with
    amax 190 of them s is one, and codes end at 127."""
    H = F = 16
    x = torch.zeros(room, H, dtype=torch.int8, device="cuda")
    x[0, 0] = 1
    w = torch.zeros(1, 2 * F, H, dtype=torch.int8, device="cuda")
    w[0, :F, 0] = 95  # silu(95) = 95
    w[0, F:F + 4, 0] = torch.tensor([2, -2, 1, -1], dtype=torch.int8, device="cuda")
    ws = torch.ones(1, 2 * F, device="cuda")
    ws.view(torch.int32)[0, F:] = 1  # 2^-149
    h = B.moe_expert_create(B.make_expert_config(1, H, F, room, B.MOE_INT8))
    codes = torch.zeros(room, F, dtype=torch.int8, device="cuda")
    scale = torch.ones(room, device="cuda")
    B.moe_expert_gated(h, offsets([1]), x, torch.ones(room, device="cuda"), w, ws, codes, scale)
    assert scale.view(torch.int32)[0].item() == 1
    assert codes[0].tolist() == [127, -127, 95, -95] + [0] * 12


@pytest.mark.parametrize("rows", [6, 900])
def test_segments_of_the_callers_own(gpu, rows):
    """Offsets past the rows, below zero and descending are held to ascending ones in range; rows
    before the first and after the last stay as they were."""
    H, F, E = 128, 80, 4
    n = rows // 3
    raw = [n, n + 2, n - 1, n + 4, 10 * rows]  # the third end descends, the last is past the rows
    off = torch.tensor(raw, dtype=torch.int32, device="cuda")
    counts = [0, 2, 0, 2, rows - n - 4]
    x, xs = codes_of(rows, H), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    w13, ws = weights(E, 2 * F, H, 3)
    hid, hs = poisoned(rows, F, dtype=torch.uint8).view(torch.int8), poisoned(
        rows, dtype=torch.float32)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_INT8))
    B.moe_expert_gated(h, off, x, xs, w13, ws, hid, hs)
    v, e = Q.gated(x[n:], xs[n:], w13, ws, counts[1:])
    Q.check_quantised(hid[n:], hs[n:], v, e)
    assert untouched(hid[:n]) and untouched(hs[:n])
    off[0] = -7  # the first expert's segment begins at row 0
    B.moe_expert_gated(h, off, x, xs, w13, ws, hid, hs)
    v, e = Q.gated(x, xs, w13, ws, [n + 2, 0, 2, rows - n - 4])
    Q.check_quantised(hid, hs, v, e)


@pytest.mark.parametrize("case", [(1, 1, 16, 4, 128, 128, 0), (2, 37, 8, 2, 272, 80, 0),
                                  (4, 40, 8, 3, 144, 64, 45), (2, 700, 4, 2, 256, 192, 0)])
@pytest.mark.parametrize("graph", [False, True])
def test_layer(gpu, case, graph):
    """Route, dispatch, experts and combine, eagerly or captured and replayed with new tokens."""
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, F, cap = case
    T = P * Tr
    layer = MoeLayer(P, Tr, E, k, H, B.MOE_INT8, cap)
    w13, s13 = Q.quantise(torch.randn(E, 2 * F, H, device="cuda", generator=gen(1)) / H ** 0.5)
    w2, s2 = Q.quantise(torch.randn(E, H, F, device="cuda", generator=gen(2)) / F ** 0.5)
    layer.set_experts(w13, w2, s13, s2)
    x = torch.randn(T, H, device="cuda", generator=gen(3)).to(torch.bfloat16)
    logits = torch.randn(T, E, device="cuda", generator=gen(4))

    def check():
        kept = layer.layout_view()["inv"].view(T, k) >= 0
        want = plain(x.double(), Q.dequantise(w13, s13), Q.dequantise(w2, s2), layer.ids,
                     layer.w.double(), kept)
        # x and h are each off by half a step of their row's largest value at most, which is
        # amax / 254 an element; amax of normal rows is below 6 deviations (h: of a product of
        # two, below 20), so 6/254 and 20/254 of the norm, and three roundings to bf16
        off = (layer.out.double() - want).norm() / want.norm().clamp_min(1e-300)
        assert off <= 26 / 254 + 3 * R.BF16, float(off)
        assert layer.status() == 0 and layer.experts.status() == 0

    layer.forward(x, logits=logits)
    check()
    if graph:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            layer.forward(x, logits=logits)
        for seed in (5, 6):
            x.copy_(torch.randn(T, H, device="cuda", generator=gen(seed)))
            logits.copy_(torch.randn(T, E, device="cuda", generator=gen(seed + 10)))
            layer.out.fill_(float("nan"))
            g.replay()
            check()


def test_two_handles_on_two_streams(gpu):
    """Each has its own workspace: calls that overlap do not meet."""
    H, F, E, rows = 512, 256, 4, 600
    counts = [200, 0, 390, 10]
    jobs = []
    for i in range(2):
        x, xs = codes_of(rows, H, seed=i), torch.rand(rows, device="cuda", generator=gen(i)) / 30
        w13, ws = weights(E, 2 * F, H, 10 + i)
        jobs.append((B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_INT8)), x, xs,
                     w13, ws, torch.empty(rows, F, dtype=torch.int8, device="cuda"),
                     torch.empty(rows, device="cuda"), torch.cuda.Stream()))
    off = offsets(counts)
    torch.cuda.synchronize()
    for _ in range(20):
        for h, x, xs, w13, ws, hid, hs, st in jobs:
            B.moe_expert_gated(h, off, x, xs, w13, ws, hid, hs, stream=st)
    torch.cuda.synchronize()
    for h, x, xs, w13, ws, hid, hs, st in jobs:
        Q.check_quantised(hid, hs, *Q.gated(x, xs, w13, ws, counts))


def test_example(gpu):
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(os.path.dirname(__file__), "..", "examples",
                                          "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.serve_int8()


def test_refusals(gpu, cuda_lib):
    from combine_top_histogram_gb300 import MoeError, MoeLayer
    with pytest.raises(MoeError):
        MoeLayer(1, 4, 2, 1, 24, B.MOE_INT8)  # H is a multiple of 16
    layer = MoeLayer(2, 8, 4, 2, 64, B.MOE_INT8)
    x, (ids, w) = tokens(16, 64), routed(16, 4, 2)
    for mode in ("fused", "allgather"):
        with pytest.raises(ValueError):
            layer.forward(x, ids=ids, w=w, **{mode: True})
    layer.layout(ids)
    with pytest.raises(MoeError) as err:
        B.moe_layout_dispatch_fused(layer.handle, None, ids, w, x, layer.recv_x, layer.recv_scale,
                                    layer.meta)
    assert err.value.code == -2
    with pytest.raises(MoeError) as err:
        B.moe_dispatch_allgather(layer.handle, x, w, layer.recv_x, layer.recv_scale, layer.recv_x,
                                 layer.recv_scale, layer.meta)
    assert err.value.code == -2
    with pytest.raises(MoeError):
        B.moe_dispatch(layer.handle, x, w, layer.recv_x, None, layer.meta)  # no scales
    bf = torch.zeros(4, 32, 64, dtype=torch.bfloat16, device="cuda")
    w13, w2 = codes_of(4, 32, 64), codes_of(4, 64, 16)
    s13, s2 = torch.ones(4, 32, device="cuda"), torch.ones(4, 64, device="cuda")
    for args in ((bf, bf[:, :16].transpose(1, 2).contiguous()), (w13, w2), (w13, w2, s13),
                 (w13, bf[:, :16].transpose(1, 2).contiguous(), s13, s2)):
        with pytest.raises(ValueError):
            layer.set_experts(*args)
    with pytest.raises(MoeError):
        layer.set_experts(w13, w2, s13, s2, train=True)
    layer.set_experts(w13, w2, s13, s2)
    layer.forward(x, ids=ids, w=w)
    with pytest.raises(ValueError):
        layer.backward(x, w)
    other = MoeLayer(2, 8, 4, 2, 64)
    with pytest.raises(ValueError):
        other.set_experts(w13, w2, s13, s2)
    h = layer.experts.handle
    off = layer.layout_view()["expert_offset"]
    e = layer.experts
    with pytest.raises(ValueError, match="hid_scale"):
        B.moe_expert_down(h, off, e.hid, e.hid_scale[:-1].contiguous(), w2, s2, layer.y)
    with pytest.raises(ValueError, match="w2_scale"):
        B.moe_expert_down(h, off, e.hid, e.hid_scale, w2, s2[:-1], layer.y)
    # misaligned buffers, at the C entry
    p = [ctypes.c_void_p(t.data_ptr()) for t in (off, layer.recv_x, layer.recv_scale, w13, s13,
                                                 e.hid, e.hid_scale)]
    for i in (1, 3, 5):
        q = list(p)
        q[i] = ctypes.c_void_p(p[i].value + 8)
        assert cuda_lib.moe_expert_gated(h.ptr, *q, None, None) == -1
    for i in (2, 4, 6):
        q = list(p)
        q[i] = None
        assert cuda_lib.moe_expert_gated(h.ptr, *q, None, None) == -1
    assert cuda_lib.moe_expert_gated(h.ptr, *p, ctypes.c_void_p(layer.y.data_ptr()), None) == -1
