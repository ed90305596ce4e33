"""The expert operators at the edges of their contracts: states of a layer that a call
order leaves behind, descending offsets, other streams, ties of e4m3 codes, waits that run
out in pairs of CTAs; and the kernel forms that only larger or uneven calls reach."""
import pytest
import torch

import expert_reference as R
from combine_top_histogram_gb300 import binding as B
from test_experts_gpu import normal, poisoned, quant_rows, quant_weights, untouched

pytestmark = pytest.mark.gpu


def test_combine_backward_after_a_partial_dispatch(gpu):
    """Tokens that a chunked dispatch has not covered since a fixed-slot one still name slot
    rows: those past the receive rows are reported and touch nothing."""
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H = 1, 64, 16, 2, 136
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.rand(Tr, E, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn(Tr, k, device="cuda", generator=g), 1)
    layer, x = MoeLayer(P, Tr, E, k, H), normal(Tr, H)
    layer.layout(ids)
    layer.dispatch_fixed_slots(x, w)
    B.moe_dispatch_tokens(layer.handle, 0, Tr // 2, x, w, layer.recv_x, None, layer.meta)
    inv = layer.layout_view()["inv"].view(Tr, k).long().clone()
    past = inv >= layer.rows
    assert past[Tr // 2:].any() and not past[:Tr // 2].any()
    y, dout = normal(layer.rows, H, seed=1), normal(Tr, H, seed=2)
    whole = poisoned(B.moe_fixed_slot_rows(layer.cfg), H)  # room for every row inv names
    dy, dw = whole[:layer.rows], poisoned(Tr, k, dtype=torch.float32)
    B.moe_combine_backward(layer.handle, dout, y, w, dy, dw)
    assert layer.status() == B.MOE_STATUS_BOUNDS and layer.status() == 0
    assert untouched(whole[layer.rows:]) and not dw[past].any()
    first = inv[:Tr // 2]
    prod = y[first].double() * dout[:Tr // 2].double()[:, None, :]
    R.check("dw", dw[:Tr // 2], prod.sum(2), prod.abs().sum(2) * (H + 8) * 2.0 ** -23)


def busy(ms=100):
    """Work on the current stream that takes about so long."""
    a = torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(a)
    for _ in range(ms):  # 0.6 to 0.8 ms each
        torch.matmul(a, a, out=out)
        torch.matmul(a, a, out=out)


def test_layer_on_a_side_stream_beside_a_busy_one(gpu):
    """The first forward and backward of a training layer on a stream of its own, while the
    current stream has work queued, give what they give on the current stream."""
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H, F = 2, 37, 8, 2, 264, 72
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    x, dout = normal(P * Tr, H), normal(P * Tr, H, std=0.1, seed=4)
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.rand(P * Tr, E, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn(P * Tr, k, device="cuda", generator=g), 1)

    def step(stream=None):
        layer = MoeLayer(P, Tr, E, k, H)
        busy(1)
        layer.set_experts(w13, w2, train=True)
        side = stream is not None
        if side:
            busy()
        out = layer.forward(x, ids=ids, w=w, stream=stream)
        grad = layer.backward(dout, w, stream=stream)
        if side:
            stream.synchronize()
            assert not torch.cuda.current_stream().query()  # it was busy all the while
        return layer, [out, *(grad[n] for n in ("dx", "dw", "dw13", "dw2"))]

    keep, want = step()
    torch.cuda.synchronize()
    other, got = step(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert keep.status() == other.status() == 0
    assert keep.experts.status() == other.experts.status() == 0


DESCENDING = [[0, 6, 2, 8], [0, 1 << 30, 3, 7], [-5, 4, -1, 8], [0, 8, 0, 8], [8, 0, 5, 8],
              [2, 9, 2147483647, -2147483648], [0, 0, 0, 0], [5, 3, 2, 1]]


@pytest.mark.parametrize("off", DESCENDING)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("roomy", [False, True])
def test_descending_offsets_are_clamped_alike(gpu, off, dtype, roomy):
    """Few rows and many (the buffers' room decides): the segments of the running maximum of the
    offsets, each held to the buffers."""
    E, H, F, rows, fp8 = 3, 256, 128, 8, dtype == "fp8"
    room = 4096 if roomy else rows
    top, clamped = 0, []
    for i, o in enumerate(off):
        top = max(top if i else 0, min(max(o, 0), room))
        clamped.append(top)
    x, w13 = normal(room, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1)
    w2 = normal(E, H, F, std=F ** -0.5, seed=2)
    xs = s13 = s2 = None
    if fp8:
        (x, xs), (w13, s13), (w2, s2) = quant_rows(x), quant_weights(w13), quant_weights(w2)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, room, int(fp8)))

    def run(offsets):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        hid = poisoned(room, F, dtype=torch.uint8 if fp8 else torch.bfloat16)
        hs = poisoned(room, F // 128, dtype=torch.float32) if fp8 else None
        y = poisoned(room, H)
        B.moe_expert_gated(h, o, x, xs, w13, s13, hid, hs)
        given = hid.clone()
        if fp8:  # every row finite, for the rows that only `down` is given
            given, scale = quant_rows(normal(room, F, seed=3))
        B.moe_expert_down(h, o, given, scale if fp8 else None, w2, s2, y)
        return [t for t in (hid, hs, y) if t is not None]

    got, want = run(off), run(clamped)
    assert B.moe_expert_read_status(h) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert untouched(a[:clamped[0]]) and untouched(a[clamped[-1]:])
        assert all(not untouched(r) for r in a[clamped[0]:clamped[-1]])


def test_codes_beside_ties_are_those_of_the_quotient(gpu):
    """h within a few units of s times a midpoint of two e4m3 values: few rows and many give the
    same scales and the codes of the quotient h / s, rounded once before the code is."""
    E, per, H, F = 16, 3, 128, 256
    n = E * per
    g = torch.Generator(device="cuda").manual_seed(5)
    e = torch.randint(4, 8, (E, F), device="cuda", generator=g)
    c = (8 + torch.randint(0, 8, (E, F), device="cuda", generator=g)) * 2.0 ** (e - 3)
    w = torch.zeros(E, 2 * F, H, device="cuda")
    w[:, :F, 0] = 64.0         # the sigmoid of 32 or more is 1
    w[:, F:, 0] = c            # 16 to 240, and half a step above
    w[:, F:, 1] = 2.0 ** (e - 4)
    w[:, F::128, 0], w[:, F::128, 1] = 448.0, 0.0  # the largest of each 128 channels
    codes = lambda v: v.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    ws = torch.ones(E, 2 * F // 128, 1, device="cuda")
    ws[:, F // 128:] = 0.5 + torch.rand(E, F // 128, 1, device="cuda", generator=g)
    x = torch.zeros(n, H, device="cuda")
    x[:, :2] = 1.0
    xs = 0.5 + 0.5 * torch.rand(n, 1, device="cuda", generator=g)
    off = torch.arange(0, n + 1, per, dtype=torch.int32, device="cuda")

    def run(rows):
        big = lambda t: torch.cat([t, t.new_zeros(rows - n, *t.shape[1:])])  # noqa: E731
        hid = poisoned(rows, F, dtype=torch.uint8)
        hs = poisoned(rows, F // 128, dtype=torch.float32)
        h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_FP8_E4M3))
        B.moe_expert_gated(h, off, big(codes(x)), big(xs), codes(w), ws, hid, hs)
        return hid[:n], hs[:n]

    (few, few_s), (many, many_s) = run(n), run(4096)
    gate = 64 * xs                                               # exact
    of_row = torch.arange(E, device="cuda").repeat_interleave(per)
    scale = (xs * ws[of_row, F // 128:, 0]).repeat_interleave(128, 1)  # one rounding
    h = gate * ((w[of_row, F:, 0] + w[of_row, F:, 1]) * scale)   # one rounding each
    amax = h.view(n, -1, 128).amax(2)
    s = amax / torch.full_like(amax, 448.0)  # torch multiplies by a scalar's reciprocal
    want = codes(h / s.repeat_interleave(128, 1))
    for got, got_s in ((few, few_s), (many, many_s)):
        assert torch.equal(got_s, s) and torch.equal(got, want)


@pytest.mark.parametrize("cycles", [0, 300, 2000, 8000, 30000])
def test_waits_that_run_out_in_pairs(gpu, cycles):
    """Two CTAs on one tile (enough rows an expert, ragged segments): whatever wait runs out
    first, every kernel leaves and says so, and the next call with the usual limit is right."""
    counts, H, F = [1300, 0, 215, 1029], 1032, 520
    E, n = len(counts), sum(counts)
    rows = 768 * E + 5
    x, gu, hid = normal(rows, H), poisoned(rows, 2 * F), poisoned(rows, F)
    w13, w2 = normal(E, 2 * F, H, std=H ** -0.5, seed=1), normal(E, H, F, std=F ** -0.5, seed=2)
    dy, y, dx = normal(rows, H, std=0.1, seed=3), poisoned(rows, H), poisoned(rows, H)
    dw13, dw2 = poisoned(E, 2 * F, H), poisoned(E, H, F)
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, train=True))
    calls = (lambda: B.moe_expert_gated(h, off, x, None, w13, None, hid, None, gu),
             lambda: B.moe_expert_down(h, off, hid, None, w2, None, y),
             lambda: B.moe_expert_backward(h, off, x, gu, hid, dy, w13, w2, dx, dw13, dw2))
    B.moe_expert_set_wait_limit(h, cycles)
    for _ in range(5):
        for call in calls:
            call()
            status = B.moe_expert_read_status(h)
            assert status == B.MOE_STATUS_TIMEOUT or (cycles > 0 and status == 0)
    B.moe_expert_set_wait_limit(h, 1 << 32)
    for call in calls:
        call()
    assert B.moe_expert_read_status(h) == 0
    both, err = R.rows_times(x[:n].double(), w13.double(), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid[:n], *R.bf16_out(v, e))
    R.check("y", y[:n], *R.bf16_out(*R.rows_times(hid[:n].double(), w2.double(), counts)))
    want = R.backward(*(t[:n].double() for t in (x, gu, hid, dy)), w13.double(), w2.double(),
                      counts)
    for name, got, ref in (("dx", dx[:n], want[0]), ("dw13", dw13, want[1]), ("dw2", dw2, want[2])):
        R.check(name, got, *ref)


def test_handles_made_beside_a_busy_stream(gpu):
    """A handle's control words are cleared when its creation returns, and a status that was read
    is cleared on its stream, whatever the default stream has queued."""
    from combine_top_histogram_gb300 import MoeLayer
    H, F, rows = 512, 256, 320
    x, w13 = normal(rows, H), normal(2, 2 * F, H, std=H ** -0.5, seed=1)
    hid = poisoned(rows, F)
    off = torch.tensor([0, 300, 320], dtype=torch.int32, device="cuda")
    P, Tr, E, k = 2, 37, 8, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = torch.rand(P * Tr, E, device="cuda", generator=g).topk(k, 1).indices.to(torch.int32)
    w = torch.softmax(torch.randn(P * Tr, k, device="cuda", generator=g), 1)
    t = normal(P * Tr, 64)
    want = MoeLayer(P, Tr, E, k, 64).forward(t, ids=ids, w=w).clone()
    dirty = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirty  # the next workspaces' memory
    side = torch.cuda.Stream()
    busy()
    h = B.moe_expert_create(B.make_expert_config(2, H, F, rows))
    busy()
    B.moe_expert_set_wait_limit(h, 0)
    for _ in range(3):
        B.moe_expert_gated(h, off, x, None, w13, None, hid, stream=side)
        assert B.moe_expert_read_status(h, side) == B.MOE_STATUS_TIMEOUT
        assert B.moe_expert_read_status(h, side) == 0
    assert not torch.cuda.current_stream().query()
    layer = MoeLayer(P, Tr, E, k, 64)
    busy()
    layer.forward(t, ids=ids, w=w, stream=side)
    assert layer.status(side) == 0
    assert not torch.cuda.current_stream().query()
    assert torch.equal(layer.out, want)
