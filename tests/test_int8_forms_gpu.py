"""Every form of the int8 experts' products -- single rows, tiles of 64, 128 and
192 tokens, and codes widened to fp16 in memory -- with uneven segments, odd
sizes and several tiles a CTA: against 64 bits, with waits that run out, in
captured graphs, and past 32-bit offsets."""
import pytest
import torch

import expert_reference as R
import int8_reference as Q
from combine_top_histogram_gb300 import binding as B
from test_experts_gpu import offsets, poisoned, untouched
from test_int8_gpu import codes_of, gen, weights

pytestmark = pytest.mark.gpu


def uneven(E, rows, seed=0):
    """A random choice of experts, some without rows and one with several tiles."""
    n = torch.bincount(torch.randint(0, E, (rows,), generator=torch.Generator().manual_seed(seed)),
                       minlength=E).tolist()
    if E > 3:
        n[E - 1] += n[1] + n[2]
        n[1] = n[2] = 0
    return n


# op: form: (E, rows, H, F). The form follows from the rows a configuration can
# have, the experts and how many tiles there are: tiles of 64 tokens where those
# fill no more than a turn of the SMs, of 128 or 192 where the rows of an expert
# mostly fit one or where fewer weight conversions pay for it (up to 768
# experts), clusters of 2, 4 or 8 CTAs for a tile where those are few and the
# reduction is long, and widened codes from 2048 rows an expert, gated from 4096.
FORMS = {
    "gated": {"rows": (24, 60, 208, 272), "rows_one": (1, 21, 272, 400),
              "few": (6, 500, 336, 144), "few_turns": (256, 8000, 48, 400),
              "some": (32, 3200, 144, 656), "some_odd": (48, 4608, 208, 400),
              "many": (30, 5100, 208, 656), "many_short": (256, 40960, 16, 144),
              "few_split8": (1, 40, 2064, 144), "few_split4": (6, 200, 4112, 400),
              "some_split2": (10, 600, 4112, 656), "many_split8": (3, 450, 4112, 400),
              "many_even": (40, 6000, 128, 528), "many_experts": (1000, 160000, 48, 144),
              "widened": (2, 9000, 2048, 960), "widened_ragged": (3, 16001, 1040, 1040)},
    "down": {"rows": (24, 60, 272, 208), "rows_one": (1, 21, 400, 272),
             "few": (6, 500, 400, 336), "few_turns": (256, 8000, 400, 48),
             "some": (32, 3200, 1296, 80), "some_odd": (48, 4608, 784, 208),
             "many": (30, 5100, 1296, 208), "many_short": (256, 40960, 272, 16),
             "few_split8": (1, 40, 400, 2064), "few_split4": (6, 200, 1008, 4112),
             "some_split2": (10, 600, 1424, 4112), "many_split8": (3, 450, 912, 4112),
             "many_even": (40, 6000, 1040, 128), "many_experts": (1000, 160000, 272, 48),
             "widened": (2, 9000, 2048, 960), "widened_ragged": (3, 16001, 1040, 1040)},
}
CASES = [(op, form) for op in FORMS for form in FORMS[op]]


class Job:
    """One product's tensors; call() runs it, check() compares its results."""

    def __init__(self, op, E, rows, H, F, spare=0, seed=0):
        self.op, self.counts, self.n = op, uneven(E, rows, seed), rows
        K, N = (H, F) if op == "gated" else (F, H)
        total = rows + spare
        self.a, self.s = codes_of(total, K, seed=seed + 1), torch.empty(total, device="cuda")
        self.fill(seed)
        self.w, self.ws = weights(E, 2 * F if op == "gated" else H, K, seed + 3)
        self.off = offsets(self.counts)
        self.h = B.moe_expert_create(B.make_expert_config(E, H, F, total, B.MOE_INT8))
        if op == "gated":
            self.out = poisoned(total, N, dtype=torch.uint8).view(torch.int8)
            self.outs = poisoned(total, dtype=torch.float32)
        else:
            self.out, self.outs = poisoned(total, N), None

    def fill(self, seed):
        self.a.copy_(codes_of(*self.a.shape, seed=seed + 1))
        self.s.copy_(torch.rand(self.s.shape, device="cuda", generator=gen(seed + 2)) / 30)
        self.s[self.n:] = float("nan")

    def call(self):
        if self.op == "gated":
            B.moe_expert_gated(self.h, self.off, self.a, self.s, self.w, self.ws, self.out,
                               self.outs)
        else:
            B.moe_expert_down(self.h, self.off, self.a, self.s, self.w, self.ws, self.out)

    def check(self):
        n, args = self.n, (self.a[:self.n], self.s[:self.n], self.w, self.ws, self.counts)
        if self.op == "gated":
            Q.check_quantised(self.out[:n], self.outs[:n], *Q.gated(*args))
            assert untouched(self.outs[n:])
        else:
            R.check("y", self.out[:n], *R.bf16_out(*Q.rows_times(*args)))
        assert untouched(self.out[n:])


@pytest.mark.parametrize("op, form", CASES)
def test_form(gpu, op, form):
    job = Job(op, *FORMS[op][form], spare=3)
    job.call()
    assert B.moe_expert_read_status(job.h) == 0
    job.check()


def agree(op, E, rows, K, N, rooms):
    H, F = (K, N) if op == "gated" else (N, K)
    counts = uneven(E, rows)
    a, s = codes_of(rows, K, seed=1), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    w, ws = weights(E, 2 * F if op == "gated" else H, K, 3)
    got = []
    for room in rooms:
        ar = torch.zeros(room, K, dtype=torch.int8, device="cuda")
        sr, ar[:rows] = torch.zeros(room, device="cuda"), a
        sr[:rows] = s
        h = B.moe_expert_create(B.make_expert_config(E, H, F, room, B.MOE_INT8))
        if op == "gated":
            o, os = torch.zeros(room, N, dtype=torch.int8, device="cuda"), torch.zeros(
                room, device="cuda")
            B.moe_expert_gated(h, offsets(counts), ar, sr, w, ws, o, os)
            got.append((o[:rows].clone(), os[:rows].clone()))
        else:
            o = torch.zeros(room, N, dtype=torch.bfloat16, device="cuda")
            B.moe_expert_down(h, offsets(counts), ar, sr, w, ws, o)
            got.append((o[:rows].clone(),))
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))


@pytest.mark.parametrize("op", ["gated", "down"])
def test_forms_agree(gpu, op):
    """Sums of codes are exact here, so the forms give the same results, bit for bit: of the
    same rows, with room for so many more that other tiles are taken."""
    K, N = (512, 1296) if op == "gated" else (1296, 512)
    agree(op, 8, 60, K, N, (60, 64 * 8, 4096 * 8))  # single rows, tiles, widened


@pytest.mark.parametrize("op", ["gated", "down"])
def test_clusters_agree(gpu, op):
    """As above, of single rows, of clusters of 8 that share a tile, and of tiles without clusters."""
    agree(op, 2, 20, 2064, 144, (20, 80, 20000))


@pytest.mark.parametrize("cycles", [0, 500, 5000, 40000])
@pytest.mark.parametrize("op, form", [c for c in CASES if c[1] in (
    "few_turns", "some", "many", "few_split8", "some_split2", "many_split8", "widened")])
def test_waits_that_run_out(gpu, op, form, cycles):
    """Whatever wait runs out first, every kernel leaves and says so, and the next call with the
    usual limit is right."""
    job = Job(op, *FORMS[op][form])
    B.moe_expert_set_wait_limit(job.h, cycles)
    for _ in range(5):
        job.call()
        status = B.moe_expert_read_status(job.h)
        assert status == B.MOE_STATUS_TIMEOUT or (cycles > 0 and status == 0)
    B.moe_expert_set_wait_limit(job.h, 1 << 32)
    job.call()
    assert B.moe_expert_read_status(job.h) == 0
    job.check()


@pytest.mark.parametrize("op, form", [c for c in CASES if c[1] in (
    "rows", "few", "some", "many", "few_split4", "many_split8", "widened")])
def test_in_a_graph(gpu, op, form):
    job = Job(op, *FORMS[op][form])
    job.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        job.call()
    for seed in (20, 30):
        job.fill(seed)
        g.replay()
        job.check()


@pytest.mark.parametrize("form", ["few_split8", "many_split8"])
@pytest.mark.parametrize("op", ["gated", "down"])
def test_clusters_without_a_tile(gpu, op, form):
    """No rows at all, and then rows of one expert only."""
    job = Job(op, *FORMS[op][form])
    full, E = job.n, len(job.counts)
    for job.counts in ([0] * E, [0] * (E - 1) + [1]):
        job.n = sum(job.counts)
        job.off.copy_(offsets(job.counts))
        job.call()
        assert B.moe_expert_read_status(job.h) == 0
        if job.n:
            job.check()
        else:
            assert untouched(job.out[:full]) and (op == "down" or untouched(job.outs[:full]))


@pytest.mark.parametrize("F", [2064, 4112])
def test_wide_rows_of_h(gpu, F):
    """Rows longer than a CTA of the quantiser holds at once."""
    job = Job("gated", 3, 50, 64, F)
    job.call()
    job.check()


@pytest.mark.parametrize("op, E, rows", [("gated", 256, 310000), ("down", 256, 310000),
                                         ("gated", 2, 310000), ("down", 2, 310000)])
def test_offsets_past_32_bits(gpu, op, E, rows):
    """Row buffers of more than 2^31 elements (E = 2: as bytes and as fp16): the last segment."""
    H, F = 7168, 64
    last = 300
    counts = [(rows - last) // (E - 1)] * (E - 1) + [0]
    counts[0] += rows - last - sum(counts)
    counts[-1] = last
    K, N = (H, F) if op == "gated" else (F, H)
    a, s = codes_of(rows, K, seed=1), torch.rand(rows, device="cuda", generator=gen(2)) / 30
    w, ws = weights(E, 2 * F if op == "gated" else H, K, 3)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, B.MOE_INT8))
    lo = rows - last
    args = (a[lo:], s[lo:], w[-1:], ws[-1:], [last])
    if op == "gated":
        o, os = (torch.empty(rows, N, dtype=torch.int8, device="cuda"),
                 torch.empty(rows, device="cuda"))
        B.moe_expert_gated(h, offsets(counts), a, s, w, ws, o, os)
        Q.check_quantised(o[lo:], os[lo:], *Q.gated(*args))
    else:
        o = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        B.moe_expert_down(h, offsets(counts), a, s, w, ws, o)
        R.check("y", o[lo:], *R.bf16_out(*Q.rows_times(*args)))
    assert B.moe_expert_read_status(h) == 0


def test_dispatch_past_32_bits(gpu):
    """More than 2^31 receive bytes."""
    from combine_top_histogram_gb300 import MoeLayer
    P, Tr, E, k, H = 8, 4800, 16, 8, 7168
    layer = MoeLayer(P, Tr, E, k, H, B.MOE_INT8)
    x = torch.randn(P * Tr, H, device="cuda", generator=gen(1)).to(torch.bfloat16)
    ids = torch.rand(P * Tr, E, device="cuda", generator=gen(2)).topk(k, 1).indices.to(torch.int32)
    w = torch.rand(P * Tr, k, device="cuda", generator=gen(3))
    layer.layout(ids.contiguous())
    layer.dispatch(x, w)
    inv = layer.layout_view()["inv"].view(-1, k)
    at = torch.arange(P * Tr - 2000, P * Tr, device="cuda")
    codes, scale = Q.quantise(x[at])
    for j in range(k):
        r = inv[at, j].long()
        assert torch.equal(layer.recv_x[r], codes) and torch.equal(layer.recv_scale[r], scale)
    assert int(inv.max()) * H > 2 ** 31 and layer.status() == 0
