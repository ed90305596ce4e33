"""The forms of the expert kernels that the smaller tests do not reach: every split of the
few-rows kernels with several passes over an expert's rows, persistent loops that take several
turns, weight gradients of uneven experts in pairs, and whole-width tiles without pairs. Each
test works out from the device which form its sizes select."""
import pytest
import torch

import expert_reference as R
from combine_top_histogram_gb300 import binding as B
from test_experts_gpu import (backward_inputs, normal, offsets, poisoned, quant_rows, quant_weights,
                              test_combine_backward as check_combine_backward, untouched)

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def split_of(op, fp8, segments, n):
    """expert_rows.cu's choice: the warps that share one pair of groups of channels."""
    channels = 16 if op == "gated" else 32
    enough = (2 if op == "gated" and fp8 else 3) * sms()
    s = 1
    while s < 8 and segments * -(-n // (channels * (8 // s))) < enough:
        s *= 2
    return s


# 9 rows: a second pass of one; 16: two whole ones; 20: a remainder in the third
FEW = {3: 9, 10: 16, 17: 20, 31: 1}


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("op", ["gated", "down"])
def test_few_rows_in_every_split(gpu, op, dtype, split):
    E, rows, fp8 = 32, 48, dtype == "fp8"
    counts = [FEW.get(e, 0) for e in range(E)]
    n, first = sum(counts), 1  # a row before the segments and one after them
    assert n + 2 == rows
    unit = 128 if fp8 else 8
    width = next(w for w in range(unit, 1 << 14, unit) if split_of(op, fp8, E, w) == split)
    if not fp8 and split < 8:
        width += 8  # no group of channels divides it
    assert split_of(op, fp8, E, width) == split
    H, F = (640 if fp8 else 520, width) if op == "gated" else (width, 640 if fp8 else 520)
    off = offsets(counts) + first
    sel = slice(first, first + n)
    outside = [0, rows - 1]
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows, int(fp8)))
    K, N = (H, F) if op == "gated" else (F, H)
    a = normal(rows, K)
    w = normal(E, 2 * F if op == "gated" else H, K, std=K ** -0.5, seed=1)
    s = ws = None
    if fp8:
        (a, s), (w, ws) = quant_rows(a), quant_weights(w)
        a[outside], s[outside] = 0x7F, float("nan")
        v, e = R.rows_times(R.dequant_rows(a[sel], s[sel]), R.dequant_weights(w, ws), counts)
    else:
        a[outside] = float("nan")
        v, e = R.rows_times(a[sel].double(), w.double(), counts)
    if op == "down":
        y = poisoned(rows, H)
        B.moe_expert_down(h, off, a, s, w, ws, y)
        R.check("y", y[sel], *R.bf16_out(v, e))
        assert untouched(y[outside])
        return
    hid = poisoned(rows, F, dtype=torch.uint8 if fp8 else torch.bfloat16)
    hs = poisoned(rows, F // 128, dtype=torch.float32) if fp8 else None
    gu = None if fp8 else poisoned(rows, 2 * F)
    B.moe_expert_gated(h, off, a, s, w, ws, hid, hs, gu)
    assert untouched(hid[outside])
    x, xe = R.silu_product(v[:, :F], v[:, F:], e[:, :F], e[:, F:])
    if not fp8:
        R.check("hid", hid[sel], *R.bf16_out(x, xe))
        R.check("gate_up", gu[sel], *R.bf16_out(v, e))
        assert untouched(gu[outside])
        return
    assert untouched(hs[outside])
    amax, e_max = x.view(n, -1, 128).abs().amax(2), xe.view(n, -1, 128).amax(2)
    R.check("hid_scale", hs[sel], amax / 448, (e_max + amax * 2.0 ** -22) / 448 + 2.0 ** -149)
    step = (amax + e_max).repeat_interleave(128, 1) / 448 * 2.0 ** -10
    R.check("hid", R.dequant_rows(hid[sel], hs[sel]), x,
            xe + (x.abs() + xe) * 2.0 ** -4 + step * 1.01)


@pytest.mark.parametrize("k", [1, 2, 3, 4, 8, 12])
@pytest.mark.parametrize("turns", [2, 3])
@pytest.mark.parametrize("fixed", [False, True])
def test_combine_backward_of_several_turns(gpu, k, turns, fixed):
    """More tokens than CTAs: each takes a second and a third token beside the slots of the
    next; some take none."""
    check_combine_backward(gpu, (1, turns * 16 * sms() + 5, 16, k, 136, 0), fixed)


def check_backward(counts, H, F, rows):
    E, n = len(counts), sum(counts)
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
    for name, got, ref in (("dx", dx[:n], want[0]), ("dw13", dw13, want[1]), ("dw2", dw2, want[2])):
        R.check(name, got, *ref)
    assert untouched(dx[n:])


@pytest.mark.parametrize("counts", [[3, 2900, 0, 1040, 130, 537], [2405, 0, 1, 65, 2111, 63]])
def test_backward_of_uneven_experts_in_pairs(gpu, counts):
    """Hot experts whose rows end off a block of 64, and more 256 x 256 tiles of each gradient
    than two turns of the pairs: the walk turns round, and both CTAs clear their rows."""
    H, F, E, n = 1544, 1032, len(counts), sum(counts)
    rows = max(768 * E, n) + 3
    tiles = lambda a, b: -(-a // 256) * -(-b // 256) * E  # noqa: E731
    assert min(tiles(2 * F, H), tiles(H, F)) > 2 * (sms() // 2)
    assert n > 128 * E and 2 * max(counts) * E > 3 * n  # uneven
    check_backward(counts, H, F, rows)


def test_whole_width_tiles_without_pairs(gpu):
    """Ragged segments of fewer than 192 rows an expert, and more 128 x 256 tiles than two per
    SM, in every product."""
    E, H, F = 24, 2056, 2056
    counts = [(37 * e) % 191 for e in range(E)]
    n = sum(counts)
    rows = n + 3
    assert rows < 192 * E
    for width in (-(-F // 128), -(-F // 256), -(-H // 256)):  # gated; dgate; down and dx
        assert (rows // 128 + E) * width > 2 * sms()
    x, w13 = normal(rows, H), normal(E, 2 * F, H, std=H ** -0.5, seed=1)
    x[n:] = float("nan")
    hid, gu, y = poisoned(rows, F), poisoned(rows, 2 * F), poisoned(rows, H)
    w2 = normal(E, H, F, std=F ** -0.5, seed=2)
    h = B.moe_expert_create(B.make_expert_config(E, H, F, rows))
    B.moe_expert_gated(h, offsets(counts), x, None, w13, None, hid, None, gu)
    B.moe_expert_down(h, offsets(counts), hid, None, w2, None, y)
    assert B.moe_expert_read_status(h) == 0
    both, err = R.rows_times(x[:n].double(), w13.double(), counts)
    v, e = R.silu_product(both[:, :F], both[:, F:], err[:, :F], err[:, F:])
    R.check("hid", hid[:n], *R.bf16_out(v, e))
    R.check("gate_up", gu[:n], *R.bf16_out(both, err))
    R.check("y", y[:n], *R.bf16_out(*R.rows_times(hid[:n].double(), w2.double(), counts)))
    assert untouched(hid[n:]) and untouched(gu[n:]) and untouched(y[n:])
    del both, err, v, e
    check_backward(counts, H, F, rows)
