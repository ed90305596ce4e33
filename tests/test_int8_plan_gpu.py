"""The int8 products' forms against one another: where sums of codes are exact, single rows,
tiles, clusters that share a tile and widened codes give the same results bit for bit; and
every form repeats its own. Which kernels the cases reach is held on the host
(test_int8_plan_cpu.py) and for the SMs of this GPU."""
import pytest
import torch

from combine_top_histogram_gb300 import binding as B
from test_int8_forms_gpu import CASES, FORMS, Job, agree

pytestmark = pytest.mark.gpu

ROWS, WIDENED = (B.MOE_FORM_ROWS, 0, 0), (B.MOE_FORM_WIDENED, 0, 0)


def tiles(tokens, split=1):
    return (B.MOE_FORM_TILES, tokens, split)


def form(op, E, rows, H, F, sms):
    cfg = B.make_expert_config(E, H, F, rows, B.MOE_INT8)
    return B.moe_expert_form(cfg, op == "down", sms)


#: experts, rows, K, N (gated, down), room for so many rows, and the form that follows from each
AGREE = {
    "few_rows": (8, 20, 512, (1296, 1296), (20, 512, 32768), [ROWS, tiles(64), WIDENED]),
    "every_tile": (24, 60, 512, (1296, 1296), (60, 1000, 2500, 8000, 98304),
                   [ROWS, tiles(64), tiles(128), tiles(192), WIDENED]),
    "clusters_of_two": (10, 600, 4112, (656, 1312), (600, 20000), [tiles(128, 2), tiles(192)]),
    "clusters_of_eight": (3, 450, 4112, (400, 912), (450, 5000), [tiles(192, 8), tiles(192)]),
}


def agreement(op, case):
    E, rows, K, N, rooms, expected = AGREE[case]
    N = N[op == "down"]
    H, F = (K, N) if op == "gated" else (N, K)
    return E, rows, K, N, H, F, rooms, expected


@pytest.mark.parametrize("op", ["gated", "down"])
@pytest.mark.parametrize("case", list(AGREE))
def test_unlike_forms_agree(gpu, op, case):
    """Sums of K products of two random codes stay below 2^24: a code's deviation is 74, theirs
    K^0.5 74^2, of which 2^24 is more than forty at K = 4112."""
    E, rows, K, N, H, F, rooms, expected = agreement(op, case)
    sms = torch.cuda.get_device_properties(gpu).multi_processor_count
    assert [form(op, E, room, H, F, sms) for room in rooms] == expected
    agree(op, E, rows, K, N, rooms)


@pytest.mark.parametrize("op, name", CASES)
def test_every_form_repeats_itself(gpu, op, name):
    job = Job(op, *FORMS[op][name])
    outs = [t for t in (job.out, job.outs) if t is not None]
    job.call()
    first = [t.clone() for t in outs]
    for _ in range(3):
        for t in outs:
            t.view(torch.uint8).fill_(0x5a)
        job.call()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(first, outs))
    assert B.moe_expert_read_status(job.h) == 0
