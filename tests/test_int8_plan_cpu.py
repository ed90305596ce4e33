"""Which kernels the int8 products of a configuration run (no GPU): what the tests of every
form (test_int8_forms_gpu.py, test_int8_plan_gpu.py) say that they reach is what the host
chooses, so that a rule that is measured anew takes no kernel out of the tests unseen."""
import ctypes

import pytest

import test_int8_forms_gpu as forms
import test_int8_plan_gpu as plan
from combine_top_histogram_gb300 import binding as B

SMS = 152  # of a GB300

#: form: (kernels, rows of a tile, CTAs that share one)
EXPECTED = {
    "rows": plan.ROWS, "rows_one": plan.ROWS, "few": (B.MOE_FORM_TILES, 64, 1),
    "few_turns": (B.MOE_FORM_TILES, 64, 1), "some": (B.MOE_FORM_TILES, 128, 1),
    "some_odd": (B.MOE_FORM_TILES, 128, 1), "many": (B.MOE_FORM_TILES, 192, 1),
    "many_short": (B.MOE_FORM_TILES, 192, 1), "many_even": (B.MOE_FORM_TILES, 192, 1),
    "many_experts": (B.MOE_FORM_TILES, 128, 1),  # too many for tiles of 192
    "few_split8": (B.MOE_FORM_TILES, 64, 8), "few_split4": (B.MOE_FORM_TILES, 64, 4),
    "some_split2": (B.MOE_FORM_TILES, 128, 2), "many_split8": (B.MOE_FORM_TILES, 192, 8),
    "widened": plan.WIDENED, "widened_ragged": plan.WIDENED,
}


@pytest.mark.parametrize("spare", [0, 3])
@pytest.mark.parametrize("op, form", forms.CASES)
def test_forms_are_what_they_are_called(cuda_lib, op, form, spare):
    E, rows, H, F = forms.FORMS[op][form]
    assert plan.form(op, E, rows + spare, H, F, SMS) == EXPECTED[form]


@pytest.mark.parametrize("op", ["gated", "down"])
@pytest.mark.parametrize("case", list(plan.AGREE))
def test_agreement_compares_unlike_kernels(cuda_lib, op, case):
    E, rows, _, _, H, F, rooms, expected = plan.agreement(op, case)
    assert rows <= min(rooms)
    got = [plan.form(op, E, room, H, F, SMS) for room in rooms]
    assert got == expected and len(set(got)) == len(got)


def test_other_types_and_refusals(cuda_lib):
    bf16 = B.make_expert_config(8, 128, 128, 24)
    assert B.moe_expert_form(bf16, False, SMS) == plan.ROWS
    assert B.moe_expert_form(B.make_expert_config(8, 128, 128, 65), True, SMS) == (
        B.MOE_FORM_TILES, 0, 0)
    e4m3 = B.make_expert_config(32, 128, 128, 60, B.MOE_FP8_E4M3)
    assert B.moe_expert_form(e4m3, False, SMS) == plan.ROWS
    assert B.moe_expert_form(e4m3, True, SMS) == (B.MOE_FORM_TILES, 0, 0)
    for cfg, sms in ((B.make_expert_config(8, 24, 128, 24, B.MOE_INT8), SMS), (bf16, 0)):
        with pytest.raises(B.MoeError):
            B.moe_expert_form(cfg, False, sms)
    out = B.moe_expert_form_t()
    assert cuda_lib.moe_expert_form(ctypes.byref(bf16), 2, SMS, ctypes.byref(out)) == -1
    assert cuda_lib.moe_expert_form(ctypes.byref(bf16), 0, SMS, None) == -1
    assert cuda_lib.moe_expert_form(None, 0, SMS, ctypes.byref(out)) == -1


def test_widening_needs_both_many_rows_an_expert_and_a_large_product(cuda_lib):
    """4096 rows of one expert, and rows x H x F of 2^33 or 2^34."""
    H, F, rows = 2048, 1024, 4096
    h32 = 256 + rows * F * 4
    small = B.make_expert_config(1, H, F, rows, B.MOE_INT8)
    assert B.moe_expert_workspace_bytes(small) == h32
    assert B.moe_expert_form(small, True, SMS)[0] == B.MOE_FORM_TILES
    large = B.make_expert_config(1, 2 * H, F, rows, B.MOE_INT8)
    assert B.moe_expert_workspace_bytes(large) == h32 + rows * 2 * H * 2 + 2 * F * 2 * H * 2
    assert B.moe_expert_form(large, True, SMS) == plan.WIDENED
    assert B.moe_expert_form(large, False, SMS) == plan.WIDENED
