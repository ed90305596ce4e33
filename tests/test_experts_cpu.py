"""Host-side rules of the expert operators: sizes they accept, workspace sizes,
and entry points called without a handle. No GPU."""
import ctypes

import pytest

from combine_top_histogram_gb300 import binding as B


def test_workspace_bytes(cuda_lib):
    assert B.moe_expert_workspace_bytes(B.make_expert_config(4, 64, 64, 100)) == 256
    assert B.moe_expert_workspace_bytes(
        B.make_expert_config(4, 64, 40, 100, train=True)) == 256 + 100 * 2 * 40 * 2
    # a training layer past 2^32 bytes
    assert B.moe_expert_workspace_bytes(
        B.make_expert_config(8, 4096, 1408, 1 << 20, train=True)) == 256 + (1 << 20) * 2 * 1408 * 2


@pytest.mark.parametrize("cfg, rc", [
    ((0, 64, 64, 8), -1), ((2, 0, 64, 8), -1), ((2, 64, 0, 8), -1), ((2, 64, 64, 0), -1),
    ((2, 64, 64, 8, 7), -1), ((2, 60, 64, 8), -2), ((2, 64, 60, 8), -2), ((1025, 64, 64, 8), -2),
    ((2, 64, 128, 8, B.MOE_FP8_E4M3), -2), ((2, 128, 64, 8, B.MOE_FP8_E4M3), -2),
    ((2, 128, 128, 8, B.MOE_FP8_E4M3, True), -2), ((2, 64, 64, (1 << 31) - 1), -2),
])
def test_refused_configurations(cuda_lib, cfg, rc):
    c = B.make_expert_config(*cfg)
    assert B.moe_expert_workspace_bytes(c) == 0
    out = ctypes.c_void_p()
    assert cuda_lib.moe_expert_create(ctypes.byref(c), ctypes.c_void_p(256), 1 << 20,
                                      ctypes.byref(out)) == rc
    assert not out.value


def test_calls_without_a_handle(cuda_lib):
    assert cuda_lib.moe_expert_gated(*[None] * 10) == -1
    assert cuda_lib.moe_expert_down(*[None] * 8) == -1
    assert cuda_lib.moe_expert_backward(*[None] * 12) == -1
    assert cuda_lib.moe_combine_backward(*[None] * 7) == -1
    assert cuda_lib.moe_expert_set_wait_limit(None, 1) == -1
    assert cuda_lib.moe_expert_read_status(None, None, None) == -1
    assert cuda_lib.moe_expert_destroy(None) == 0
