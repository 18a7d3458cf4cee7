"""Host-only checks of the plan queries: which kernels the sizes named beside the rules, and those of
the GPU tests, take."""

import ctypes

import pytest

import unpermute_ffnwb_batching_amd as F
from test_expert_ffn_checks import _layer


def _layer_plan(T, K, E, H, inter, bf16=False):
    over = dict(weight_dtype=1, w13_scale=None, w2_scale=None) if bf16 else {}
    return F.moe_layer_plan(_layer(num_tokens=T, slots=K, hidden=H, inter_size=inter, num_experts=E, **over))


def test_layer_plan_refuses_what_the_call_refuses():
    info = F.LayerPlanInfo()
    assert F.lib().moe_layer_plan(None, ctypes.byref(info)) == F.FFNWB_ERR_PARAM_NULLPTR
    assert F.lib().moe_layer_plan(ctypes.byref(_layer()), None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert F.lib().moe_layer_plan(ctypes.byref(_layer(num_tokens=65)), ctypes.byref(info)) == F.FFNWB_ERR_PARAM_INVALID
    with pytest.raises(F.FfnwbError):
        F.moe_layer_plan(_layer(hidden=24))


@pytest.mark.parametrize("T,tokens", [(1, 16), (16, 16), (17, 64), (64, 64)])
@pytest.mark.parametrize("H,waves", [(16, 1), (384, 1), (400, 4), (1920, 4), (1936, 8), (7168, 8)])
def test_layer_first_launch(T, tokens, H, waves):
    p = _layer_plan(T, 2, 4, H, 32)
    assert (p["up_tokens"], p["up_waves"], p["lane_routing"]) == (tokens, waves, int(2 * T <= 64))


def test_layer_first_launch_with_many_tiles():
    # experts x inter / 16 from 1024 on: four waves to a tile whatever H
    assert _layer_plan(1, 8, 256, 7168, 2032)["up_waves"] == 8
    assert _layer_plan(1, 8, 256, 7168, 2048)["up_waves"] == 4


def test_layer_second_launch():
    # the sizes that the rule's comment names, and its limits
    assert _layer_plan(5, 8, 23, 576, 1024, bf16=True)["down_parts"] == 12
    assert _layer_plan(1, 6, 16, 2944, 496)["down_parts"] == 1
    assert _layer_plan(64, 8, 64, 4080, 1024)["down_parts"] == 2     # 255 column tiles
    assert _layer_plan(64, 8, 64, 4096, 1024)["down_parts"] == 1     # 256
    assert _layer_plan(64, 8, 64, 64, 2048)["down_parts"] == 32
