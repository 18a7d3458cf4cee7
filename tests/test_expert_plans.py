"""Host-only checks of the plan queries: which kernels the sizes named beside the rules, and those of
the GPU tests, take."""

import ctypes

import pytest

import test_gpu_layer_forms
import test_gpu_product_forms
import unpermute_ffnwb_batching_amd as F
from test_expert_ffn_checks import _layer, _matmul
from test_gpu_product_forms import BF16, EXACT_FORMS, FORMS, FP8, FP16, FP32


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


@pytest.mark.parametrize("size,form", test_gpu_layer_forms.FORMS, ids=str)
def test_the_layers_gpu_tests_reach_their_forms(size, form):
    p = _layer_plan(*size)
    assert (p["up_tokens"], p["up_waves"], p["lane_routing"]) == form


def test_product_plan_refuses_what_the_call_refuses():
    info = F.GroupedMatmulFp8PlanInfo()
    plan = F.lib().moe_grouped_matmul_fp8_plan
    assert plan(None, ctypes.byref(info)) == F.FFNWB_ERR_PARAM_NULLPTR
    assert plan(ctypes.byref(_matmul()), None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert plan(ctypes.byref(_matmul(in_features=24)), ctypes.byref(info)) == F.FFNWB_ERR_PARAM_INVALID
    with pytest.raises(F.FfnwbError):
        F.moe_grouped_matmul_fp8_plan(_matmul(num_experts=0))


def _product_plan(size, dtype, epilogue, exact=False, **over):
    rows, k, n, experts = size
    groups = test_gpu_product_forms._groups(rows, experts)
    over.update(dict(group_list=None, num_groups=0, num_experts=1) if groups is None else
                dict(num_groups=len(groups), num_experts=4))
    return F.moe_grouped_matmul_fp8_plan(_matmul(
        num_rows=rows, in_features=k, out_features=n, epilogue=int(epilogue == "swiglu") + (F.FFNWB_EPI_EXACT if exact else 0), x_row_stride=k + 48,
        out_dtype={FP16: 0, BF16: 1, FP32: 3, FP8: 6}[dtype], **over))


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", FORMS, ids=test_gpu_product_forms._ids)
def test_the_products_gpu_tests_reach_their_kernels(size, dtype, epilogue, kernel, how):
    test_gpu_product_forms.check_form(_product_plan(size, dtype, epilogue), size, dtype, epilogue, kernel, how)


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", EXACT_FORMS, ids=test_gpu_product_forms._ids)
def test_the_exact_products_gpu_tests_reach_their_kernels(size, dtype, epilogue, kernel, how):
    plan = _product_plan(size, dtype, epilogue, exact=True)
    test_gpu_product_forms.check_form(plan, size, dtype, epilogue, kernel, how, exact=True)


def test_exact_is_a_flag_of_the_epilogue():
    for epilogue, ok in ((0, True), (1, True), (2, False), (512, False), (-1, False), (-256, False)):
        d = _matmul(epilogue=epilogue | F.FFNWB_EPI_EXACT)
        st = F.lib().moe_grouped_matmul_fp8_plan(ctypes.byref(d), ctypes.byref(F.GroupedMatmulFp8PlanInfo()))
        assert st == (F.FFNWB_OK if ok else F.FFNWB_ERR_PARAM_INVALID), epilogue
    # e4m3 results still need SwiGLU
    d = _matmul(epilogue=F.FFNWB_EPI_EXACT, out_dtype=6)
    assert F.lib().moe_grouped_matmul_fp8_plan(ctypes.byref(d), ctypes.byref(F.GroupedMatmulFp8PlanInfo())) == F.FFNWB_ERR_PARAM_INVALID


def test_every_kernel_of_the_products_has_a_size():
    # direct: 3 heights, results of 3 types, plain and SwiGLU, and e4m3 ones; tiles: 16-bit results of 4 heights, plain
    # and SwiGLU, FP32 ones of 3, e4m3 ones of 3; split: 3 heights of all of them
    have = {(kernel, dtype, epilogue, "split" in how) for _, dtype, epilogue, kernel, how in FORMS}
    for epilogue in ("none", "swiglu"):
        for dtype in (BF16, FP16, FP32) + ((FP8,) if epilogue == "swiglu" else ()):
            for rows in (16, 32, 64):
                assert (f"direct{rows}", dtype, epilogue, False) in have
            for rows in (32, 64, 128) + ((256,) if dtype in (BF16, FP16) else ()):
                assert (f"tiles{rows}", dtype, epilogue, False) in have
                if dtype in (BF16, FP16) and rows < 256:
                    assert any(f[1:4] == (dtype, epilogue, f"tiles{rows}") and "split" not in f[4] for f in EXACT_FORMS)
                if rows < 256:
                    assert (f"tiles{rows}", dtype, epilogue, True) in have
