"""Host-only checks of which kernels the INT8 products take for row tiles listed by a launch of their own, and at the
ends of what 32-bit offsets inside a tile can reach."""

import pytest

import unpermute_ffnwb_batching_amd as F
from test_gpu_int8_listed import BF16, FP16, FP32, GROUPS, I8, LISTED, PLAIN, SWIGLU, check_listed, layout
from test_int8_checks import _matmul

CODE = {BF16: F.FFNWB_DT_BF16, FP16: F.FFNWB_DT_FP16, FP32: F.FFNWB_DT_FP32, I8: F.FFNWB_DT_INT8}


def plan_of(size, dtype, epilogue, groups=GROUPS, experts=4, **kw):
    rows, k, n = size
    d = _matmul(num_rows=rows, in_features=k, out_features=n, out_dtype=CODE[dtype], epilogue=int(epilogue == "swiglu"),
                num_experts=experts if groups else 1, num_groups=groups, **kw)
    if not groups:
        d.group_list = None
    return F.moe_grouped_matmul_int8_plan(d)


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", LISTED, ids=str)
def test_the_gpu_tests_reach_their_forms(size, dtype, epilogue, kernel, how):
    plan = plan_of(size, dtype, epilogue)
    check_listed(plan, kernel)
    assert sum(m for _, m in layout(plan, size, epilogue, how)) < size[0]


def test_every_kernel_is_listed():
    tiles = {("tiles32", ""), ("tiles64", ""), ("tiles128", "halved"), ("tiles128", "whole"), ("tiles256", "halved"), ("tiles256", "whole")}
    assert {(k, h) for _, k, h in PLAIN} == tiles | {(f"direct{s}", "") for s in ("16x16", "32x16", "32x32", "64x32", "64x64")}
    assert {(k, h) for _, k, h in SWIGLU} == tiles | {(f"direct{s}", "") for s in ("16x16", "32x16", "64x16", "64x32")}


@pytest.mark.parametrize("size,dtype,epilogue", [((131072, 4096, 2048), BF16, "swiglu"), ((131072, 4096, 2048), I8, "swiglu"),
                                                 ((131072, 1024, 4096), BF16, "none")], ids=str)
def test_both_products_of_a_prefill_take_a_listed_form(size, dtype, epilogue):
    plan = plan_of(size, dtype, epilogue, groups=128, experts=128)
    check_listed(plan, "tiles256")


def test_strides_past_the_offsets_of_a_tile_take_the_direct_kernel():
    # 256 rows of x lie within 32 bits up to 2^22 bytes a row
    for size in ((8754, 256, 512), (654, 80, 11910)):
        assert all(plan_of(size, FP32, "none", 0, x_row_stride=s)["lds_tiles"] for s in (0, 1 << 22))
        assert not any(plan_of(size, FP32, "none", 0, x_row_stride=s)["lds_tiles"] for s in ((1 << 22) + 16, 1 << 32))


def test_up_rows_past_the_offsets_of_a_tile_take_the_direct_kernel():
    # (F + 128) K below 2^32: F = 32640 is the last for K = 131040
    for dtype in (BF16, FP16, FP32, I8):
        assert plan_of((300, 131040, 2 * 32640), dtype, "swiglu", 0)["lds_tiles"]
        assert not plan_of((300, 131040, 2 * 32656), dtype, "swiglu", 0)["lds_tiles"]
    assert plan_of((300, 131040, 2 * 32656), BF16, "none", 0)["lds_tiles"]   # one block of weight rows: no such bound
