"""Host-only checks of the INT8 products' plan: the kernels that the sizes of the GPU tests and those named
beside the rules take, and what a workspace holds."""

import pytest

import unpermute_ffnwb_batching_amd as F
from test_gpu_int8_forms import BF16, FORMS, FP16, FP32, I8, check_form
from test_int8_checks import _matmul, _ws

CODE = {BF16: F.FFNWB_DT_BF16, FP16: F.FFNWB_DT_FP16, FP32: F.FFNWB_DT_FP32, I8: F.FFNWB_DT_INT8}


def _plan(size, dtype=BF16, epilogue="none"):
    rows, k, n, groups = size
    d = _matmul(num_rows=rows, in_features=k, out_features=n, out_dtype=CODE[dtype], epilogue=int(epilogue == "swiglu"),
                num_experts=4 if groups else 1, num_groups=4 if groups == 3 else groups)
    if not groups:
        d.group_list = None
    return F.moe_grouped_matmul_int8_plan(d)


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", FORMS, ids=str)
def test_the_gpu_tests_reach_their_forms(size, dtype, epilogue, kernel, how):
    check_form(_plan(size, dtype, epilogue), size, epilogue, kernel, how)


def test_every_kernel_is_among_the_forms():
    kinds = {(d, e, k) for _, d, e, k, h in FORMS}
    tiles = ("tiles32", "tiles64", "tiles128", "tiles256")
    plain = ("direct16x16", "direct32x16", "direct32x32", "direct64x32", "direct64x64") + tiles
    swiglu = ("direct16x16", "direct32x16", "direct64x16", "direct64x32") + tiles
    assert kinds >= {(d, "none", k) for d in (BF16, FP16, FP32) for k in plain}
    assert kinds >= {(d, "swiglu", k) for d in (BF16, FP16, FP32, I8) for k in swiglu}
    assert {f"waves {w}" for w in (1, 2, 4, 8, 16)} <= {h for _, d, e, k, h in FORMS}


def test_sizes_named_beside_the_rule():
    assert not _plan((1, 7168, 4096, 0))["lds_tiles"]
    assert not _plan((64, 7168, 4096, 0))["lds_tiles"]
    assert _plan((8191, 5120, 7168, 0)) == dict(lds_tiles=1, tile_rows=256, tile_columns=256, waves=0, listed=0)


def test_workspaces():
    # FP32 rows and a float for each 16 columns; nothing for a plain call
    d = _matmul(num_rows=8, in_features=256, out_features=96, epilogue=1, out_dtype=F.FFNWB_DT_INT8)
    assert _ws("moe_grouped_matmul_int8", d) == (0, 8 * 48 * 4 + 256)
    assert _ws("moe_grouped_matmul_int8", _matmul()) == (0, 0)
