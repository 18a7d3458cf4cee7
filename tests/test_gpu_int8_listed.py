"""Every kernel of the INT8 products on row tiles that a launch of its own lists, whole: 300 groups of very
different size, some empty, some of no expert, one with two fifths of the rows, and rows behind the last.  Tiles
of 128 and 256 rows with their last round halved and whole; the kernel form that a prefill of 128 experts and
131072 rows takes is among them (tiles of 256 rows, listed)."""

import numpy as np
import pytest
import torch

from _int8 import matmul_inputs
from test_gpu_int8_products import NAMES, check

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8

GROUPS, EXPERTS = 300, 4

# (rows, K, N), kernel and its tile, last round of tiles of 128 and 256 rows
PLAIN = [((259, 144, 3), "direct16x16", ""), ((6642, 144, 74), "direct32x16", ""), ((311, 144, 394), "direct32x32", ""),
         ((14993, 544, 81), "direct64x32", ""), ((26000, 144, 97), "direct64x64", ""), ((338, 144, 246), "tiles32", ""),
         ((267, 144, 553), "tiles64", ""), ((28168, 416, 136), "tiles128", "halved"), ((28168, 416, 136), "tiles128", "whole"),
         ((58246, 144, 119), "tiles256", "halved"), ((58246, 144, 119), "tiles256", "whole"), ((137142, 16, 69), "tiles256", "whole")]
SWIGLU = [((260, 144, 32), "direct16x16", ""), ((2980, 144, 288), "direct32x16", ""), ((14998, 608, 96), "direct64x16", ""),
          ((25691, 144, 128), "direct64x32", ""), ((261, 192, 608), "tiles32", ""), ((263, 160, 608), "tiles64", ""),
          ((20995, 416, 352), "tiles128", "halved"), ((20995, 416, 352), "tiles128", "whole"), ((56932, 144, 128), "tiles256", "halved"),
          ((56932, 144, 128), "tiles256", "whole"), ((123229, 16, 96), "tiles256", "whole")]
LISTED = [(s, d, "none", k, h) for s, k, h in PLAIN for d in (BF16, FP16, FP32)] + \
         [(s, d, "swiglu", k, h) for s, k, h in SWIGLU for d in (BF16, FP16, FP32, I8)]


def _layout(seed, rows):
    rng = np.random.default_rng(seed)
    share = rng.exponential(size=GROUPS) ** 3 * (rng.random(GROUPS) < 0.8)
    share[rng.integers(GROUPS)] = share.sum() * 2 / 3
    counts = np.floor((rows - 7) * share / share.sum()).astype(int)
    return [(int(i % (EXPERTS + 1)), int(n)) for i, n in enumerate(counts)]  # the last key is no expert's


def _last_round(plan, groups, n, epilogue):
    """The tiles of the last round of each of the 8 XCDs, 32 at a time."""
    mt = sum(-(-m // plan["tile_rows"]) for key, m in groups if key < EXPERTS)
    return -(-mt * -(-(n // 2 if epilogue == "swiglu" else n) // plan["tile_columns"]) // 8) % 32


def layout(plan, size, epilogue, how):
    """The first layout of a size whose last round is as asked for."""
    for seed in range(200):
        groups = _layout(seed, size[0])
        if how == "" or (0 < _last_round(plan, groups, size[2], epilogue) <= 16) == (how == "halved"):
            return groups
    raise AssertionError("no such layout")


def check_listed(plan, kernel):
    assert plan["listed"]
    assert (f"tiles{plan['tile_rows']}" if plan["lds_tiles"] else f"direct{plan['tile_rows']}x{plan['tile_columns']}") == kernel


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", LISTED,
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else NAMES.get(v, v))
def test_listed(size, dtype, epilogue, kernel, how):
    from test_int8_listed_plans import plan_of
    rows, k, n = size
    groups = layout(plan_of(size, dtype, epilogue), size, epilogue, how)
    plan = check(matmul_inputs(rows + k + n, rows, k, n, EXPERTS), groups, epilogue, dtype, pad=0 if dtype == I8 else 3, what=f"{kernel} listed {how}")
    check_listed(plan, kernel)
