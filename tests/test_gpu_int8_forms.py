"""Every kernel of the INT8 products, whole: each size asserts the kernel that it takes, so that the
tests keep reaching all of them when the rule that chooses changes.

Every element of every row is compared with the definition in 64 bits.  K ends inside a block of 128
and widths inside a tile; rows of no expert lie between the groups, and the last expert has no rows."""

import numpy as np
import pytest
import torch

from _int8 import matmul_inputs
from test_gpu_int8_products import NAMES, check

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8

# (rows, K, N, groups), type of the results, epilogue, kernel and its tile, and how: the "waves" that split K; row
# tiles "listed" by a launch of their own; of 128 and 256 rows, whether the last round of tiles is "halved"
FORMS = [
    ((20, 48, 48, 0), BF16, "none", "direct16x16", ""),
    ((8037, 48, 65, 3), BF16, "none", "direct32x16", ""),
    ((243, 48, 2820, 0), BF16, "none", "direct32x32", ""),
    ((8639, 48, 279, 3), BF16, "none", "direct64x32", ""),
    ((8874, 320, 303, 3), BF16, "none", "direct64x64", ""),
    ((229, 48, 3508, 3), BF16, "none", "tiles32", ""),
    ((8754, 48, 141, 3), BF16, "none", "tiles64", ""),
    ((2393, 432, 2932, 3), BF16, "none", "tiles128", "halved"),
    ((8256, 400, 411, 0), BF16, "none", "tiles128", "whole"),
    ((4739, 80, 2845, 3), BF16, "none", "tiles256", "halved"),
    ((8036, 48, 906, 3), BF16, "none", "tiles256", "whole"),
    ((22, 48, 43, 300), BF16, "none", "direct16x16", "listed"),
    ((6940, 160, 70, 300), BF16, "none", "direct32x16", "listed"),
    ((73, 144, 1666, 300), BF16, "none", "direct32x32", "listed"),
    ((37, 1440, 3456, 300), BF16, "none", "direct64x64", "listed"),
    ((43, 48, 2245, 300), BF16, "none", "tiles32", "listed"),
    ((66, 48, 3020, 300), BF16, "none", "tiles64", "listed"),
    ((101, 1312, 969, 300), BF16, "none", "tiles128", "listed"),
    ((20, 48, 48, 0), BF16, "none", "direct16x16", "waves 1"),
    ((20, 144, 47, 0), BF16, "none", "direct16x16", "waves 2"),
    ((21, 400, 44, 0), BF16, "none", "direct16x16", "waves 4"),
    ((20, 1744, 41, 3), BF16, "none", "direct16x16", "waves 8"),
    ((21, 7888, 42, 0), BF16, "none", "direct16x16", "waves 16"),
    ((8037, 48, 65, 3), BF16, "none", "direct32x16", "waves 1"),
    ((54, 464, 3698, 0), BF16, "none", "direct32x16", "waves 2"),
    ((1959, 1008, 49, 0), BF16, "none", "direct32x16", "waves 4"),
    ((21, 2608, 1147, 3), BF16, "none", "direct32x16", "waves 8"),
    ((243, 48, 2820, 0), BF16, "none", "direct32x32", "waves 1"),
    ((58, 416, 3756, 3), BF16, "none", "direct32x32", "waves 2"),
    ((24, 1984, 2187, 3), BF16, "none", "direct32x32", "waves 4"),
    ((22, 4816, 1851, 3), BF16, "none", "direct32x32", "waves 8"),
    ((8639, 48, 279, 3), BF16, "none", "direct64x32", "waves 1"),
    ((3580, 928, 233, 3), BF16, "none", "direct64x32", "waves 2"),
    ((7547, 2032, 42, 3), BF16, "none", "direct64x32", "waves 4"),
    ((8874, 320, 303, 3), BF16, "none", "direct64x64", "waves 1"),
    ((8719, 1216, 161, 3), BF16, "none", "direct64x64", "waves 2"),
    ((119, 2496, 3573, 3), BF16, "none", "direct64x64", "waves 4"),
    ((20, 48, 64, 3), BF16, "swiglu", "direct16x16", ""),
    ((492, 48, 1248, 3), BF16, "swiglu", "direct32x16", ""),
    ((8437, 48, 288, 3), BF16, "swiglu", "direct64x16", ""),
    ((8472, 304, 320, 3), BF16, "swiglu", "direct64x32", ""),
    ((252, 48, 3616, 3), BF16, "swiglu", "tiles32", ""),
    ((4517, 48, 288, 3), BF16, "swiglu", "tiles64", ""),
    ((4317, 432, 1664, 3), BF16, "swiglu", "tiles128", "halved"),
    ((5752, 400, 576, 3), BF16, "swiglu", "tiles128", "whole"),
    ((8709, 48, 1600, 3), BF16, "swiglu", "tiles256", "halved"),
    ((8664, 48, 832, 3), BF16, "swiglu", "tiles256", "whole"),
    ((20, 48, 64, 300), BF16, "swiglu", "direct16x16", "listed"),
    ((129, 880, 96, 300), BF16, "swiglu", "direct32x16", "listed"),
    ((4135, 3408, 64, 300), BF16, "swiglu", "direct64x32", "listed"),
    ((131, 64, 736, 300), BF16, "swiglu", "tiles32", "listed"),
    ((57, 64, 3392, 300), BF16, "swiglu", "tiles64", "listed"),
    ((4881, 928, 224, 300), BF16, "swiglu", "tiles128", "listed"),
    ((20, 48, 64, 3), BF16, "swiglu", "direct16x16", "waves 1"),
    ((20, 144, 64, 0), BF16, "swiglu", "direct16x16", "waves 2"),
    ((20, 800, 64, 3), BF16, "swiglu", "direct16x16", "waves 4"),
    ((20, 2592, 64, 3), BF16, "swiglu", "direct16x16", "waves 8"),
    ((492, 48, 1248, 3), BF16, "swiglu", "direct32x16", "waves 1"),
    ((308, 400, 1152, 3), BF16, "swiglu", "direct32x16", "waves 2"),
    ((21, 832, 2208, 3), BF16, "swiglu", "direct32x16", "waves 4"),
    ((21, 4016, 2176, 3), BF16, "swiglu", "direct32x16", "waves 8"),
    ((8437, 48, 288, 3), BF16, "swiglu", "direct64x16", "waves 1"),
    ((447, 736, 2336, 0), BF16, "swiglu", "direct64x16", "waves 2"),
    ((1004, 1424, 512, 0), BF16, "swiglu", "direct64x16", "waves 4"),
    ((8472, 304, 320, 3), BF16, "swiglu", "direct64x32", "waves 1"),
    ((4366, 1200, 384, 3), BF16, "swiglu", "direct64x32", "waves 2"),
    ((160, 2368, 3168, 3), BF16, "swiglu", "direct64x32", "waves 4"),
    ((20, 48, 41, 0), FP16, "none", "direct16x16", ""),
    ((367, 48, 1453, 3), FP16, "none", "direct32x16", ""),
    ((681, 48, 994, 3), FP16, "none", "direct32x32", ""),
    ((8356, 48, 271, 3), FP16, "none", "direct64x32", ""),
    ((8612, 368, 289, 3), FP16, "none", "direct64x64", ""),
    ((308, 48, 2835, 3), FP16, "none", "tiles32", ""),
    ((8773, 48, 130, 0), FP16, "none", "tiles64", ""),
    ((2846, 448, 2587, 0), FP16, "none", "tiles128", "halved"),
    ((5493, 448, 551, 3), FP16, "none", "tiles128", "whole"),
    ((5310, 48, 2585, 3), FP16, "none", "tiles256", "halved"),
    ((4694, 48, 1549, 3), FP16, "none", "tiles256", "whole"),
    ((23, 48, 40, 300), FP16, "none", "direct16x16", "listed"),
    ((7529, 144, 71, 300), FP16, "none", "direct32x16", "listed"),
    ((43, 144, 2900, 300), FP16, "none", "direct32x32", "listed"),
    ((36, 4064, 1402, 300), FP16, "none", "direct64x64", "listed"),
    ((63, 48, 1532, 300), FP16, "none", "tiles32", "listed"),
    ((265, 64, 578, 300), FP16, "none", "tiles64", "listed"),
    ((4630, 832, 200, 300), FP16, "none", "tiles128", "listed"),
    ((20, 48, 64, 0), FP16, "swiglu", "direct16x16", ""),
    ((220, 48, 2560, 3), FP16, "swiglu", "direct32x16", ""),
    ((8792, 48, 288, 0), FP16, "swiglu", "direct64x16", ""),
    ((8801, 352, 320, 0), FP16, "swiglu", "direct64x32", ""),
    ((241, 48, 3936, 3), FP16, "swiglu", "tiles32", ""),
    ((8653, 48, 160, 3), FP16, "swiglu", "tiles64", ""),
    ((2872, 432, 2368, 3), FP16, "swiglu", "tiles128", "halved"),
    ((5928, 448, 544, 0), FP16, "swiglu", "tiles128", "whole"),
    ((8698, 48, 1568, 3), FP16, "swiglu", "tiles256", "halved"),
    ((8351, 48, 800, 3), FP16, "swiglu", "tiles256", "whole"),
    ((20, 48, 64, 300), FP16, "swiglu", "direct16x16", "listed"),
    ((126, 816, 96, 300), FP16, "swiglu", "direct32x16", "listed"),
    ((4131, 1712, 128, 300), FP16, "swiglu", "direct64x32", "listed"),
    ((49, 64, 1984, 300), FP16, "swiglu", "tiles32", "listed"),
    ((199, 48, 864, 300), FP16, "swiglu", "tiles64", "listed"),
    ((4789, 944, 224, 300), FP16, "swiglu", "tiles128", "listed"),
    ((20, 48, 46, 0), FP32, "none", "direct16x16", ""),
    ((8056, 48, 65, 3), FP32, "none", "direct32x16", ""),
    ((4474, 48, 149, 3), FP32, "none", "direct32x32", ""),
    ((8983, 48, 258, 0), FP32, "none", "direct64x32", ""),
    ((8950, 336, 312, 3), FP32, "none", "direct64x64", ""),
    ((353, 48, 2451, 3), FP32, "none", "tiles32", ""),
    ((8390, 48, 130, 3), FP32, "none", "tiles64", ""),
    ((6207, 400, 1237, 3), FP32, "none", "tiles128", "halved"),
    ((6143, 432, 519, 3), FP32, "none", "tiles128", "whole"),
    ((5271, 48, 2606, 3), FP32, "none", "tiles256", "halved"),
    ((6730, 48, 1034, 3), FP32, "none", "tiles256", "whole"),
    ((20, 48, 44, 300), FP32, "none", "direct16x16", "listed"),
    ((8883, 48, 104, 300), FP32, "none", "direct32x16", "listed"),
    ((43, 144, 2841, 300), FP32, "none", "direct32x32", "listed"),
    ((177, 1840, 569, 300), FP32, "none", "direct64x64", "listed"),
    ((30, 48, 3251, 300), FP32, "none", "tiles32", "listed"),
    ((61, 48, 3117, 300), FP32, "none", "tiles64", "listed"),
    ((4710, 816, 199, 300), FP32, "none", "tiles128", "listed"),
    ((21, 48, 64, 0), FP32, "swiglu", "direct16x16", ""),
    ((186, 48, 2912, 3), FP32, "swiglu", "direct32x16", ""),
    ((8909, 48, 288, 0), FP32, "swiglu", "direct64x16", ""),
    ((8156, 288, 320, 3), FP32, "swiglu", "direct64x32", ""),
    ((393, 48, 2464, 3), FP32, "swiglu", "tiles32", ""),
    ((8317, 48, 160, 3), FP32, "swiglu", "tiles64", ""),
    ((7820, 480, 832, 3), FP32, "swiglu", "tiles128", "halved"),
    ((5669, 416, 544, 3), FP32, "swiglu", "tiles128", "whole"),
    ((3446, 48, 3936, 3), FP32, "swiglu", "tiles256", "halved"),
    ((8530, 48, 800, 0), FP32, "swiglu", "tiles256", "whole"),
    ((21, 48, 64, 300), FP32, "swiglu", "direct16x16", "listed"),
    ((129, 784, 96, 300), FP32, "swiglu", "direct32x16", "listed"),
    ((4288, 2976, 64, 300), FP32, "swiglu", "direct64x32", "listed"),
    ((188, 64, 512, 300), FP32, "swiglu", "tiles32", "listed"),
    ((115, 48, 1600, 300), FP32, "swiglu", "tiles64", "listed"),
    ((6119, 816, 192, 300), FP32, "swiglu", "tiles128", "listed"),
    ((20, 48, 64, 0), I8, "swiglu", "direct16x16", ""),
    ((214, 48, 2624, 3), I8, "swiglu", "direct32x16", ""),
    ((8187, 48, 288, 3), I8, "swiglu", "direct64x16", ""),
    ((8846, 288, 320, 3), I8, "swiglu", "direct64x32", ""),
    ((271, 48, 3456, 3), I8, "swiglu", "tiles32", ""),
    ((4503, 48, 288, 3), I8, "swiglu", "tiles64", ""),
    ((4301, 400, 1664, 3), I8, "swiglu", "tiles128", "halved"),
    ((5487, 400, 608, 3), I8, "swiglu", "tiles128", "whole"),
    ((5838, 48, 2400, 3), I8, "swiglu", "tiles256", "halved"),
    ((8232, 48, 800, 3), I8, "swiglu", "tiles256", "whole"),
    ((20, 48, 64, 300), I8, "swiglu", "direct16x16", "listed"),
    ((32, 816, 384, 300), I8, "swiglu", "direct32x16", "listed"),
    ((2896, 2752, 128, 300), I8, "swiglu", "direct64x32", "listed"),
    ((190, 48, 512, 300), I8, "swiglu", "tiles32", "listed"),
    ((88, 48, 2208, 300), I8, "swiglu", "tiles64", "listed"),
    ((4724, 944, 224, 300), I8, "swiglu", "tiles128", "listed"),
    ((20, 48, 64, 0), I8, "swiglu", "direct16x16", "waves 1"),
    ((20, 144, 64, 0), I8, "swiglu", "direct16x16", "waves 2"),
    ((21, 832, 64, 3), I8, "swiglu", "direct16x16", "waves 4"),
    ((21, 2656, 64, 3), I8, "swiglu", "direct16x16", "waves 8"),
    ((214, 48, 2624, 3), I8, "swiglu", "direct32x16", "waves 1"),
    ((102, 400, 2816, 3), I8, "swiglu", "direct32x16", "waves 2"),
    ((21, 800, 2368, 3), I8, "swiglu", "direct32x16", "waves 4"),
    ((20, 3904, 2272, 3), I8, "swiglu", "direct32x16", "waves 8"),
    ((8187, 48, 288, 3), I8, "swiglu", "direct64x16", "waves 1"),
    ((2480, 720, 416, 0), I8, "swiglu", "direct64x16", "waves 2"),
    ((97, 2224, 3904, 0), I8, "swiglu", "direct64x16", "waves 4"),
    ((8846, 288, 320, 3), I8, "swiglu", "direct64x32", "waves 1"),
    ((2671, 1200, 576, 3), I8, "swiglu", "direct64x32", "waves 2"),
    ((126, 2416, 3648, 3), I8, "swiglu", "direct64x32", "waves 4"),
]


def _groups(rows, groups):
    """{key, rows} pairs: ragged groups and a tiny one, rows of no expert; or many groups."""
    if groups == 0:
        return None
    if groups == 3:
        return [(2, rows * 9 // 20), (0, 5), (1, rows - rows * 9 // 20 - 9), (9, 4)]
    return [(i % 3, rows // groups + (i < rows % groups)) for i in range(groups)]


def _last_round_halved(plan, groups, rows, n, epilogue):
    """Whether the last tiles of each of the 8 XCDs, 32 at a time, are at most half a round."""
    mt = sum(-(-m // plan["tile_rows"]) for key, m in groups if key < 3) if groups else -(-rows // plan["tile_rows"])
    nt = -(-(n // 2 if epilogue == "swiglu" else n) // plan["tile_columns"])
    return 2 * (-(-mt * nt // 8) % 32) <= 32


def check_form(plan, size, epilogue, kernel, how):
    rows, _, n, groups = size
    assert (f"tiles{plan['tile_rows']}" if plan["lds_tiles"] else f"direct{plan['tile_rows']}x{plan['tile_columns']}") == kernel
    assert bool(plan["listed"]) == (how == "listed") and (plan["waves"] == 0) == bool(plan["lds_tiles"])
    if how.startswith("waves"):
        assert how == f"waves {plan['waves']}"
    if plan["tile_rows"] >= 128 and plan["lds_tiles"] and how != "listed":
        assert _last_round_halved(plan, _groups(rows, groups), rows, n, epilogue) == (how == "halved")


@pytest.mark.parametrize("size,dtype,epilogue,kernel,how", FORMS,
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else NAMES.get(v, v))
def test_form(size, dtype, epilogue, kernel, how):
    rows, k, n, groups = size
    c = matmul_inputs(rows + k + n, rows, k, n, 4 if groups else 1)
    plan = check(c, _groups(rows, groups), epilogue, dtype, pad=0 if dtype == I8 else 3, what=kernel + " " + how)
    check_form(plan, size, epilogue, kernel, how)


def test_a_row_of_each_kind_of_kernel_is_the_same():
    # the same rows in calls of different sizes: whole-number sums, so the same bits whatever the kernel
    import unpermute_ffnwb_batching_amd as F
    from _expert import dev
    c = matmul_inputs(77, 6000, 1040, 1304)
    args = [dev(c[k]) for k in ("x", "xs", "w", "ws")]
    kinds = set()
    for dtype in (FP32, BF16):
        want = None
        for rows in (1, 20, 90, 300, 1100, 6000):
            call = F.GroupedMatmulInt8Call(args[0][:rows], args[1][:rows], args[2], args[3], out_dtype=dtype)
            kinds.add(tuple(F.moe_grouped_matmul_int8_plan(call.desc).values()))
            y = call.run()["y"][0]
            torch.cuda.synchronize()
            want = y if want is None else want
            assert torch.equal(y.view(torch.uint8), want.view(torch.uint8)), rows
    assert len(kinds) >= 4
