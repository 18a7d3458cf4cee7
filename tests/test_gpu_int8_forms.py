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

# (rows, K, N, groups), type of the results, epilogue, kernel and tile rows, and how: "split" over K; row
# tiles "listed" by a launch of their own; of 128 and 256 rows, whether the last round of tiles is "halved"
FORMS = [
    ((20, 304, 148, 0), BF16, "none", "direct16", ""),
    ((20, 1136, 2033, 0), BF16, "none", "direct32", ""),
    ((623, 400, 950, 3), BF16, "none", "direct64", ""),
    ((131, 416, 3209, 3), BF16, "none", "tiles32", ""),
    ((4327, 272, 276, 0), BF16, "none", "tiles64", ""),
    ((1878, 272, 1839, 3), BF16, "none", "tiles128", "halved"),
    ((8454, 288, 283, 3), BF16, "none", "tiles128", "whole"),
    ((6340, 944, 2543, 0), BF16, "none", "tiles256", "halved"),
    ((8873, 912, 841, 3), BF16, "none", "tiles256", "whole"),
    ((20, 6768, 3134, 3), BF16, "none", "tiles32", "split"),
    ((21, 7824, 3383, 3), BF16, "none", "tiles64", "split"),
    ((88, 3728, 2032, 3), BF16, "none", "tiles128", "split halved"),
    ((48, 5008, 2388, 3), BF16, "none", "tiles128", "split whole"),
    ((22, 352, 145, 300), BF16, "none", "direct16", "listed"),
    ((218, 400, 354, 300), BF16, "none", "direct32", "listed"),
    ((52, 272, 930, 300), BF16, "none", "tiles32", "listed"),
    ((117, 272, 685, 300), BF16, "none", "tiles64", "listed"),
    ((40, 368, 2080, 300), BF16, "none", "tiles128", "listed"),
    ((22, 288, 288, 0), BF16, "swiglu", "direct16", ""),
    ((23, 992, 3360, 3), BF16, "swiglu", "direct32", ""),
    ((276, 400, 2208, 3), BF16, "swiglu", "direct64", ""),
    ((53, 1104, 3392, 3), BF16, "swiglu", "tiles32", ""),
    ((2819, 272, 576, 3), BF16, "swiglu", "tiles64", ""),
    ((6310, 272, 1152, 0), BF16, "swiglu", "tiles128", "halved"),
    ((8870, 320, 288, 3), BF16, "swiglu", "tiles128", "whole"),
    ((6957, 976, 2176, 0), BF16, "swiglu", "tiles256", "halved"),
    ((8472, 912, 800, 3), BF16, "swiglu", "tiles256", "whole"),
    ((54, 2096, 3424, 3), BF16, "swiglu", "tiles32", "split"),
    ((65, 2352, 3296, 3), BF16, "swiglu", "tiles64", "split"),
    ((94, 4896, 2400, 3), BF16, "swiglu", "tiles128", "split halved"),
    ((64, 3648, 3072, 3), BF16, "swiglu", "tiles128", "split whole"),
    ((20, 272, 352, 300), BF16, "swiglu", "direct16", "listed"),
    ((42, 912, 640, 300), BF16, "swiglu", "direct32", "listed"),
    ((39, 272, 1760, 300), BF16, "swiglu", "tiles32", "listed"),
    ((49, 272, 2272, 300), BF16, "swiglu", "tiles64", "listed"),
    ((179, 624, 384, 300), BF16, "swiglu", "tiles128", "listed"),
    ((20, 320, 132, 0), FP16, "none", "direct16", ""),
    ((20, 1216, 2154, 0), FP16, "none", "direct32", ""),
    ((396, 416, 1356, 3), FP16, "none", "direct64", ""),
    ((164, 272, 3532, 3), FP16, "none", "tiles32", ""),
    ((8112, 288, 136, 3), FP16, "none", "tiles64", ""),
    ((6078, 272, 1083, 3), FP16, "none", "tiles128", "halved"),
    ((8096, 288, 269, 3), FP16, "none", "tiles128", "whole"),
    ((4405, 1056, 3565, 0), FP16, "none", "tiles256", "halved"),
    ((4003, 944, 1793, 3), FP16, "none", "tiles256", "whole"),
    ((57, 3264, 2705, 3), FP16, "none", "tiles32", "split"),
    ((27, 5952, 2837, 3), FP16, "none", "tiles64", "split"),
    ((120, 3168, 1964, 3), FP16, "none", "tiles128", "split halved"),
    ((56, 4208, 2515, 3), FP16, "none", "tiles128", "split whole"),
    ((23, 304, 131, 300), FP16, "none", "direct16", "listed"),
    ((186, 432, 283, 300), FP16, "none", "direct32", "listed"),
    ((328, 272, 145, 300), FP16, "none", "tiles32", "listed"),
    ((235, 272, 339, 300), FP16, "none", "tiles64", "listed"),
    ((60, 272, 1404, 300), FP16, "none", "tiles128", "listed"),
    ((21, 304, 288, 0), FP16, "swiglu", "direct16", ""),
    ((22, 1072, 3008, 0), FP16, "swiglu", "direct32", ""),
    ((187, 416, 2848, 3), FP16, "swiglu", "direct64", ""),
    ((76, 1056, 2720, 3), FP16, "swiglu", "tiles32", ""),
    ((5528, 288, 288, 0), FP16, "swiglu", "tiles64", ""),
    ((1643, 464, 2112, 3), FP16, "swiglu", "tiles128", "halved"),
    ((8397, 320, 288, 0), FP16, "swiglu", "tiles128", "whole"),
    ((5205, 928, 2688, 3), FP16, "swiglu", "tiles256", "halved"),
    ((8638, 912, 896, 3), FP16, "swiglu", "tiles256", "whole"),
    ((55, 2208, 3328, 3), FP16, "swiglu", "tiles32", "split"),
    ((68, 2384, 3424, 3), FP16, "swiglu", "tiles64", "split"),
    ((123, 4432, 2528, 3), FP16, "swiglu", "tiles128", "split halved"),
    ((64, 3088, 3488, 3), FP16, "swiglu", "tiles128", "split whole"),
    ((21, 304, 288, 300), FP16, "swiglu", "direct16", "listed"),
    ((24, 912, 1152, 300), FP16, "swiglu", "direct32", "listed"),
    ((71, 288, 1024, 300), FP16, "swiglu", "tiles32", "listed"),
    ((101, 272, 1120, 300), FP16, "swiglu", "tiles64", "listed"),
    ((180, 544, 320, 300), FP16, "swiglu", "tiles128", "listed"),
    ((20, 272, 148, 3), FP32, "none", "direct16", ""),
    ((22, 608, 3469, 0), FP32, "none", "direct32", ""),
    ((3697, 400, 162, 3), FP32, "none", "direct64", ""),
    ((137, 400, 2958, 3), FP32, "none", "tiles32", ""),
    ((8168, 288, 130, 3), FP32, "none", "tiles64", ""),
    ((8633, 304, 792, 3), FP32, "none", "tiles128", "halved"),
    ((8056, 272, 270, 3), FP32, "none", "tiles128", "whole"),
    ((8115, 928, 788, 3), FP32, "none", "tiles256", "whole"),
    ((68, 3104, 2139, 3), FP32, "none", "tiles32", "split"),
    ((22, 7248, 3325, 3), FP32, "none", "tiles64", "split"),
    ((121, 4304, 1574, 3), FP32, "none", "tiles128", "split halved"),
    ((47, 4752, 2430, 3), FP32, "none", "tiles128", "split whole"),
    ((20, 272, 139, 300), FP32, "none", "direct16", "listed"),
    ((198, 400, 272, 300), FP32, "none", "direct32", "listed"),
    ((62, 272, 771, 300), FP32, "none", "tiles32", "listed"),
    ((231, 288, 322, 300), FP32, "none", "tiles64", "listed"),
    ((45, 288, 1896, 300), FP32, "none", "tiles128", "listed"),
    ((21, 272, 288, 0), FP32, "swiglu", "direct16", ""),
    ((24, 1104, 3040, 0), FP32, "swiglu", "direct32", ""),
    ((260, 400, 2336, 3), FP32, "swiglu", "direct64", ""),
    ((67, 1072, 2976, 3), FP32, "swiglu", "tiles32", ""),
    ((5066, 272, 320, 3), FP32, "swiglu", "tiles64", ""),
    ((1872, 464, 1824, 3), FP32, "swiglu", "tiles128", "halved"),
    ((8228, 336, 288, 3), FP32, "swiglu", "tiles128", "whole"),
    ((5180, 912, 2592, 3), FP32, "swiglu", "tiles256", "halved"),
    ((8042, 1008, 800, 3), FP32, "swiglu", "tiles256", "whole"),
    ((76, 2208, 2880, 3), FP32, "swiglu", "tiles32", "split"),
    ((127, 2080, 2048, 3), FP32, "swiglu", "tiles64", "split"),
    ((96, 5568, 2272, 3), FP32, "swiglu", "tiles128", "split halved"),
    ((58, 3104, 3456, 3), FP32, "swiglu", "tiles128", "split whole"),
    ((21, 272, 352, 300), FP32, "swiglu", "direct16", "listed"),
    ((225, 400, 288, 300), FP32, "swiglu", "direct32", "listed"),
    ((49, 272, 1472, 300), FP32, "swiglu", "tiles32", "listed"),
    ((176, 400, 384, 300), FP32, "swiglu", "tiles64", "listed"),
    ((3252, 288, 416, 300), FP32, "swiglu", "tiles128", "listed"),
    ((21, 272, 288, 3), I8, "swiglu", "direct16", ""),
    ((20, 1104, 3296, 0), I8, "swiglu", "direct32", ""),
    ((218, 400, 2624, 3), I8, "swiglu", "direct64", ""),
    ((54, 1040, 3488, 3), I8, "swiglu", "tiles32", ""),
    ((4960, 272, 320, 0), I8, "swiglu", "tiles64", ""),
    ((1642, 320, 2080, 3), I8, "swiglu", "tiles128", "halved"),
    ((8345, 272, 288, 3), I8, "swiglu", "tiles128", "whole"),
    ((5162, 912, 2752, 3), I8, "swiglu", "tiles256", "halved"),
    ((8472, 944, 832, 3), I8, "swiglu", "tiles256", "whole"),
    ((54, 2256, 3424, 3), I8, "swiglu", "tiles32", "split"),
    ((92, 2144, 2528, 3), I8, "swiglu", "tiles64", "split"),
    ((94, 5088, 2400, 3), I8, "swiglu", "tiles128", "split halved"),
    ((58, 3168, 3424, 3), I8, "swiglu", "tiles128", "split whole"),
    ((20, 272, 288, 300), I8, "swiglu", "direct16", "listed"),
    ((96, 912, 288, 300), I8, "swiglu", "direct32", "listed"),
    ((36, 272, 1920, 300), I8, "swiglu", "tiles32", "listed"),
    ((173, 272, 640, 300), I8, "swiglu", "tiles64", "listed"),
    ((72, 608, 1120, 300), I8, "swiglu", "tiles128", "listed"),
    ((5820, 1568, 2347, 3), FP32, "none", "tiles256", "halved"),
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
    bm, parts = plan["tile_rows"], plan["k_parts"]
    mt = sum(-(-m // bm) for key, m in groups if key < 3) if groups else -(-rows // bm)
    nt = -(-n // 256) * parts
    return 2 * (-(-mt * nt // 8) % 32) <= 32


def check_form(plan, size, epilogue, kernel, how):
    rows, _, n, groups = size
    assert ("tiles" if plan["lds_tiles"] else "direct") + str(plan["tile_rows"]) == kernel
    assert (plan["k_parts"] > 1) == ("split" in how) and bool(plan["listed"]) == ("listed" in how)
    if plan["tile_rows"] >= 128 and plan["lds_tiles"] and "listed" not in how:
        assert _last_round_halved(plan, _groups(rows, groups), rows, n, epilogue) == ("halved" in how)


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
