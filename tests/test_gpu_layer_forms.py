"""Every form of the layer's first launch against the definition in 64 bits: 1, 4 or 8 waves to a
tile, compiled for 16 or 64 tokens, slots found by lanes or through LDS, on all three pairs of
types.  Each size asserts the form that it takes.  Hidden sizes end inside a block of 128 and have numbers
of blocks that the waves do not divide; activations lie in wider rows whose gaps hold NaN."""

import numpy as np
import pytest
import torch

import unpermute_ffnwb_batching_amd as F
from _expert import canary, close, dev, fp8, layer_inputs, layer_reference, untouched

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16

# (tokens, slots, experts, hidden, inter), (up_tokens, up_waves, lane_routing)
FORMS = [
    ((4, 3, 5, 272, 144), (16, 1, 1)), ((16, 5, 6, 336, 80), (16, 1, 0)),
    ((30, 2, 3, 272, 48), (64, 1, 1)), ((40, 3, 4, 144, 80), (64, 1, 0)),
    ((1, 2, 4, 400, 16), (16, 4, 1)), ((3, 2, 5, 528, 80), (16, 4, 1)), ((13, 6, 9, 1040, 48), (16, 4, 0)),
    ((20, 3, 4, 656, 48), (64, 4, 1)), ((40, 4, 5, 912, 64), (64, 4, 0)), ((64, 2, 3, 784, 32), (64, 4, 0)),
    ((1, 1, 2, 1936, 16), (16, 8, 1)), ((2, 2, 3, 2064, 32), (16, 8, 1)), ((16, 5, 6, 2192, 48), (16, 8, 0)),
    ((1, 2, 2, 7168, 32), (16, 8, 1)),
    ((18, 2, 3, 2064, 32), (64, 8, 1)), ((33, 4, 4, 1936, 48), (64, 8, 0)), ((64, 3, 3, 3216, 16), (64, 8, 0)),
    # many experts times inter: four waves although the hidden size is long
    ((9, 8, 40, 1936, 416), (16, 4, 0)),
]


@pytest.mark.parametrize("dtype,weights", [(BF16, "fp8"), (FP16, "fp8"), (BF16, "bf16")], ids=["bf16-fp8", "fp16-fp8", "bf16-bf16"])
@pytest.mark.parametrize("size,form", FORMS, ids=lambda v: "x".join(map(str, v)))
def test_first_launch(size, form, dtype, weights):
    T, K, E, H, inter = size
    c = layer_inputs(sum(size), *size, weights)
    rng = np.random.default_rng(sum(size))
    c["ids"][rng.random((T, K)) < 0.1] = -1
    mask = rng.random((T, K)) < 0.9
    wide = torch.full((T, H + 64), float("nan"), dtype=dtype, device="cuda")
    wide[:, 32:32 + H] = dev(c["x"], dtype)
    x = wide[:, 32:32 + H]
    y = canary((T, H + 16), dtype)
    w = [fp8(c["w13"]), fp8(c["w2"])] if weights == "fp8" else [c["w13"].cuda(), c["w2"].cuda()]
    call = F.LayerCall(x, dev(c["ids"]), *w, w13_scale=dev(c["w13s"]) if weights == "fp8" else None,
                       w2_scale=dev(c["w2s"]) if weights == "fp8" else None, expert_scales=dev(c["scales"]),
                       active_mask=dev(mask), out={"y": y[:, 8:8 + H]})
    plan = F.moe_layer_plan(call.desc)
    assert (plan["up_tokens"], plan["up_waves"], plan["lane_routing"]) == form
    print(f"layer {size} {dtype} {weights}: {plan}", flush=True)
    call.run()
    torch.cuda.synchronize()
    want, off = layer_reference(c, x, mask)
    close(call.out["y"], want, off, dtype)
    assert untouched(y[:, :8]) and untouched(y[:, 8 + H:])
    first = y.clone()
    for _ in range(3):
        call.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.uint8), y.view(torch.uint8))
