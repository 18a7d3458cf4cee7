"""One-shot calls on a stream the caller names, whose inputs were made on the current one and are
dropped right after the call: the allocator may not hand their memory out before the call's
kernels have run.  Only addresses are compared, nothing is written to the new memory."""

import pytest
import torch

import synth
import unpermute_ffnwb_batching_amd as F
from _expert import dev, fp8, layer_inputs, matmul_inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _quant():
    x = torch.randn(3000, 1024, device="cuda")
    return lambda s: F.moe_quant_fp8(x, stream=s), [x]


def _matmul():
    c = matmul_inputs(201, 1200, 1040, 520)
    x, xs, w, ws = fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"])
    out = torch.empty((1200, 520), dtype=BF16, device="cuda")    # an output made on the current stream too
    return lambda s: F.moe_grouped_matmul_fp8(x, xs, w, ws, out={"y": out}, stream=s), [x, xs, w, ws, out]


def _layer():
    c = layer_inputs(202, 64, 2, 4, 1040, 528)
    t = [dev(c["x"], BF16), dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"]), dev(c["w13s"]), dev(c["w2s"])]
    return lambda s: F.moe_layer(*t[:4], w13_scale=t[4], w2_scale=t[5], stream=s), t


def _permute():
    x = torch.randn(2048, 512, device="cuda").to(BF16)
    rmap = torch.zeros(2048, 16, dtype=torch.int8, device="cuda")
    rmap[:, 3] = 1
    return lambda s: F.moe_permute(x, rmap, num_out_rows=2048, stream=s), [x, rmap]


def _unpermute():
    x = torch.randn(2048, 512, device="cuda").to(BF16)
    at = torch.arange(2048, dtype=torch.int32, device="cuda")
    return lambda s: F.moe_unpermute(x, at, padded_mode=False, restore_shape=(2048, 512), stream=s), [x, at]


def _batching():
    case = synth.batching_case(203, 8, 16, 9, 512, 64, 1, synth.BF16)
    x, ids = dev(case["token_bytes"]), dev(case["expert_ids"])
    return lambda s: F.ffnwb_batching(x, ids, expert_num=64, layer_num=1, max_out_shape=(8, 16, 9, 512),
                                      token_dtype=F.FFNWB_DT_BF16, token_row_stride=case["stride"], stream=s), [x, ids]


def _update_expert():
    ue = synth.update_expert_case(204, 400, 4, 12, 6, 3, F=7)
    ids, table = dev(ue["expert_ids"]), dev(ue["eplb_table"])
    return lambda s: F.moe_update_expert(ids, table, local_rank_id=2, world_size=6, balance_mode=0, stream=s), [ids, table]


@pytest.mark.parametrize("make", [_quant, _matmul, _layer, _permute, _unpermute, _batching, _update_expert],
                         ids=lambda f: f.__name__[1:])
def test_dropped_inputs_are_kept_until_the_call_has_run(make):
    side = torch.cuda.Stream()
    first = make()           # loads the kernels; held, so that its memory is not what is handed out
    torch.cuda.synchronize()
    first[0](side)
    call, tensors = make()
    torch.cuda.synchronize()
    print(make.__name__[1:], flush=True)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)    # about a tenth of a second
    held = call(side)
    old = {t.data_ptr(): t.untyped_storage().nbytes() for t in tensors}
    del call, tensors, held
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in old.values()]
    still_held_back = not side.query()
    assert not {t.data_ptr() for t in again} & set(old)
    torch.cuda.synchronize()
    assert still_held_back, "the spin was too short to show anything"


def test_a_prepared_call_marks_each_stream_once_and_keeps_its_results():
    x = torch.randn(64, 512, device="cuda").to(BF16)
    call = F.QuantFp8Call(x)
    call.run()
    torch.cuda.synchronize()
    want = call.out["q"].view(torch.uint8).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(4):
        for s in streams:
            call.out["q"].view(torch.uint8).zero_()
            s.wait_stream(torch.cuda.current_stream())
            call.run(s)
            torch.cuda.current_stream().wait_stream(s)
            assert torch.equal(call.out["q"].view(torch.uint8), want)
    assert len(call._marked) == 3
