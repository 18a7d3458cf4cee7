"""The expert operators as a worker uses them: behind the batching and before the unpermute,
on several streams at once, captured in graphs, with timing hooks."""

import numpy as np
import pytest
import torch

import synth
import unpermute_ffnwb_batching_amd as F
from _expert import (FP8, canary, close, codes, dev, fp8, host, layer_inputs, layer_reference, matmul_inputs, matmul_reference,
                     quantised_close, untouched)
from oracle import expert_ffn as O
from unpermute_ffnwb_batching_amd.hip_events import HipEvent

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _weights(seed, experts, hidden, inter):
    c = layer_inputs(seed, 1, 1, experts, hidden, inter)
    return {k: c[k] for k in ("w13", "w13s", "w2", "w2s")}


def test_batching_then_the_experts_products():
    # 16 experts in 2 layers, a few slots masked; every step checked on the step before's output
    A, BS, K1, H, inter = 4, 8, 5, 272, 144
    case = synth.batching_case(81, A, BS, K1, H, 16, 2, synth.BF16, n_masked=20)
    Y = A * BS * K1
    opt = {k: dev(case[k]) if case[k] is not None else None for k in ("mask", "layer_ids")}
    b = F.ffnwb_batching(dev(case["token_bytes"]), dev(case["expert_ids"]), expert_num=16, layer_num=2,
                         max_out_shape=(A, BS, K1, H), token_dtype=F.FFNWB_DT_BF16, token_row_stride=case["stride"], **opt)
    w = _weights(82, 16, H, inter)
    q_out = {"q": canary((Y, H), FP8), "scale": canary((Y, 3), FP32)}
    q = F.moe_quant_fp8(b["y"], actual_rows=b["actual_token_num"], out=q_out)
    h_out = {"y": canary((Y, inter), FP8), "y_scale": canary((Y, 2), FP32)}
    h = F.moe_grouped_matmul_fp8(q["q"], q["scale"], fp8(w["w13"]), dev(w["w13s"]), group_list=b["group_list"],
                                 epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=FP8, out=h_out)
    y = F.moe_grouped_matmul_fp8(h["y"], h["y_scale"], fp8(w["w2"]), dev(w["w2s"]), group_list=b["group_list"],
                                 out={"y": canary((Y, H), BF16)})["y"]
    print("batching, quantising, gate and up, down", flush=True)
    torch.cuda.synchronize()
    act = int(b["actual_token_num"].item())
    assert 0 < act < Y
    groups = [tuple(g) for g in b["group_list"].tolist()]
    x_codes, x_scales = O.quantise_rows(b["y"][:act].float().cpu().numpy())
    np.testing.assert_array_equal(q["q"][:act].view(torch.uint8).cpu().numpy(), x_codes)
    np.testing.assert_array_equal(q["scale"][:act].cpu().numpy(), x_scales)
    c = dict(x=x_codes, xs=x_scales, w=w["w13"], ws=w["w13s"])
    want, off, written = matmul_reference(c, groups, "swiglu")
    assert written.all()
    quantised_close(h["y"][:act], h["y_scale"][:act], want, off)
    c = dict(x=h["y"][:act].view(torch.uint8).cpu().numpy(), xs=h["y_scale"][:act].cpu().numpy(), w=w["w2"], ws=w["w2s"])
    want, off, _ = matmul_reference(c, groups, "none", narrow=True)
    close(y[:act], want, off, BF16)
    for t in (q["q"], q["scale"], h["y"], h["y_scale"], y):
        assert untouched(t[act:])


def test_permute_products_unpermute_agree_with_the_layer():
    # the two ways of a layer: rows regrouped by expert, products in e4m3, weighted unpermute; and
    # moe_layer on the same experts, which keeps activations in BF16.  They differ by the
    # quantising of x and of h, each half a step of e4m3 (2^-4) of an element at most; over sums of hundreds of
    # terms of either sign that is some percent of the result's size.
    T, K, E, H, inter = 24, 3, 8, 512, 256
    c = layer_inputs(83, T, K, E, H, inter)
    x = dev(c["x"], BF16)
    ids = dev(c["ids"]).long()
    rmap = torch.zeros((T, E), dtype=torch.int8, device="cuda").scatter_(1, ids, 1)
    probs = torch.zeros((T, E), device="cuda").scatter_(1, ids, dev(c["scales"]))
    counts = rmap.sum(0, dtype=torch.int64)
    group_list = torch.stack([torch.arange(E, device="cuda"), counts], 1).contiguous()
    p = F.moe_permute(x, rmap, num_out_rows=T * K)
    q = F.moe_quant_fp8(p["permuted_tokens"])
    h = F.moe_grouped_matmul_fp8(q["q"], q["scale"], fp8(c["w13"]), dev(c["w13s"]), group_list=group_list,
                                 epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=FP8)
    d = F.moe_grouped_matmul_fp8(h["y"], h["y_scale"], fp8(c["w2"]), dev(c["w2s"]), group_list=group_list, out_dtype=BF16)
    u = F.moe_unpermute(d["y"], p["sorted_indices"], rmap, probs, padded_mode=False, restore_shape=(T, H))["unpermuted"]
    y = F.moe_layer(x, dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"]), w13_scale=dev(c["w13s"]), w2_scale=dev(c["w2s"]),
                    expert_scales=dev(c["scales"]))["y"]
    print("permute, products, unpermute against the layer", flush=True)
    torch.cuda.synchronize()
    want, off = layer_reference(c, x)
    close(y, want, off, BF16)
    a, b = host(u), host(y)
    assert np.linalg.norm(a - b) <= 0.15 * np.linalg.norm(b)
    assert np.linalg.norm(a - b) >= 1e-4 * np.linalg.norm(b)   # they are two computations


def test_layer_takes_the_expert_updates_outputs():
    c = layer_inputs(84, 30, 4, 12, 144, 48)
    ue = synth.update_expert_case(85, 30, 4, 12, 6, 3, F=7, scale_dtype=synth.FP32, n_active=20, n_bad_ids=6)
    kw = dict(local_rank_id=2, world_size=6, balance_mode=0)
    u = F.moe_update_expert(dev(ue["expert_ids"]), dev(ue["eplb_table"]), expert_scales=dev(ue["expert_scales"]),
                            pruning_threshold=dev(ue["pruning_threshold"]), active_mask=dev(ue["active_mask"]), **kw)
    ids, mask = u["balanced_expert_ids"], u["balanced_active_mask"]
    y = F.moe_layer(dev(c["x"], BF16), ids, fp8(c["w13"]), fp8(c["w2"]), w13_scale=dev(c["w13s"]), w2_scale=dev(c["w2s"]),
                    expert_scales=dev(ue["expert_scales"]), active_mask=mask)["y"]
    print("expert update, then the layer", flush=True)
    torch.cuda.synchronize()
    c["ids"] = ids.cpu().numpy()   # instances past the 12 experts are no experts here
    want, off = layer_reference(c, dev(c["x"], BF16), mask.cpu().numpy(), ue["expert_scales"])
    close(y, want, off, BF16)


def _calls(seed):
    rng = np.random.default_rng(seed)
    m, lc = matmul_inputs(seed, 300, 528, 288, 6), layer_inputs(seed + 1, 20, 4, 12, 272, 144)
    gl = torch.tensor([[0, 40], [2, 130], [3, 1], [5, 100]], device="cuda")
    x = dev(rng.normal(size=(100, 700)).astype(np.float32), BF16)
    few = layer_inputs(seed + 2, 3, 2, 6, 128, 640)
    lm = matmul_inputs(seed + 3, 192, 7168, 700)   # split over K
    long = (fp8(lm["x"]), dev(lm["xs"]), fp8(lm["w"]), dev(lm["ws"]))

    def layer(c):
        return F.LayerCall(dev(c["x"], BF16), dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"]), w13_scale=dev(c["w13s"]),
                           w2_scale=dev(c["w2s"]), expert_scales=dev(c["scales"]))

    args = (fp8(m["x"]), dev(m["xs"]), fp8(m["w"]), dev(m["ws"]))
    return [F.QuantFp8Call(x, actual_rows=torch.tensor([90], device="cuda"),
                           out={"q": canary((100, 700), FP8), "scale": canary((100, 6), FP32)}),
            F.GroupedMatmulFp8Call(*args, group_list=gl, epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=FP8,
                                   out={"y": canary((300, 144), FP8), "y_scale": canary((300, 2), FP32)}),
            F.GroupedMatmulFp8Call(*args, group_list=gl, out={"y": canary((300, 288), BF16)}),
            F.GroupedMatmulFp8Call(*long, out={"y": canary((192, 700), BF16)}), layer(lc), layer(few)]


def _outputs(calls):
    return [{k: v.clone().view(torch.uint8) for k, v in c.out.items()} for c in calls]


def _same(a, b):
    for i, (p, q) in enumerate(zip(a, b)):
        for k in q:
            assert torch.equal(p[k], q[k]), (i, k)


def test_calls_on_streams_at_once():
    calls = _calls(91)
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    want = _outputs(calls)
    again = _calls(91)
    streams = [torch.cuda.Stream() for _ in again]
    torch.cuda.synchronize()
    print("six calls on six streams", flush=True)
    for _ in range(5):
        for c, s in zip(again, streams):
            c.run(s)
    torch.cuda.synchronize()
    _same(_outputs(again), want)


def test_one_shot_on_a_side_stream():
    c = layer_inputs(92, 33, 3, 8, 256, 144)
    side = torch.cuda.Stream()
    args = [dev(c["x"], BF16), dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"])]
    kw = dict(w13_scale=dev(c["w13s"]), w2_scale=dev(c["w2s"]), expert_scales=dev(c["scales"]))
    side.wait_stream(torch.cuda.current_stream())
    print("one-shot layer on a held-back side stream", flush=True)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    y = F.moe_layer(*args, stream=side, **kw)["y"]
    junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want, off = layer_reference(c, args[0])
    close(y, want, off, BF16)
    assert all(int(j.min()) == 7 == int(j.max()) for j in junk)


def test_two_graphs_replayed_with_new_inputs():
    eager, graphs = {s: _calls(s) for s in (101, 111, 121)}, []
    want = {}
    for s, calls in eager.items():
        for c in calls:
            c.run()
        torch.cuda.synchronize()
        want[s] = _outputs(calls)
    captured = [_calls(101), _calls(111)]
    for calls in captured:
        torch.cuda.synchronize()
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                for c in calls:
                    c.run(side)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(g)
    print("two graphs, replayed in turn with eager work between", flush=True)
    for rep, seeds in enumerate(((101, 111), (121, 101), (111, 121), (101, 101))):
        for calls, s in zip(captured, seeds):
            for c, e in zip(calls, eager[s]):
                for t, src in zip(c._keep, e._keep):
                    if t is not None:
                        t.view(torch.uint8).reshape(-1).copy_(src.view(torch.uint8).reshape(-1))
        torch.ones(1 << 20, device="cuda").mul_(3.0).sum().item()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for calls, s in zip(captured, seeds):
            _same(_outputs(calls), want[s])


def test_repeats_of_split_layers_are_bit_identical():
    # few columns: the second launch is split over workgroups, whose order of arrival changes
    for size in ((5, 4, 16, 64, 2048), (64, 8, 40, 128, 640), (17, 2, 9, 16, 1040)):
        c = layer_inputs(sum(size), *size)
        call = F.LayerCall(dev(c["x"], BF16), dev(c["ids"]), fp8(c["w13"]), fp8(c["w2"]), w13_scale=dev(c["w13s"]),
                           w2_scale=dev(c["w2s"]), expert_scales=dev(c["scales"]))
        print(f"layer {size}, 40 times", flush=True)
        call.run()
        torch.cuda.synchronize()
        first = call.out["y"].clone()
        want, off = layer_reference(c, dev(c["x"], BF16))
        close(first, want, off, BF16)
        for _ in range(40):
            call.run()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.uint8), call.out["y"].view(torch.uint8))


@pytest.mark.parametrize("both", [True, False], ids=["both", "end-only"])
def test_timing_hooks(both):
    c = matmul_inputs(131, 200, 256, 96, 4)
    lc = layer_inputs(132, 4, 2, 6, 128, 64)
    x = dev(np.random.default_rng(133).normal(size=(64, 512)).astype(np.float32))
    events = [(HipEvent(), HipEvent()) for _ in range(3)]
    ev = [(b if both else None, e) for b, e in events]
    calls = [F.QuantFp8Call(x, ev_quant=ev[0]),
             F.GroupedMatmulFp8Call(fp8(c["x"]), dev(c["xs"]), fp8(c["w"]), dev(c["ws"]), out_dtype=FP32, ev_matmul=ev[1],
                                    group_list=torch.tensor([[1, 90], [3, 110]], device="cuda")),
             F.LayerCall(dev(lc["x"], BF16), dev(lc["ids"]), fp8(lc["w13"]), fp8(lc["w2"]), w13_scale=dev(lc["w13s"]),
                         w2_scale=dev(lc["w2s"]), expert_scales=dev(lc["scales"]), ev_layer=ev[2])]
    print(f"hooks both={both}", flush=True)
    for call, (b, e) in zip(calls, events):
        call.run()
        torch.cuda.synchronize()
        if both:
            ms = b.elapsed_ms(e)
            assert np.isfinite(ms) and 0.0 < ms < 1000.0
        else:
            e.synchronize()
    want, off, _ = matmul_reference(c, [(1, 90), (3, 110)])
    close(calls[1].out["y"], want, off, FP32)


def test_tensors_made_on_another_stream():
    # inputs come from work on a side stream that the current one waits for; the call runs on a third
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        x = torch.randn(50, 384, device="cuda").to(FP16)
    third.wait_stream(side)
    q = F.moe_quant_fp8(x, stream=third)
    torch.cuda.synchronize()
    want, scales = O.quantise_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(q["q"].view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(q["scale"].cpu().numpy(), scales)
