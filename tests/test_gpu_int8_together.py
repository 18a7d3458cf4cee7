"""The INT8 operators as a worker and its attention side use them: the norm into the rows that the
batching takes, the products behind the batching and between permute and unpermute; on several
streams at once, in two graphs replayed in turn, with hooks, with inputs dropped early."""

import numpy as np
import pytest
import torch

import synth
import unpermute_ffnwb_batching_amd as F
from _expert import FP8, canary, dev, host, untouched
from _int8 import close, codes, matmul_inputs, matmul_reference, norm_error, quantised_close
from oracle import int8_rows as O
from unpermute_ffnwb_batching_amd.hip_events import HipEvent

pytestmark = pytest.mark.gpu

BF16, FP16, FP32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


def _weights(seed, experts, hidden, inter):
    rng = np.random.default_rng(seed)
    w = {}
    for name, n, k in (("13", 2 * inter, hidden), ("2", hidden, inter)):
        w["w" + name] = codes(rng, (experts, n, k))
        w["s" + name] = (rng.uniform(0.5, 1.5, (experts, n)) / (50 * np.sqrt(k))).astype(np.float32)
    return w


def _check_product(got, x, xs, w, ws, groups, epilogue, dtype):
    """One product of a chain against the definition, on the device rows that went into it."""
    c = dict(x=x.cpu().numpy(), xs=xs.cpu().numpy(), w=w, ws=ws)
    want, off, written = matmul_reference(c, groups, epilogue, dtype)
    assert written.all()
    if dtype == I8:
        quantised_close(got["y"][:len(want)], got["y_scale"][:len(want)], want, off)
    else:
        close(got["y"][:len(want)], want, off, dtype)


def test_norm_batching_and_the_experts_products():
    # the attention side norms 32 tokens into INT8 rows with their scale behind them, as the data area
    # holds them; every slot of a token carries its row; the worker batches them and runs its experts
    A, BS, K1, H, inter, E = 4, 8, 5, 272, 144, 16
    T, Y = A * BS, A * BS * K1
    case = synth.batching_case(81, A, BS, K1, H, E, 2, synth.INT8, n_masked=20)
    g = torch.Generator().manual_seed(82)
    x, res = (torch.randn((T, H), generator=g).to(BF16).cuda() for _ in range(2))
    gamma = (1 + 0.2 * torch.randn(H, generator=g)).cuda()
    packed = torch.zeros((T, H + 4), dtype=I8, device="cuda")
    n = F.moe_rmsnorm_quant(x, gamma, residual=res, out={"q": packed[:, :H], "scale": packed.view(FP32)[:, H // 4]})
    slots = packed.repeat_interleave(K1, dim=0).contiguous()
    opt = {k: dev(case[k]) if case[k] is not None else None for k in ("mask", "layer_ids")}
    b = F.ffnwb_batching(slots, dev(case["expert_ids"]), expert_num=E, layer_num=2, max_out_shape=(A, BS, K1, H),
                         token_dtype=F.FFNWB_DT_INT8, token_row_stride=H + 4, **opt)
    w = _weights(83, E, H, inter)
    h = F.moe_grouped_matmul_int8(b["y"], b["dynamic_scale"], dev(w["w13"]), dev(w["s13"]), group_list=b["group_list"],
                                  epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=I8, out={"y": canary((Y, inter), I8), "y_scale": canary((Y,), FP32)})
    y = F.moe_grouped_matmul_int8(h["y"], h["y_scale"], dev(w["w2"]), dev(w["s2"]), group_list=b["group_list"],
                                  out={"y": canary((Y, H), BF16)})
    print("norm, batching, gate and up, down", flush=True)
    torch.cuda.synchronize()
    s, want = O.rmsnorm(x.float().cpu().numpy(), gamma.cpu().numpy(), res.float().cpu().numpy(), 1e-6)
    quantised_close(n["q"], n["scale"], want, norm_error(H) * np.abs(want))
    assert torch.equal(n["residual_out"].cpu(), torch.from_numpy(s).to(BF16))
    act = int(b["actual_token_num"].item())
    assert 0 < act < Y
    token = b["token_ids"][:act].long() // K1
    assert torch.equal(b["y"][:act], n["q"][token]) and torch.equal(b["dynamic_scale"][:act], n["scale"][token])
    groups = [tuple(v) for v in b["group_list"].tolist()]
    _check_product(h, b["y"][:act], b["dynamic_scale"][:act], w["w13"], w["s13"], groups, "swiglu", I8)
    _check_product(y, h["y"][:act], h["y_scale"][:act], w["w2"], w["s2"], groups, "none", BF16)
    for t in (h["y"], h["y_scale"], y["y"]):
        assert untouched(t[act:])


def test_bf16_batching_quantised_for_the_products():
    A, BS, K1, H, inter, E = 2, 16, 3, 144, 80, 8
    Y = A * BS * K1
    case = synth.batching_case(84, A, BS, K1, H, E, 1, synth.BF16, n_masked=9)
    b = F.ffnwb_batching(dev(case["token_bytes"]), dev(case["expert_ids"]), expert_num=E, layer_num=1, max_out_shape=(A, BS, K1, H),
                         token_dtype=F.FFNWB_DT_BF16, token_row_stride=case["stride"], mask=dev(case["mask"]))
    w = _weights(85, E, H, inter)
    q = F.moe_quant_int8(b["y"], actual_rows=b["actual_token_num"], out={"q": canary((Y, H), I8), "scale": canary((Y,), FP32)})
    h = F.moe_grouped_matmul_int8(q["q"], q["scale"], dev(w["w13"]), dev(w["s13"]), group_list=b["group_list"],
                                  epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=FP16, out={"y": canary((Y, inter), FP16)})
    torch.cuda.synchronize()
    act = int(b["actual_token_num"].item())
    want, scales = O.quantise_rows(b["y"][:act].float().cpu().numpy())
    np.testing.assert_array_equal(q["q"][:act].cpu().numpy(), want)
    np.testing.assert_array_equal(q["scale"][:act].cpu().numpy(), scales)
    _check_product(h, q["q"][:act], q["scale"][:act], w["w13"], w["s13"], [tuple(v) for v in b["group_list"].tolist()], "swiglu", FP16)
    for t in (q["q"], q["scale"], h["y"]):
        assert untouched(t[act:])


def test_norm_permute_products_unpermute():
    # INT8 rows with their scale behind them, 16 bytes wide so that rows stay aligned, moved whole by the permute
    T, K, E, H, inter = 24, 3, 8, 256, 128
    rng = np.random.default_rng(86)
    x = dev(rng.normal(size=(T, H)).astype(np.float32), FP16)
    gamma = torch.ones(H, dtype=FP16, device="cuda")
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:K] for _ in range(T)])).cuda()
    rmap = torch.zeros((T, E), dtype=torch.int8, device="cuda").scatter_(1, ids, 1)
    probs = torch.zeros((T, E), device="cuda").scatter_(1, ids, dev(rng.uniform(0.1, 1, (T, K)).astype(np.float32)))
    group_list = torch.stack([torch.arange(E, device="cuda"), rmap.sum(0, dtype=torch.int64)], 1).contiguous()
    packed = torch.zeros((T, H + 16), dtype=I8, device="cuda")
    F.moe_rmsnorm_quant(x, gamma, out={"q": packed[:, :H], "scale": packed.view(FP32)[:, H // 4]})
    p = F.moe_permute(packed, rmap, num_out_rows=T * K)
    rows, scale = p["permuted_tokens"][:, :H], p["permuted_tokens"].view(FP32)[:, H // 4]
    w = _weights(87, E, H, inter)
    h = F.moe_grouped_matmul_int8(rows, scale, dev(w["w13"]), dev(w["s13"]), group_list=group_list, epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=I8)
    d = F.moe_grouped_matmul_int8(h["y"], h["y_scale"], dev(w["w2"]), dev(w["s2"]), group_list=group_list, out_dtype=BF16)
    u = F.moe_unpermute(d["y"], p["sorted_indices"], rmap, probs, padded_mode=False, restore_shape=(T, H))["unpermuted"]
    print("norm, permute, products, unpermute", flush=True)
    torch.cuda.synchronize()
    groups = [tuple(v) for v in group_list.tolist()]
    _check_product(h, rows, scale, w["w13"], w["s13"], groups, "swiglu", I8)
    _check_product(d, h["y"], h["y_scale"], w["w2"], w["s2"], groups, "none", BF16)
    at = p["sorted_indices"].view(T, K).long()
    terms = host(d["y"])[at.cpu().numpy()] * np.take_along_axis(host(probs), np.sort(ids.cpu().numpy(), 1), 1)[:, :, None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    assert (np.abs(host(u) - want) <= 2.0 ** -8 * np.abs(want) + 2 * K * 2.0 ** -24 * size * (1 + 2.0 ** -7)).all()


def _calls(seed):
    rng = np.random.default_rng(seed)
    m = matmul_inputs(seed, 300, 528, 288, 6)
    gl = torch.tensor([[0, 40], [2, 130], [3, 1], [5, 100]], device="cuda")
    x, res = (dev(rng.normal(size=(100, 700)).astype(np.float32), BF16) for _ in range(2))
    gamma = dev(rng.normal(size=700).astype(np.float32), BF16)
    actual = torch.tensor([90], device="cuda")
    args = [dev(m[k]) for k in ("x", "xs", "w", "ws")]
    lm = matmul_inputs(seed + 1, 256, 7168, 2048)     # K split over waves
    long = [dev(lm[k]) for k in ("x", "xs", "w", "ws")]
    many = matmul_inputs(seed + 2, 900, 64, 64, 6)    # listed by a launch of its own
    groups = dev(np.stack([np.arange(300) % 6, np.full(300, 3)], 1).astype(np.int64))

    def rows(n, h, *dtypes):
        return [canary((n, h), t) for t in dtypes]

    q8, qf, s8, sf = *rows(100, 700, I8, FP8), canary((100,), FP32), canary((100, 6), FP32)
    ro, y = rows(100, 700, BF16, BF16)
    return [F.QuantInt8Call(x, actual_rows=actual, out={"q": canary((100, 700), I8), "scale": canary((100,), FP32)}),
            F.RmsNormQuantCall(x, gamma, residual=res, actual_rows=actual, out={"q": q8, "scale": s8, "residual_out": ro}),
            F.RmsNormQuantCall(x, gamma, q_dtype=FP8, out={"q": qf, "scale": sf, "y": y}),
            F.GroupedMatmulInt8Call(*args, group_list=gl, epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=I8,
                                    out={"y": canary((300, 144), I8), "y_scale": canary((300,), FP32)}),
            F.GroupedMatmulInt8Call(*args, group_list=gl, out={"y": canary((300, 288), BF16)}),
            F.GroupedMatmulInt8Call(*long, out={"y": canary((256, 2048), BF16)}),
            F.GroupedMatmulInt8Call(*[dev(many[k]) for k in ("x", "xs", "w", "ws")], group_list=groups, epilogue=F.FFNWB_EPI_SWIGLU,
                                    out_dtype=I8, out={"y": canary((900, 32), I8), "y_scale": canary((900,), FP32)})]


def _outputs(calls):
    return [{k: v.clone().view(torch.uint8) for k, v in c.out.items()} for c in calls]


def _same(a, b):
    for i, (p, q) in enumerate(zip(a, b)):
        for k in q:
            assert torch.equal(p[k], q[k]), (i, k)


def test_the_calls_cover_the_workspaces():
    plans = [F.moe_grouped_matmul_int8_plan(c.desc) for c in _calls(7)[3:]]
    assert plans[2]["waves"] > 1 and plans[3]["listed"] and all(_calls(7)[i].ws_bytes > 0 for i in (3, 6))


def test_calls_on_streams_at_once():
    calls = _calls(91)
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    want = _outputs(calls)
    again = _calls(91)
    streams = [torch.cuda.Stream() for _ in again]
    torch.cuda.synchronize()
    print("seven calls on seven streams", flush=True)
    for _ in range(5):
        for c, s in zip(again, streams):
            c.run(s)
    torch.cuda.synchronize()
    _same(_outputs(again), want)


def test_two_graphs_replayed_with_new_inputs():
    eager, graphs, want = {s: _calls(s) for s in (101, 111, 121)}, [], {}
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
    for seeds in ((101, 111), (121, 101), (111, 121), (101, 101)):
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


@pytest.mark.parametrize("both", [True, False], ids=["both", "end-only"])
def test_timing_hooks(both):
    c = matmul_inputs(131, 200, 256, 96, 4)
    long = matmul_inputs(132, 256, 7168, 2048)
    x = dev(np.random.default_rng(133).normal(size=(64, 512)).astype(np.float32))
    events = [(HipEvent(), HipEvent()) for _ in range(5)]
    ev = [(b if both else None, e) for b, e in events]
    args, largs = ([dev(m[k]) for k in ("x", "xs", "w", "ws")] for m in (c, long))
    gl = torch.tensor([[1, 90], [3, 110]], device="cuda")
    calls = [F.QuantInt8Call(x, ev_quant=ev[0]), F.RmsNormQuantCall(x, torch.ones(512, device="cuda"), ev_norm=ev[1]),
             F.GroupedMatmulInt8Call(*args, out_dtype=FP32, ev_matmul=ev[2], group_list=gl),
             F.GroupedMatmulInt8Call(*args, out_dtype=I8, epilogue=F.FFNWB_EPI_SWIGLU, ev_matmul=ev[3], group_list=gl),
             F.GroupedMatmulInt8Call(*largs, ev_matmul=ev[4])]
    print(f"hooks both={both}", flush=True)
    for call, (b, e) in zip(calls, events):
        call.run()
        torch.cuda.synchronize()
        if both:
            ms = b.elapsed_ms(e)
            assert np.isfinite(ms) and 0.0 < ms < 1000.0
        else:
            e.synchronize()
    want, off, _ = matmul_reference(c, [(1, 90), (3, 110)], "none", FP32)
    close(calls[2].out["y"], want, off, FP32)


def test_empty_calls_record_their_events():
    e = [(HipEvent(), HipEvent()) for _ in range(3)]
    x = torch.zeros(0, 64, device="cuda")
    F.moe_quant_int8(x, ev_quant=e[0])
    F.moe_rmsnorm_quant(x, torch.ones(64, device="cuda"), ev_norm=e[1])
    F.moe_grouped_matmul_int8(torch.zeros(0, 64, device="cuda", dtype=I8), torch.zeros(0, device="cuda"),
                              torch.zeros(32, 64, device="cuda", dtype=I8), torch.zeros(32, device="cuda"), ev_matmul=e[2])
    torch.cuda.synchronize()
    for b, end in e:
        assert 0.0 <= b.elapsed_ms(end) < 1000.0


def _quant():
    x = torch.randn(3000, 1024, device="cuda")
    return lambda s: F.moe_quant_int8(x, stream=s), [x]


def _norm():
    x, r, g = torch.randn(3000, 1024, device="cuda"), torch.randn(3000, 1024, device="cuda"), torch.ones(1024, device="cuda")
    return lambda s: F.moe_rmsnorm_quant(x, g, residual=r, stream=s), [x, r, g]


def _matmul():
    c = matmul_inputs(201, 1200, 1040, 544)
    t = [dev(c[k]) for k in ("x", "xs", "w", "ws")]
    out = torch.empty((1200, 272), dtype=I8, device="cuda")
    return lambda s: F.moe_grouped_matmul_int8(*t, epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=I8, out={"y": out}, stream=s), [*t, out]


@pytest.mark.parametrize("make", [_quant, _norm, _matmul], ids=lambda f: f.__name__[1:])
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
