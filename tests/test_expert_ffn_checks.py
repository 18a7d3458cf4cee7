"""Host-only checks of the expert operators: descriptor layouts, status codes of bad
arguments before any device work, and the binding's refusals."""

import ctypes

import pytest
import torch

import unpermute_ffnwb_batching_amd as F

FAKE = 0x1000
FP8, BF16, f32, i32, i64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.int64


def _ws(name, d):
    n = ctypes.c_size_t(0)
    return getattr(F.lib(), name + "_workspace_size")(ctypes.byref(d), ctypes.byref(n)), n.value


def _fill(d, vals, ptrs, over):
    for k, v in vals.items():
        setattr(d, k, v)
    for p in ptrs:
        setattr(d, p, FAKE)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def _quant(**over):
    return _fill(F.QuantFp8Desc(), dict(dtype=1, num_rows=4, hidden=256), ("x", "q", "scale"), over)


def _matmul(**over):
    return _fill(F.GroupedMatmulFp8Desc(), dict(epilogue=0, out_dtype=1, num_rows=8, in_features=256, out_features=96,
                                                num_experts=4, num_groups=4),
                 ("x", "x_scale", "w", "w_scale", "group_list", "y", "y_scale"), over)


def _layer(**over):
    return _fill(F.LayerDesc(), dict(dtype=1, weight_dtype=6, id_dtype=4, scale_dtype=3, num_tokens=4, slots=3, hidden=256,
                                     inter_size=96, num_experts=8),
                 ("x", "expert_ids", "expert_scales", "active_mask", "w13", "w13_scale", "w2", "w2_scale", "y"), over)


def test_descriptor_layouts():
    L = F.lib()
    assert L.moe_quant_fp8_desc_size() == ctypes.sizeof(F.QuantFp8Desc)
    assert L.moe_grouped_matmul_fp8_desc_size() == ctypes.sizeof(F.GroupedMatmulFp8Desc)
    assert L.moe_layer_desc_size() == ctypes.sizeof(F.LayerDesc)


MAKE = {"moe_quant_fp8": _quant, "moe_grouped_matmul_fp8": _matmul, "moe_layer": _layer}


@pytest.mark.parametrize("name", list(MAKE))
def test_null_descriptor_and_size(name):
    n = ctypes.c_size_t(0)
    assert getattr(F.lib(), name + "_workspace_size")(None, ctypes.byref(n)) == F.FFNWB_ERR_PARAM_NULLPTR
    assert getattr(F.lib(), name + "_workspace_size")(ctypes.byref(MAKE[name]()), None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert getattr(F.lib(), name)(None, None, 0, None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert _ws(name, MAKE[name]())[0] == F.FFNWB_OK


@pytest.mark.parametrize("name,field", [("moe_quant_fp8", p) for p in ("x", "q", "scale")] +
                         [("moe_grouped_matmul_fp8", p) for p in ("x", "x_scale", "w", "w_scale", "y")] +
                         [("moe_layer", p) for p in ("x", "expert_ids", "w13", "w2", "y")])
def test_required_pointers(name, field):
    assert _ws(name, MAKE[name](**{field: None}))[0] == F.FFNWB_ERR_PARAM_NULLPTR


def test_optional_pointers():
    assert _ws("moe_quant_fp8", _quant(actual_rows=FAKE))[0] == 0
    assert _ws("moe_grouped_matmul_fp8", _matmul(group_list=None, num_groups=0, num_experts=1))[0] == 0
    assert _ws("moe_grouped_matmul_fp8", _matmul(y_scale=None))[0] == 0
    assert _ws("moe_grouped_matmul_fp8", _matmul(out_dtype=6, epilogue=1, y_scale=None))[0] == F.FFNWB_ERR_PARAM_NULLPTR
    assert _ws("moe_layer", _layer(expert_scales=None, active_mask=None))[0] == 0
    assert _ws("moe_layer", _layer(weight_dtype=1, w13_scale=None, w2_scale=None))[0] == 0


@pytest.mark.parametrize("name,over", [
    *[("moe_quant_fp8", o) for o in (
        dict(dtype=2), dict(dtype=6), dict(dtype=-1), dict(reserved0=1), dict(num_rows=-1), dict(hidden=0),
        dict(hidden=(1 << 20) + 1), dict(num_rows=1 << 29), dict(num_rows=1 << 62), dict(x_row_stride=511), dict(x_row_stride=510),
        dict(x_row_stride=-512), dict(q_row_stride=255), dict(scale_row_stride=1), dict(x=FAKE + 1), dict(dtype=3, x=FAKE + 2),
        dict(x_row_stride=1 << 62), dict(q_row_stride=1 << 62), dict(scale_row_stride=1 << 62))],
    *[("moe_grouped_matmul_fp8", o) for o in (
        dict(epilogue=2), dict(epilogue=-1), dict(out_dtype=2), dict(out_dtype=6), dict(out_dtype=7), dict(num_rows=-1),
        dict(num_rows=(1 << 24) + 1), dict(in_features=0), dict(in_features=24), dict(in_features=(1 << 18) + 16),
        dict(out_features=0), dict(out_features=(1 << 18) + 1), dict(epilogue=1, out_features=48),
        dict(num_experts=0), dict(num_experts=8193), dict(num_groups=0), dict(num_groups=8193), dict(group_list=None),
        dict(group_list=None, num_groups=0), dict(x_row_stride=240), dict(x_row_stride=264), dict(x_scale_stride=1),
        dict(x_row_stride=1 << 40), dict(x_scale_stride=1 << 40), dict(y_row_stride=1 << 40),
        dict(y_row_stride=190), dict(y_row_stride=193), dict(epilogue=1, out_features=512, out_dtype=6, y_scale_stride=1),
        dict(x=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 1),
        dict(num_rows=1 << 24, out_features=1 << 18, group_list=None, num_groups=0, num_experts=1))],
    *[("moe_layer", o) for o in (
        dict(dtype=3), dict(dtype=2), dict(weight_dtype=0), dict(dtype=0, weight_dtype=1, w13_scale=None, w2_scale=None),
        dict(weight_dtype=1), dict(w13_scale=None), dict(w2_scale=None), dict(id_dtype=3), dict(scale_dtype=6),
        dict(num_tokens=-1), dict(num_tokens=65), dict(slots=0), dict(slots=65), dict(hidden=0), dict(hidden=24),
        dict(hidden=(1 << 18) + 16), dict(inter_size=0), dict(inter_size=24), dict(inter_size=(1 << 17) + 16),
        dict(num_experts=0), dict(num_experts=8193), dict(x_row_stride=504), dict(x_row_stride=520), dict(y_row_stride=511),
        dict(expert_ids_stride=2), dict(expert_scales_stride=2), dict(active_mask_stride=2), dict(x=FAKE + 2), dict(w13=FAKE + 8),
        dict(w2=FAKE + 8), dict(y=FAKE + 1), dict(x_row_stride=1 << 62),
        dict(num_tokens=64, slots=64, inter_size=1 << 17, num_experts=8192))],
])
def test_invalid_parameters(name, over):
    assert _ws(name, MAKE[name](**over))[0] == F.FFNWB_ERR_PARAM_INVALID
    assert getattr(F.lib(), name)(ctypes.byref(MAKE[name](**over)), None, 0, None) == F.FFNWB_ERR_PARAM_INVALID


@pytest.mark.parametrize("name,most,past", [
    ("moe_quant_fp8", dict(num_rows=(1 << 28) - 16, hidden=128), dict(num_rows=(1 << 28) - 15, hidden=128)),
    ("moe_quant_fp8", dict(num_rows=32767, hidden=1 << 20, x_row_stride=1 << 40), dict(num_rows=32768, hidden=1 << 20)),
    ("moe_quant_fp8", dict(num_rows=1 << 27, hidden=128, x_row_stride=1 << 33), dict(num_rows=1 << 27, hidden=128, x_row_stride=(1 << 33) + 2)),
    # the widest tiles are 256 x 256 (16-bit results) and 128 x 256 (FP32)
    ("moe_grouped_matmul_fp8", dict(num_rows=1 << 24, out_features=(1 << 14) - 256), dict(num_rows=1 << 24, out_features=1 << 14)),
    ("moe_grouped_matmul_fp8", dict(num_rows=1 << 23, out_features=(1 << 14) - 256, out_dtype=3),
     dict(num_rows=1 << 23, out_features=1 << 14, out_dtype=3)),
    # rows too far apart for the tiles: 64 x 16
    ("moe_grouped_matmul_fp8", dict(num_rows=1 << 24, out_features=240, x_row_stride=1 << 32),
     dict(num_rows=1 << 24, out_features=256, x_row_stride=1 << 32)),
    ("moe_layer", dict(num_tokens=64, slots=64, num_experts=4096, inter_size=(2047) * 16),
     dict(num_tokens=64, slots=64, num_experts=4096, inter_size=2048 * 16)),
])
def test_largest_sizes(name, most, past):
    if name == "moe_grouped_matmul_fp8":
        most, past = ({**o, "num_groups": 1} for o in (most, past))
    assert _ws(name, MAKE[name](**most))[0] == F.FFNWB_OK
    assert _ws(name, MAKE[name](**past))[0] == F.FFNWB_ERR_PARAM_INVALID


def test_a_call_whose_widest_tiles_fit_is_never_refused():
    # (ceil(R / 64) + num_groups) * ceil(F / 16) up to the workgroups of a launch, whatever the times expected
    for groups in (1, 300, 8192):
        for f in (16, 512, 1 << 12, 1 << 17):
            rows = min(((1 << 22) - 8) // (f // 16) - groups, 1 << 18) * 64
            if rows <= 0:
                continue
            for over in (dict(out_features=f), dict(out_features=f, out_dtype=3), dict(out_features=2 * f, epilogue=1),
                         dict(out_features=2 * f, epilogue=1, out_dtype=6)):
                for stride in (0, 1 << 30):
                    d = _matmul(num_rows=rows, num_groups=groups, num_experts=64, in_features=128, x_row_stride=stride, **over)
                    assert _ws("moe_grouped_matmul_fp8", d)[0] == F.FFNWB_OK, (groups, f, over, stride)


def test_calls_on_the_cpu_do_not_run():
    for make in (_quant_call, _matmul_call, _layer_call):
        with pytest.raises(ValueError, match="GPU"):
            make().run()


def test_workspace_is_checked_before_any_device_work():
    for name, over in (("moe_grouped_matmul_fp8", dict(num_groups=2000)),
                       ("moe_grouped_matmul_fp8", dict(num_rows=520, in_features=8192, out_features=1024, epilogue=1, out_dtype=6)),
                       ("moe_layer", {})):
        d = MAKE[name](**over)
        st, n = _ws(name, d)
        assert st == 0 and n > 0
        call = getattr(F.lib(), name)
        assert call(ctypes.byref(d), None, n, None) == F.FFNWB_ERR_WORKSPACE
        assert call(ctypes.byref(d), FAKE, n - 1, None) == F.FFNWB_ERR_WORKSPACE
        assert call(ctypes.byref(d), FAKE + 16, n, None) == F.FFNWB_ERR_WORKSPACE
    assert _ws("moe_grouped_matmul_fp8", _matmul(num_rows=0))[0] == 0
    assert _ws("moe_layer", _layer(num_tokens=0)) == (0, 0)
    assert _ws("moe_quant_fp8", _quant()) == (0, 0)


# ----------------------------------------------------------------------------- binding

def _quant_call(**over):
    a = dict(x=torch.zeros(4, 200))
    a.update(over)
    return F.QuantFp8Call(a.pop("x"), **a)


def _matmul_call(**over):
    a = dict(x=torch.zeros(8, 256, dtype=FP8), x_scale=torch.zeros(8, 2), w=torch.zeros(4, 96, 256, dtype=FP8),
             w_scale=torch.zeros(4, 1, 2), group_list=torch.zeros(4, 2, dtype=i64))
    a.update(over)
    return F.GroupedMatmulFp8Call(a.pop("x"), a.pop("x_scale"), a.pop("w"), a.pop("w_scale"), **a)


def _layer_call(**over):
    a = dict(x=torch.zeros(4, 256, dtype=BF16), expert_ids=torch.zeros(4, 3, dtype=i32), w13=torch.zeros(8, 192, 256, dtype=FP8),
             w2=torch.zeros(8, 256, 96, dtype=FP8), w13_scale=torch.zeros(8, 2, 2), w2_scale=torch.zeros(8, 2, 1))
    a.update(over)
    return F.LayerCall(a.pop("x"), a.pop("expert_ids"), a.pop("w13"), a.pop("w2"), **a)


def test_valid_calls_build():
    assert _quant_call().out["scale"].shape == (4, 2)
    assert _quant_call(x=torch.zeros(4, 300, dtype=BF16)[:, 3:203]).desc.x_row_stride == 600
    assert _matmul_call().out["y"].shape == (8, 96)
    c = _matmul_call(epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=FP8)
    assert c.out["y"].dtype == FP8 and c.out["y"].shape == (8, 48) and c.out["y_scale"].shape == (8, 1)
    assert _matmul_call(w=torch.zeros(96, 256, dtype=FP8), w_scale=torch.zeros(1, 2), group_list=None).desc.num_experts == 1
    assert _layer_call().out["y"].shape == (4, 256)
    _layer_call(w13=torch.zeros(8, 192, 256, dtype=BF16), w2=torch.zeros(8, 256, 96, dtype=BF16), w13_scale=None, w2_scale=None)
    _layer_call(expert_ids=torch.zeros(4, 5, dtype=i64)[:, :3], active_mask=torch.ones(4, 3, dtype=torch.bool))


@pytest.mark.parametrize("make,over", [
    *[(_quant_call, o) for o in (
        dict(x=torch.zeros(4, 200, dtype=i32)), dict(x=torch.zeros(800)), dict(x=torch.zeros(4, 400)[:, ::2]), dict(x=torch.zeros(4, 0)),
        dict(actual_rows=torch.zeros(1, dtype=i32)), dict(actual_rows=torch.zeros(2, dtype=i64)),
        dict(out={"q": torch.zeros(4, 200, dtype=torch.uint8)}), dict(out={"q": torch.zeros(4, 199, dtype=FP8)}),
        dict(out={"scale": torch.zeros(4, 1)}), dict(out={"scale": torch.zeros(4, 2, dtype=BF16)}), dict(out={"y": torch.zeros(1)}))],
    *[(_matmul_call, o) for o in (
        dict(x=torch.zeros(8, 256, dtype=torch.uint8)), dict(x=torch.zeros(8, 240, dtype=FP8)), dict(x_scale=torch.zeros(8, 3)),
        dict(x_scale=torch.zeros(8, 2, dtype=BF16)), dict(w=torch.zeros(4, 96, 256, dtype=BF16)), dict(w=torch.zeros(96, 256, dtype=FP8)),
        dict(w=torch.zeros(4, 256, 96, dtype=FP8).transpose(1, 2)), dict(w_scale=torch.zeros(4, 2, 2)), dict(w_scale=None),
        dict(group_list=torch.zeros(4, 2, dtype=i32)), dict(group_list=torch.zeros(8, dtype=i64)),
        dict(group_list=torch.zeros(4, 4, dtype=i64)[:, ::2]), dict(out_dtype=torch.int8),
        dict(out={"y": torch.zeros(8, 95, dtype=BF16)}), dict(out={"y": torch.zeros(8, 96)}), dict(out={"y_scale": torch.zeros(8, 1)}),
        dict(workspace=torch.zeros(8, dtype=torch.uint8), group_list=torch.zeros(2000, 2, dtype=i64)),
        dict(workspace=torch.zeros(1 << 16), group_list=torch.zeros(2000, 2, dtype=i64)))],
    *[(_layer_call, o) for o in (
        dict(x=torch.zeros(4, 256)), dict(x=torch.zeros(4, 512, dtype=BF16)[:, ::2]), dict(expert_ids=torch.zeros(3, 3, dtype=i32)),
        dict(expert_ids=torch.zeros(4, 3)), dict(expert_scales=torch.zeros(4, 2)), dict(active_mask=torch.ones(4)),
        dict(w13=torch.zeros(8, 191, 256, dtype=FP8)), dict(w13=torch.zeros(8, 192, 240, dtype=FP8)), dict(w2=torch.zeros(8, 256, 97, dtype=FP8)),
        dict(w2=torch.zeros(8, 256, 96, dtype=BF16)), dict(w13_scale=None), dict(w2_scale=torch.zeros(8, 1, 1)),
        dict(out={"y": torch.zeros(4, 256)}), dict(out={"x": torch.zeros(1)}), dict(workspace=torch.zeros(1, dtype=torch.uint8)))],
])
def test_binding_rejects(make, over):
    with pytest.raises(ValueError):
        make(**over)


@pytest.mark.parametrize("make,over", [
    (_matmul_call, dict(x=torch.zeros(8, 24, dtype=FP8), x_scale=torch.zeros(8, 1), w=torch.zeros(4, 96, 24, dtype=FP8),
                        w_scale=torch.zeros(4, 1, 1))),                               # K not a multiple of 16
    (_matmul_call, dict(out_dtype=FP8)),                                              # e4m3 without SwiGLU
    (_matmul_call, dict(group_list=None)),                                            # several experts, no list
    (_layer_call, dict(x=torch.zeros(65, 256, dtype=BF16), expert_ids=torch.zeros(65, 3, dtype=i32))),
])
def test_library_refusals_reach_python(make, over):
    with pytest.raises(F.FfnwbError) as e:
        make(**over)
    assert e.value.status == F.FFNWB_ERR_PARAM_INVALID
