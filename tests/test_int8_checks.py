"""Host-only checks of the INT8 operators: descriptor layouts, status codes of bad arguments before
any device work, the largest sizes, and the binding's refusals."""

import ctypes

import pytest
import torch

import unpermute_ffnwb_batching_amd as F

FAKE = 0x1000
FP8, BF16, FP16, f32, i32, i64, I8 = (torch.float8_e4m3fn, torch.bfloat16, torch.float16, torch.float32, torch.int32,
                                      torch.int64, torch.int8)
DT16, DTB, DT8, DT32, DTF8 = (F.FFNWB_DT_FP16, F.FFNWB_DT_BF16, F.FFNWB_DT_INT8, F.FFNWB_DT_FP32, F.FFNWB_DT_FP8_E4M3)


def _ws(name, d):
    n = ctypes.c_size_t(0)
    return getattr(F.lib(), name + "_workspace_size")(ctypes.byref(d), ctypes.byref(n)), n.value


def _fill(d, vals, ptrs, over):
    for k, v in vals.items():
        setattr(d, k, v)
    for i, p in enumerate(ptrs):
        setattr(d, p, FAKE * (i + 1))
    for k, v in over.items():
        setattr(d, k, v)
    return d


def _quant(**over):
    return _fill(F.QuantInt8Desc(), dict(dtype=DTB, num_rows=4, hidden=256), ("x", "q", "scale"), over)


def _norm(**over):
    return _fill(F.RmsNormQuantDesc(), dict(dtype=DTB, gamma_dtype=DTB, q_dtype=DT8, epsilon=1e-6, num_rows=4, hidden=256),
                 ("x", "residual", "gamma", "residual_out", "q", "scale"), over)


def _matmul(**over):
    return _fill(F.GroupedMatmulInt8Desc(), dict(epilogue=0, out_dtype=DTB, num_rows=8, in_features=256, out_features=96,
                                                 num_experts=4, num_groups=4),
                 ("x", "x_scale", "w", "w_scale", "group_list", "y", "y_scale"), over)


MAKE = {"moe_quant_int8": _quant, "moe_rmsnorm_quant": _norm, "moe_grouped_matmul_int8": _matmul}


def test_descriptor_layouts():
    L = F.lib()
    assert L.moe_quant_int8_desc_size() == ctypes.sizeof(F.QuantInt8Desc)
    assert L.moe_rmsnorm_quant_desc_size() == ctypes.sizeof(F.RmsNormQuantDesc)
    assert L.moe_grouped_matmul_int8_desc_size() == ctypes.sizeof(F.GroupedMatmulInt8Desc)


@pytest.mark.parametrize("name", list(MAKE))
def test_null_descriptor_and_size(name):
    n = ctypes.c_size_t(0)
    assert getattr(F.lib(), name + "_workspace_size")(None, ctypes.byref(n)) == F.FFNWB_ERR_PARAM_NULLPTR
    assert getattr(F.lib(), name + "_workspace_size")(ctypes.byref(MAKE[name]()), None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert getattr(F.lib(), name)(None, None, 0, None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert _ws(name, MAKE[name]())[0] == F.FFNWB_OK


def test_plan_refuses_what_the_call_refuses():
    info = F.GroupedMatmulInt8PlanInfo()
    plan = F.lib().moe_grouped_matmul_int8_plan
    assert plan(None, ctypes.byref(info)) == F.FFNWB_ERR_PARAM_NULLPTR
    assert plan(ctypes.byref(_matmul()), None) == F.FFNWB_ERR_PARAM_NULLPTR
    assert plan(ctypes.byref(_matmul(num_experts=0)), ctypes.byref(info)) == F.FFNWB_ERR_PARAM_INVALID
    with pytest.raises(F.FfnwbError):
        F.moe_grouped_matmul_int8_plan(_matmul(in_features=24))


@pytest.mark.parametrize("name,field", [("moe_quant_int8", p) for p in ("x", "q", "scale")] +
                         [("moe_rmsnorm_quant", p) for p in ("x", "gamma", "q", "scale", "residual", "residual_out")] +
                         [("moe_grouped_matmul_int8", p) for p in ("x", "x_scale", "w", "w_scale", "y")])
def test_required_pointers(name, field):
    assert _ws(name, MAKE[name](**{field: None}))[0] == F.FFNWB_ERR_PARAM_NULLPTR


def test_optional_pointers():
    assert _ws("moe_quant_int8", _quant(actual_rows=FAKE)) == (0, 0)
    assert _ws("moe_rmsnorm_quant", _norm(residual=None, residual_out=None)) == (0, 0)
    assert _ws("moe_rmsnorm_quant", _norm(y=FAKE, actual_rows=FAKE)) == (0, 0)
    assert _ws("moe_rmsnorm_quant", _norm(residual_out=2 * FAKE)) == (0, 0)               # in place
    assert _ws("moe_rmsnorm_quant", _norm(residual_out=2 * FAKE, residual_row_stride=1024, residual_out_row_stride=1024)) == (0, 0)
    assert _ws("moe_rmsnorm_quant", _norm(gamma_dtype=DT32)) == (0, 0)
    assert _ws("moe_grouped_matmul_int8", _matmul(group_list=None, num_groups=0, num_experts=1))[0] == 0
    assert _ws("moe_grouped_matmul_int8", _matmul(y_scale=None))[0] == 0
    assert _ws("moe_grouped_matmul_int8", _matmul(out_dtype=DT8, epilogue=1))[0] == 0
    assert _ws("moe_grouped_matmul_int8", _matmul(out_dtype=DT8, epilogue=1, y_scale=None))[0] == F.FFNWB_ERR_PARAM_NULLPTR


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("name,over", [
    *[("moe_quant_int8", o) for o in (
        dict(dtype=DT8), dict(dtype=DTF8), dict(dtype=-1), dict(reserved0=1), dict(num_rows=-1), dict(num_rows=(1 << 24) + 1),
        dict(num_rows=1 << 62), dict(hidden=0), dict(hidden=-8), dict(hidden=(1 << 20) + 1), dict(x_row_stride=511), dict(x_row_stride=510),
        dict(x_row_stride=513), dict(x_row_stride=-512), dict(q_row_stride=255), dict(q_row_stride=-256), dict(scale_row_stride=-1),
        dict(x=FAKE + 1), dict(dtype=DT32, x=FAKE + 2), dict(scale=FAKE + 2), dict(x_row_stride=1 << 33), dict(q_row_stride=1 << 33),
        dict(scale_row_stride=1 << 33), dict(x_row_stride=1 << 62))],
    *[("moe_rmsnorm_quant", o) for o in (
        dict(dtype=DT8), dict(dtype=DT32), dict(gamma_dtype=DT16), dict(gamma_dtype=DT8), dict(q_dtype=DTB), dict(q_dtype=-1),
        dict(epsilon=0.0), dict(epsilon=-1e-6), dict(epsilon=NAN), dict(epsilon=INF), dict(epsilon=1e-40), dict(num_rows=-1),
        dict(num_rows=(1 << 24) + 1), dict(hidden=0), dict(hidden=(1 << 20) + 1),
        *[{s: v} for s in ("x_row_stride", "residual_row_stride", "residual_out_row_stride", "y_row_stride") for v in (510, 513, -512, 1 << 33)],
        dict(q_row_stride=255), dict(q_row_stride=1 << 33), dict(scale_row_stride=-1), dict(q_dtype=DTF8, scale_row_stride=1),
        *[{p: FAKE + 1} for p in ("x", "residual", "gamma", "residual_out", "y")], dict(gamma_dtype=DT32, gamma=FAKE + 2), dict(scale=FAKE + 1),
        dict(residual_out=2 * FAKE, residual_out_row_stride=1024))],
    *[("moe_grouped_matmul_int8", o) for o in (
        dict(epilogue=2), dict(epilogue=-1), dict(epilogue=256), dict(epilogue=257), dict(out_dtype=DT8), dict(out_dtype=DTF8),
        dict(epilogue=1, out_dtype=DTF8), dict(out_dtype=7), dict(num_rows=-1), dict(num_rows=(1 << 24) + 1), dict(in_features=0),
        dict(in_features=24), dict(in_features=131072), dict(out_features=0), dict(out_features=(1 << 18) + 1),
        dict(epilogue=1, out_features=48), dict(num_experts=0), dict(num_experts=8193), dict(num_groups=0), dict(num_groups=8193),
        dict(group_list=None), dict(group_list=None, num_groups=0), dict(x_row_stride=240), dict(x_row_stride=264),
        dict(x_scale_stride=-1), dict(x_row_stride=1 << 40), dict(x_scale_stride=1 << 40), dict(y_row_stride=1 << 40),
        dict(y_row_stride=190), dict(y_row_stride=193), dict(epilogue=1, out_dtype=DT8, y_scale_stride=-1),
        dict(epilogue=1, out_dtype=DT8, y_scale=FAKE + 2), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 1), dict(x_scale=FAKE + 2),
        dict(w_scale=FAKE + 1), dict(num_rows=1 << 24, out_features=1 << 18, group_list=None, num_groups=0, num_experts=1))],
])
def test_invalid_parameters(name, over):
    assert _ws(name, MAKE[name](**over))[0] == F.FFNWB_ERR_PARAM_INVALID
    assert getattr(F.lib(), name)(ctypes.byref(MAKE[name](**over)), None, 0, None) == F.FFNWB_ERR_PARAM_INVALID


@pytest.mark.parametrize("name,most", [
    ("moe_quant_int8", dict(num_rows=1 << 24, hidden=1 << 20, x_row_stride=1 << 32, q_row_stride=1 << 32, scale_row_stride=1 << 32)),
    ("moe_rmsnorm_quant", dict(num_rows=1 << 24, hidden=1 << 20, x_row_stride=1 << 32, q_row_stride=1 << 32, epsilon=2.0 ** -126)),
    ("moe_grouped_matmul_int8", dict(in_features=131056, x_row_stride=1 << 32, x_scale_stride=1 << 32, y_row_stride=1 << 32)),
    ("moe_grouped_matmul_int8", dict(num_rows=1 << 24, out_features=(1 << 14) - 256, num_groups=1)),
])
def test_largest_sizes(name, most):
    assert _ws(name, MAKE[name](**most))[0] == F.FFNWB_OK


def test_a_call_whose_widest_tiles_fit_is_never_refused():
    # (ceil(R / 64) + num_groups) * max(ceil(F / 16), 16) up to the workgroups of a launch, whatever the times expected
    for groups in (1, 300, 8192):
        for f in (16, 512, 1 << 12, 1 << 17):
            rows = min(((1 << 22) - 8) // max(f // 16, 16) - groups, 1 << 18) * 64
            if rows <= 0:
                continue
            for over in (dict(out_features=f), dict(out_features=f, out_dtype=DT32), dict(out_features=2 * f, epilogue=1),
                         dict(out_features=2 * f, epilogue=1, out_dtype=DT8)):
                for stride in (0, 1 << 30):
                    d = _matmul(num_rows=rows, num_groups=groups, num_experts=64, in_features=128, x_row_stride=stride, **over)
                    assert _ws("moe_grouped_matmul_int8", d)[0] == F.FFNWB_OK, (groups, f, over, stride)


def test_workspace_is_checked_before_any_device_work():
    for over in (dict(num_groups=2000), dict(num_rows=520, in_features=8192, out_features=1024, epilogue=1, out_dtype=DT8)):
        d = _matmul(**over)
        st, n = _ws("moe_grouped_matmul_int8", d)
        assert st == 0 and n > 0
        call = F.lib().moe_grouped_matmul_int8
        assert call(ctypes.byref(d), None, n, None) == F.FFNWB_ERR_WORKSPACE
        assert call(ctypes.byref(d), FAKE, n - 1, None) == F.FFNWB_ERR_WORKSPACE
        assert call(ctypes.byref(d), FAKE + 16, n, None) == F.FFNWB_ERR_WORKSPACE
    assert _ws("moe_grouped_matmul_int8", _matmul(num_rows=0))[0] == 0


# ----------------------------------------------------------------------------- binding

def _quant_call(**over):
    a = dict(x=torch.zeros(4, 200))
    a.update(over)
    return F.QuantInt8Call(a.pop("x"), **a)


def _norm_call(**over):
    a = dict(x=torch.zeros(4, 200, dtype=BF16), gamma=torch.zeros(200, dtype=BF16), residual=torch.zeros(4, 200, dtype=BF16))
    a.update(over)
    return F.RmsNormQuantCall(a.pop("x"), a.pop("gamma"), **a)


def _matmul_call(**over):
    a = dict(x=torch.zeros(8, 256, dtype=I8), x_scale=torch.zeros(8), w=torch.zeros(4, 96, 256, dtype=I8),
             w_scale=torch.zeros(4, 96), group_list=torch.zeros(4, 2, dtype=i64))
    a.update(over)
    return F.GroupedMatmulInt8Call(a.pop("x"), a.pop("x_scale"), a.pop("w"), a.pop("w_scale"), **a)


def test_calls_on_the_cpu_do_not_run():
    for make in (_quant_call, _norm_call, _matmul_call):
        with pytest.raises(ValueError, match="GPU"):
            make().run()


def test_valid_calls_build():
    assert _quant_call().out["scale"].shape == (4,)
    c = _quant_call(x=torch.zeros(4, 300, dtype=BF16)[:, 3:203])
    assert c.desc.x_row_stride == 600 and c.out["q"].dtype == I8
    packed = torch.zeros(4, 204, dtype=I8)
    c = _quant_call(out={"q": packed[:, :200], "scale": packed.view(f32)[:, 50]})
    assert (c.desc.q_row_stride, c.desc.scale_row_stride) == (204, 51)
    c = _norm_call()
    assert set(c.out) == {"q", "scale", "residual_out"} and c.out["scale"].shape == (4,)
    c = _norm_call(residual=None, with_y=True, q_dtype=FP8, gamma=torch.zeros(200))
    assert set(c.out) == {"q", "scale", "y"} and c.out["scale"].shape == (4, 2) and c.desc.gamma_dtype == DT32
    y = torch.zeros(4, 200, dtype=BF16)
    assert _norm_call(out={"y": y}).out["y"] is y
    res = torch.zeros(4, 256, dtype=BF16)[:, :200]
    c = _norm_call(residual=res, out={"residual_out": res})
    assert c.desc.residual == c.desc.residual_out and c.desc.residual_out_row_stride == 512
    assert _matmul_call().out["y"].shape == (8, 96)
    c = _matmul_call(epilogue=F.FFNWB_EPI_SWIGLU, out_dtype=I8)
    assert c.out["y"].dtype == I8 and c.out["y"].shape == (8, 48) and c.out["y_scale"].shape == (8,)
    assert _matmul_call(w=torch.zeros(96, 256, dtype=I8), w_scale=torch.zeros(96), group_list=None).desc.num_experts == 1
    assert _matmul_call(x_scale=torch.zeros(8, 5)[:, 2]).desc.x_scale_stride == 5


@pytest.mark.parametrize("make,over", [
    *[(_quant_call, o) for o in (
        dict(x=torch.zeros(4, 200, dtype=i32)), dict(x=torch.zeros(800)), dict(x=torch.zeros(4, 400)[:, ::2]), dict(x=torch.zeros(4, 0)),
        dict(x=None), dict(actual_rows=torch.zeros(1, dtype=i32)), dict(actual_rows=torch.zeros(2, dtype=i64)),
        dict(out={"q": torch.zeros(4, 200, dtype=torch.uint8)}), dict(out={"q": torch.zeros(4, 199, dtype=I8)}),
        dict(out={"scale": torch.zeros(4, 1)}), dict(out={"scale": torch.zeros(4, dtype=BF16)}), dict(out={"scale": torch.zeros(1).expand(4)}),
        dict(out={"y": torch.zeros(1)}))],
    *[(_norm_call, o) for o in (
        dict(x=torch.zeros(4, 200, dtype=i32)), dict(x=torch.zeros(4, 0, dtype=BF16)), dict(gamma=torch.zeros(200, dtype=FP16)),
        dict(gamma=torch.zeros(199, dtype=BF16)), dict(gamma=torch.zeros(1, 200, dtype=BF16)), dict(gamma=torch.zeros(400, dtype=BF16)[::2]),
        dict(gamma=None), dict(residual=torch.zeros(4, 200)), dict(residual=torch.zeros(3, 200, dtype=BF16)), dict(q_dtype=torch.uint8),
        dict(q_dtype=BF16), dict(actual_rows=torch.zeros(1)), dict(out={"q": torch.zeros(4, 200, dtype=FP8)}),
        dict(out={"y": torch.zeros(4, 200)}), dict(out={"residual_out": torch.zeros(4, 201, dtype=BF16)}),
        dict(residual=None, out={"residual_out": torch.zeros(4, 200, dtype=BF16)}), dict(out={"scale": torch.zeros(4, 2)}),
        dict(q_dtype=FP8, out={"scale": torch.zeros(4)}))],
    *[(_matmul_call, o) for o in (
        dict(x=torch.zeros(8, 256, dtype=torch.uint8)), dict(x=torch.zeros(8, 240, dtype=I8)), dict(x_scale=torch.zeros(8, 1)),
        dict(x_scale=torch.zeros(7)), dict(x_scale=torch.zeros(8, dtype=BF16)), dict(x_scale=torch.zeros(1).expand(8)),
        dict(w=torch.zeros(4, 96, 256, dtype=BF16)), dict(w=torch.zeros(96, 256, dtype=I8)),
        dict(w=torch.zeros(4, 256, 96, dtype=I8).transpose(1, 2)), dict(w_scale=torch.zeros(4, 95)), dict(w_scale=None), dict(w_scale=torch.zeros(96)),
        dict(group_list=torch.zeros(4, 2, dtype=i32)), dict(group_list=torch.zeros(8, dtype=i64)),
        dict(group_list=torch.zeros(4, 4, dtype=i64)[:, ::2]), dict(out_dtype=FP8),
        dict(out={"y": torch.zeros(8, 95, dtype=BF16)}), dict(out={"y": torch.zeros(8, 96)}), dict(out={"y_scale": torch.zeros(8)}),
        dict(workspace=torch.zeros(8, dtype=torch.uint8), group_list=torch.zeros(2000, 2, dtype=i64)),
        dict(workspace=torch.zeros(1 << 16), group_list=torch.zeros(2000, 2, dtype=i64)))],
])
def test_binding_rejects(make, over):
    with pytest.raises(ValueError):
        make(**over)


@pytest.mark.parametrize("make,over", [
    (_matmul_call, dict(x=torch.zeros(8, 24, dtype=I8), w=torch.zeros(4, 96, 24, dtype=I8))),     # K not a multiple of 16
    (_matmul_call, dict(out_dtype=I8)),                                                           # INT8 without SwiGLU
    (_matmul_call, dict(group_list=None)),                                                        # several experts, no list
    (_matmul_call, dict(epilogue=F.FFNWB_EPI_EXACT)),                                             # of the e4m3 products
    (_norm_call, dict(eps=0.0)),
])
def test_library_refusals_reach_python(make, over):
    with pytest.raises(F.FfnwbError) as e:
        make(**over)
    assert e.value.status == F.FFNWB_ERR_PARAM_INVALID
