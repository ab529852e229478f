"""Argument checks of the expert-layer calls (dfx_route, dfx_quantize_fp8, dfx_gemm_fp8,
dfx_combine) that need no GPU.

The plan is a block of zeros: the calls look at their other arguments first, and without a
device a call with nothing to refuse ends with DFX_ERR_CUDA before it touches the plan."""
import ctypes

import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes plans and pointers that are not the device's")

P = 4096  # an aligned address that is never followed
ODD = P + 8
PLAN = ctypes.create_string_buffer(4096)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    dfx.lib()


def call(name, defaults, **changes):
    args = {**defaults, **changes}
    if "params" in args and args["params"] is not None:
        args["params"] = ctypes.byref(args["params"])
    return getattr(dfx.lib(), name)(*args.values(), None)


def route_params(**kw):
    return dfx.dfx_route_params(**{**dict(score=dfx.DFX_SCORE_SOFTMAX, topk=2), **kw})


ROUTE = dict(plan=ctypes.addressof(PLAN), logits=P, type=dfx.DFX_F32, ld=16, tokens=100, experts=16, bias=None,
             params=route_params(), ids=P, weights=P, offsets=P, rows=P, slots=P, workspace=P, workspace_bytes=1 << 20)
QUANTIZE = dict(plan=ctypes.addressof(PLAN), x=P, type=dfx.DFX_BF16, ld=256, x_rows=10, index=None, rows=10, cols=256,
                block_rows=1, flags=0, q=P, ld_q=256, scales=P, ld_scales=4)
GEMM = dict(plan=ctypes.addressof(PLAN), x=P, ld_x=256, sx=P, ld_sx=4, tokens=10, w=P, ld_w=256, sw=P, ld_sw=4,
            rows=128, cols=256, experts=1, offsets=None, y=P, y_type=dfx.DFX_BF16, ld_y=128)
COMBINE = dict(plan=ctypes.addressof(PLAN), z=P, z_type=dfx.DFX_BF16, ld_z=64, z_rows=20, cols=64, slots=P, weights=P,
               tokens=10, topk=2, y=P, y_type=dfx.DFX_F32, ld_y=64)

ARG, CAPACITY, TOO_LARGE, CUDA, UNSUPPORTED = (dfx.DFX_ERR_ARG, dfx.DFX_ERR_CAPACITY, dfx.DFX_ERR_TOO_LARGE,
                                               dfx.DFX_ERR_CUDA, dfx.DFX_ERR_UNSUPPORTED)


@pytest.mark.parametrize("name,defaults", [("dfx_route", ROUTE), ("dfx_quantize_fp8", QUANTIZE),
                                           ("dfx_gemm_fp8", GEMM), ("dfx_combine", COMBINE)])
def test_a_sound_call_is_only_stopped_by_the_missing_device(name, defaults):
    assert call(name, defaults) == CUDA
    assert call(name, defaults, plan=None) == ARG


@pytest.mark.parametrize("changes,code", [
    (dict(params=None), ARG),
    (dict(params=route_params(topk=0)), ARG),
    (dict(params=route_params(topk=17)), ARG),
    (dict(params=route_params(score=2)), ARG),
    (dict(params=route_params(renormalize=2)), ARG),
    (dict(params=route_params(scale=float("nan"))), ARG),
    (dict(params=route_params(groups=3, top_groups=1)), ARG),       # 16 experts in 3 groups
    (dict(params=route_params(groups=4, top_groups=0)), ARG),
    (dict(params=route_params(groups=4, top_groups=5)), ARG),
    (dict(params=route_params(groups=4, top_groups=1, group_best=3)), ARG),
    (dict(params=route_params(groups=8, top_groups=1, topk=3)), ARG),  # 3 of 2 experts
    (dict(params=route_params(topk=33), experts=64, ld=64), UNSUPPORTED),
    (dict(params=route_params(groups=64, top_groups=2), experts=128, ld=128), UNSUPPORTED),
    (dict(experts=513, ld=513), UNSUPPORTED),
    (dict(experts=0), ARG),
    (dict(type=2), ARG),
    (dict(ld=15), ARG),
    (dict(tokens=1 << 30), TOO_LARGE),
    (dict(logits=None), ARG),
    (dict(logits=ODD), ARG),
    (dict(bias=ODD), ARG),
    (dict(ids=None), ARG),
    (dict(weights=ODD), ARG),
    (dict(offsets=None), ARG),                # lists without their offsets
    (dict(rows=None), ARG),
    (dict(slots=ODD), ARG),
    (dict(workspace=None), ARG),
    (dict(workspace_bytes=15), CAPACITY),
])
def test_route_refusals(changes, code):
    assert call("dfx_route", ROUTE, **changes) == code


def test_route_workspace():
    size = lambda t, e, **kw: dfx.dfx_route_workspace(t, e, route_params(**kw))  # noqa: E731
    assert size(0, 16) % 16 == 0 and size(1, 512) % 16 == 0
    assert size(100_000, 256) >= 256 * 4
    with pytest.raises(dfx.DfxError) as e:
        size(1, 513)
    assert e.value.code == UNSUPPORTED
    with pytest.raises(dfx.DfxError) as e:
        size(1 << 31, 16)
    assert e.value.code == TOO_LARGE
    assert dfx.lib().dfx_route_workspace(1, 16, ctypes.byref(route_params()), None) == ARG


@pytest.mark.parametrize("changes,code", [
    (dict(type=2), ARG),
    (dict(flags=2), ARG),
    (dict(block_rows=64), ARG),
    (dict(block_rows=128, index=P), UNSUPPORTED),
    (dict(block_rows=128, flags=dfx.DFX_QUANT_SWIGLU, ld=512), UNSUPPORTED),
    (dict(flags=dfx.DFX_QUANT_SWIGLU), ARG),  # rows of 256 hold no 256 gates and values
    (dict(cols=0), ARG),
    (dict(rows=11), ARG),                     # more rows than x has, without an index
    (dict(ld=255), ARG),
    (dict(ld_q=240), ARG),
    (dict(ld_q=264), ARG),
    (dict(ld_scales=3), ARG),
    (dict(cols=640, ld=640, ld_q=640), ARG),  # five blocks in four bytes
    (dict(x=ODD), ARG),
    (dict(x=None), ARG),
    (dict(q=None), ARG),
    (dict(scales=ODD), ARG),
    (dict(index=ODD), ARG),
    (dict(rows=1 << 31, x_rows=1 << 31), ARG),
])
def test_quantize_refusals(changes, code):
    assert call("dfx_quantize_fp8", QUANTIZE, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(y_type=2), ARG),
    (dict(experts=0), ARG),
    (dict(experts=2), ARG),                   # several matrices without offsets
    (dict(experts=1025, offsets=P), UNSUPPORTED),
    (dict(cols=0), ARG),
    (dict(ld_x=240), ARG),
    (dict(ld_x=264), ARG),
    (dict(ld_w=128), ARG),
    (dict(ld_sx=3), ARG),
    (dict(ld_sw=1), ARG),
    (dict(ld_y=127), ARG),
    (dict(tokens=1 << 31), TOO_LARGE),
    (dict(rows=1 << 22, experts=512, offsets=P, ld_y=1 << 22), TOO_LARGE),
    (dict(x=ODD), ARG),
    (dict(sx=ODD), ARG),
    (dict(w=ODD), ARG),
    (dict(sw=ODD), ARG),
    (dict(offsets=ODD), ARG),
    (dict(y=ODD), ARG),
    (dict(y=None), ARG),
    (dict(w=None), ARG),
])
def test_gemm_refusals(changes, code):
    assert call("dfx_gemm_fp8", GEMM, **changes) == code


@pytest.mark.parametrize("changes,code", [
    (dict(z_type=2), ARG),
    (dict(y_type=2), ARG),
    (dict(cols=0), ARG),
    (dict(topk=0), ARG),
    (dict(topk=33), UNSUPPORTED),
    (dict(ld_z=63), ARG),
    (dict(ld_y=63), ARG),
    (dict(tokens=1 << 31), TOO_LARGE),
    (dict(z=ODD), ARG),
    (dict(z=None), ARG),
    (dict(slots=None), ARG),
    (dict(weights=ODD), ARG),
    (dict(y=ODD), ARG),
])
def test_combine_refusals(changes, code):
    assert call("dfx_combine", COMBINE, **changes) == code


def test_route_params_mirror_the_header():
    from test_library import header_struct_fields

    kinds = {"uint32_t": ctypes.c_uint32, "float": ctypes.c_float}
    declared = header_struct_fields("dfx_route_params")
    assert [(n, kinds[t]) for t, n in declared] == dfx.dfx_route_params._fields_
