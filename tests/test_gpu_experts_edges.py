"""The expert-layer operators where FP32 runs out: choices that cancel, products beyond its range,
gates so low that their exponential is."""
import numpy as np
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build
from test_gpu_fp8 import quantize, reference, same_bytes, to_e4m3
from test_gpu_route import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfx.lib()


@pytest.fixture(scope="module")
def plan():
    with dfx.dfx_plan(0) as p:
        yield p


# ---------------------------------------------------------------- groups whose best two choices cancel

@pytest.mark.parametrize("experts", [96, 256, 512])
@pytest.mark.parametrize("size", [32.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_whose_choices_cancel(plan, experts, size, sigmoid):
    """A large bias beside a large negative one: the sum of a group's best two is small, its rounding is not."""
    g = torch.Generator().manual_seed(experts + int(size))
    x = 1.5 * torch.randn(1000, experts, generator=g)
    bias = torch.full((experts,), -size)
    bias[:: experts // 32] = size
    check(plan, x, 4, sigmoid=sigmoid, bias=bias, groups=32, top_groups=4, best=2, renorm=True)


def test_one_group_of_large_choices(plan):
    """Only one group's choices are large, and it is not among the best."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(300, 256, generator=g)
    bias = 0.1 * torch.randn(256, generator=g)
    bias[64:96] = -1e9
    check(plan, x, 8, sigmoid=True, bias=bias, groups=8, top_groups=4, best=2, renorm=True)
    bias[64:96] = torch.finfo(torch.float32).min
    check(plan, x, 8, sigmoid=True, bias=bias, groups=8, top_groups=7, best=2)


def test_near_group_scores_keep_their_order(plan):
    """Groups whose scores are nearer than FP32's rounding come in the order of their exact sums."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(400, 64, generator=g)
    x[:] = x[:1]
    s = 1 / (1 + torch.exp(-x[0].double()))
    check(plan, x, 6, sigmoid=True, bias=(1.0 - s).float(), groups=16, top_groups=5, best=2)
    check(plan, x, 6, sigmoid=True, bias=(1.0 - s).float(), groups=16, top_groups=5, best=1)


# ---------------------------------------------------------------- SwiGLU at the ends of FP32's range

@pytest.mark.parametrize("value", [10.0, 3e38])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_product_beyond_fp32_has_no_part_in_the_scale(plan, value, dtype):
    """The block's largest finite product stands on the border (1.75 * 2^5), where the scale is settled in 64 bits."""
    x = torch.zeros(3, 256)
    x[:, 5], x[:, 128 + 5] = 56.0, 1.0
    x[:, 9], x[:, 128 + 9] = 40.0, 0.5
    x[0, 77], x[0, 128 + 77] = 2e38, value
    x[1, 3], x[1, 128 + 3] = 2e38, -value
    q, s = quantize(plan, x.to(dtype).cuda(), 3, 128, flags=dfx.DFX_QUANT_SWIGLU)
    v = np.zeros((3, 128))
    v[:, 5], v[:, 9] = 56.0, 20.0
    v[0, 77] = v[1, 3] = np.nan
    ref_s, ref_q = reference(v, 1)
    assert np.array_equal(s, ref_s)
    assert same_bytes(q, to_e4m3(ref_q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_product_beyond_fp32_beside_the_highest_border(plan, dtype):
    """The largest product that FP32 holds is 1.75 * 2^127, the one beside it just past FP32's largest value."""
    x = torch.zeros(2, 256)
    x[:, 5], x[:, 128 + 5] = 1.75 * 2.0 ** 100, 2.0 ** 27
    x[0, 77], x[0, 128 + 77] = 2e38, 1.75
    q, s = quantize(plan, x.to(dtype).cuda(), 2, 128, flags=dfx.DFX_QUANT_SWIGLU)
    v = np.zeros((2, 128))
    v[:, 5], v[0, 77] = 1.75 * 2.0 ** 127, np.nan
    ref_s, ref_q = reference(v, 1)
    assert np.array_equal(s, ref_s)
    assert same_bytes(q, to_e4m3(ref_q))


@pytest.mark.parametrize("cols", [1, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_swiglu_of_low_gates(plan, cols, dtype):
    """Gates whose exp(-gate) is beyond FP32, beside values large enough for a product that is not."""
    gates = torch.linspace(-200.0, -70.0, 131)
    factors = torch.tensor([1.0, 1e6, -1e10, 1e20, -1e30, 1e38, 3e38])
    g, u = gates.repeat_interleave(7).to(dtype), factors.repeat(131).to(dtype)
    x = torch.cat([g[:, None].repeat(1, cols), u[:, None].repeat(1, cols)], 1)
    q, s = quantize(plan, x.cuda(), x.shape[0], cols, flags=dfx.DFX_QUANT_SWIGLU)
    gd, ud = x[:, :cols].double().numpy(), x[:, cols:].double().numpy()
    v = gd / (1 + np.exp(-gd)) * ud
    ref_s, ref_q = reference(v, 1)
    normal = np.abs(v[:, 0]) >= 2.0 ** -126  # FP32 holds it in full
    assert 0 < normal.sum() < normal.size
    assert np.array_equal(s[normal], ref_s[normal])
    got = torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy()
    # half a step of e4m3 (2^-4 of the value, 2^-10 among its subnormals), FP32's rounding of the product (2^-24)
    assert np.all(np.abs(got - ref_q)[normal] <= (np.abs(ref_q) * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10)[normal])
    # below: FP32 rounds the product to a multiple of 2^-149
    rest = ~normal
    held = got * np.ldexp(1.0, s[:, :1].astype(np.int64) - 127)
    assert np.all(np.abs(held - v)[rest] <= (np.abs(v) * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -137)[rest])
