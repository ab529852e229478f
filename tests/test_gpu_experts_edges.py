"""The expert-layer operators where FP32 runs out: choices that cancel."""
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build
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
