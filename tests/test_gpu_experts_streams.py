"""The helpers of the expert layers on a stream that is not their tensors'."""
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfx.lib()


def rand(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to("cuda", dtype)


def clones(values):
    return [dfx.Fp8(v.values.clone(), v.scales.clone(), v.cols, v.block_rows) if isinstance(v, dfx.Fp8) else v.clone()
            for v in values]


def operands(helper):
    """A call of the helper with fresh tensors of megabytes each, whose memory the allocator hands out whole."""
    if helper == "route":
        return [rand(8192, 256), 0.1 * rand(256 * 4096)[:256]], lambda x, b, **kw: dfx.route(x, 8, "sigmoid", b, **kw)
    if helper == "quantize_fp8":
        index = torch.arange(2000, -1, -1, dtype=torch.int32, device="cuda").repeat(1000)[:4000]
        return [rand(4000, 1000), index], lambda x, i, **kw: dfx.quantize_fp8(x, index=i, **kw)
    if helper == "gemm_fp8":
        x, w = dfx.quantize_fp8(rand(2000, 2048)), dfx.quantize_fp8(rand(2, 1024, 2048, seed=1), block_rows=128)
        offsets = torch.tensor([0, 900, 2000], dtype=torch.int32, device="cuda")
        return [x, w, offsets], dfx.gemm_fp8
    if helper == "combine":
        slots = torch.randperm(8000).to("cuda", torch.int32).reshape(4000, 2)
        return [rand(8000, 512), slots, rand(4000, 2)], dfx.combine
    w_in, w_out = (dfx.quantize_fp8(rand(16, 512, cols, seed=cols), block_rows=128) for cols in (512, 256))
    return [rand(4000, 512), rand(4000, 16), w_in, w_out], lambda *a, **kw: dfx.experts_fp8(*a, 2, **kw)



@pytest.mark.parametrize("helper", ["route", "quantize_fp8", "gemm_fp8", "combine", "experts_fp8"])
def test_tensors_that_are_dropped_behind_the_call(helper):
    """Memory of tensors that nobody holds any more is not handed out while the stream has yet to read them."""
    kept, call = operands(helper)
    want = call(*kept)
    stream = torch.cuda.Stream()
    with dfx.dfx_plan(0) as plan:
        call(*kept, plan=plan, stream=stream)  # loads the kernels, and the stream's memory
        given = clones(kept)
        sizes = [t.numel() * t.element_size() for g in given for t in (g[:2] if isinstance(g, dfx.Fp8) else (g,))]
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            torch.cuda._sleep(200_000_000)  # a tenth of a second
        got = call(*given, plan=plan, stream=stream)
        del given
        over = [torch.full((n,), 1, dtype=torch.uint8, device="cuda") for n in sizes]  # others' memory, written at once
        torch.cuda.synchronize()
        assert dfx.dfx_device_status(plan) == 0
    for g, w in zip(*((v,) if torch.is_tensor(v) else v[:2] if isinstance(v, dfx.Fp8) else v for v in (got, want))):
        if g.dtype == torch.uint8:  # an Fp8's rows: the bytes behind a row are nobody's
            cols = got.cols if g.shape == got.values.shape else -(-got.cols // 128)
            g, w = g[..., :cols], w[..., :cols]
        assert torch.equal(g, w)
    del over
