"""dfx_gemm_fp8 when a wait runs out half-way: copies have landed and MMAs have run by then."""
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build
from test_gpu_fp8 import check, grid_case, product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfx.lib()


@pytest.mark.parametrize("tokens,rows,cols,offsets", [
    (20, 20000, 1100, None),                # one CTA a unit, more units than CTAs
    (20, 256, 4096, None),                  # K split over a cluster
    (100, 20000, 1100, None),
    (100, 256, 4096, None),
    (300, 512, 640, None),                  # pairs of 240 tokens, fewer copies than stages ...
    (700, 3000, 3000, None),                # ... and more
    (512, 300, 3000, None),                 # pairs of 256
    (130, 200, 2000, [0, 0, 50, 130]),
    (1500, 300, 2000, [0, 700, 1480]),
])
def test_a_wait_that_runs_out_half_way(tokens, rows, cols, offsets):
    x, sx, w, sw = grid_case(tokens, rows, cols, 1 if offsets is None else len(offsets) - 1, 3)
    with dfx.dfx_plan(0) as plan:
        dfx.dfx_debug_inject(dfx.DFX_INJECT_SKIP_TILE_COPY)
        try:
            product(plan, x, sx, w, sw, rows, cols, offsets, status=dfx.DFX_STATUS_TIMEOUT)
        finally:
            dfx.dfx_debug_inject(0)
        check(product(plan, x, sx, w, sw, rows, cols, offsets), x, sx, w, sw, offsets, rows, exact=True)
