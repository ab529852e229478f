"""dfx_quantize_fp8 and dfx_gemm_fp8 against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build

pytestmark = pytest.mark.gpu

FILL = 0x5A  # what buffers hold before a call


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfx.lib()


@pytest.fixture(scope="module")
def plan():
    with dfx.dfx_plan(0) as p:
        yield p


def up(x, to):
    return -(-x // to) * to


def reference(v, block_rows):
    """(scale bytes, exact quotients) of float64 values v [rows, cols]."""
    rows, cols = v.shape
    finite = np.where(np.isfinite(v), np.abs(v), 0.0)
    full = np.zeros((up(rows, block_rows), up(cols, 128)))
    full[:rows, :cols] = finite
    peak = full.reshape(full.shape[0] // block_rows, block_rows, -1, 128).max(axis=(1, 3))
    mantissa, exponent = np.frexp(peak)  # 448 = 0.875 * 2^9
    e = np.where(peak == 0, 0, np.clip(exponent - 9 + (mantissa > 0.875), -127, 127)).astype(np.int64)
    s = np.ldexp(1.0, e).repeat(block_rows, 0)[:rows].repeat(128, 1)[:, :cols]
    return (e + 127).astype(np.uint8), v / s


def to_e4m3(q):
    """Exact quotients (float64, exact in FP32) rounded once to e4m3 bytes; NaN where not finite."""
    q = np.where(np.isfinite(q), q, np.nan).astype(np.float32)
    return torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def quantize(plan, x, rows, cols, block_rows=1, flags=0, index=None, ld=None, x_rows=None, status=0):
    q = torch.full((rows, up(cols, 16)), FILL, dtype=torch.uint8, device="cuda")
    blocks = -(-cols // 128)
    s = torch.full((-(-rows // block_rows), up(blocks, 4)), FILL, dtype=torch.uint8, device="cuda")
    dfx.dfx_quantize_fp8(plan, x, dfx.DFX_BF16 if x.dtype == torch.bfloat16 else dfx.DFX_F32, ld or x.shape[1],
                         x.shape[0] if x_rows is None else x_rows, index, rows, cols, block_rows, flags, q, q.shape[1],
                         s, s.shape[1])
    assert dfx.dfx_device_status(plan) == status
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.all(q[:, cols:] == FILL) and np.all(s[:, blocks:] == FILL), "bytes behind a row were written"
    return q[:, :cols], s[:, :blocks]


def same_bytes(a, b):
    """Equal e4m3 bytes, every NaN the same."""
    nan_a, nan_b = (a & 0x7F) == 0x7F, (b & 0x7F) == 0x7F
    return np.array_equal(nan_a, nan_b) and np.array_equal(a[~nan_a], b[~nan_b])


def values(rows, cols, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, cols, generator=g) * torch.exp2(spread * torch.randn(rows, -(-cols // 128), generator=g)
                                                          ).repeat_interleave(128, 1)[:, :cols]
    return v.to(dtype)


SIZES = [(1, 1), (1, 128), (3, 127), (5, 129), (16, 4096), (130, 1000), (7, 1032), (257, 2056), (129, 8)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_matches_the_definition(plan, rows, cols, dtype, block_rows):
    x = values(rows, cols, dtype, rows + cols)
    q, s = quantize(plan, x.cuda(), rows, cols, block_rows)
    ref_s, ref_q = reference(x.double().numpy(), block_rows)
    assert np.array_equal(s, ref_s)
    assert same_bytes(q, to_e4m3(ref_q))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_special_values(plan, block_rows, dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = values(256, 1024, dtype, 3)
    x[0, 0], x[0, 1], x[1, 130] = math.inf, -math.inf, math.nan
    x[2:4, :128] = 0.0
    x[128:, 256:384] = 0.0
    x[128:, 384:512] = -0.0
    x[:128, 512:640] = math.nan                      # nothing finite: scale 1
    x[:128, 640:768] = tiny * torch.linspace(-1, 1, 128).to(dtype)  # subnormal values: the smallest scale
    x[:128, 768:896] = big * torch.linspace(-1, 1, 128).to(dtype)
    x[5, 896] = 448.0 * 2 ** 5                       # on the border and just past it
    x[6, 896] = torch.nextafter(torch.tensor(448.0 * 2 ** 5, dtype=dtype), torch.tensor(math.inf, dtype=dtype))
    q, s = quantize(plan, x.cuda(), 256, 1024, block_rows)
    ref_s, ref_q = reference(x.double().numpy(), block_rows)
    assert np.array_equal(s, ref_s)
    assert same_bytes(q, to_e4m3(ref_q))


@pytest.mark.parametrize("block_rows,ld", [(1, 264), (1, 263), (128, 264), (128, 263)])
def test_quantize_strided_rows(plan, block_rows, ld):
    x = values(200, ld, torch.bfloat16, 8)
    q, s = quantize(plan, x.cuda(), 200, 256, block_rows, ld=ld)
    ref_s, ref_q = reference(x[:, :256].double().numpy(), block_rows)
    assert np.array_equal(s, ref_s) and same_bytes(q, to_e4m3(ref_q))


@pytest.mark.parametrize("cols", [256, 250])
def test_quantize_gathers_rows(plan, cols):
    x = values(50, cols, torch.bfloat16, 9)
    index = torch.randint(0, 50, (123,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    index[7] = index[99] = -1
    q, s = quantize(plan, x.cuda(), 123, cols, index=index.cuda())
    ref_s, ref_q = reference(x[index.long()].double().numpy(), 1)
    kept = index.numpy() >= 0
    assert np.array_equal(s[kept], ref_s[kept]) and same_bytes(q[kept], to_e4m3(ref_q)[kept])
    assert np.all(q[~kept] == FILL) and np.all(s[~kept] == FILL)
    index[3] = 50  # one past the last row
    q, s = quantize(plan, x.cuda(), 123, cols, index=index.cuda(), status=dfx.DFX_STATUS_INDEX)
    assert np.all(q[3] == FILL) and np.all(s[3] == FILL)


@pytest.mark.parametrize("rows,cols,dtype", [(1, 128, torch.bfloat16), (33, 1000, torch.bfloat16),
                                             (9, 129, torch.float32), (64, 2048, torch.float32)])
def test_quantize_swiglu(plan, rows, cols, dtype):
    x = torch.cat([values(rows, cols, dtype, 4, 0.5) * 3, values(rows, cols, dtype, 5)], 1)
    x[0, 0] = -200.0  # exp(200) is beyond FP32
    x[0, 1] = 300.0
    q, s = quantize(plan, x.cuda(), rows, cols, flags=dfx.DFX_QUANT_SWIGLU)
    g, u = x[:, :cols].double().numpy(), x[:, cols:].double().numpy()
    with np.errstate(over="ignore"):
        v = g / (1 + np.exp(-g)) * u
    ref_s, ref_q = reference(v, 1)
    assert np.array_equal(s, ref_s)
    got = torch.from_numpy(q).view(torch.float8_e4m3fn).double().numpy()
    # half a step of e4m3 (2^-4 of the value, 2^-10 among its subnormals), and FP32's error of the
    # product: exponential and quotient within 2^-20 together
    assert np.all(np.abs(got - ref_q) <= np.abs(ref_q) * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10)


def test_quantize_swiglu_scale_at_its_border(plan):
    """Largest values within FP32's rounding of 1.75 * 2^k: the scale goes by the exact product."""
    g = np.linspace(0.5, 9.0, 4096).astype(np.float32)
    silu = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64)))
    u = (1.75 / silu).astype(np.float32)
    rows = []
    for step in (-1, 0, 1):
        t = u.copy()
        for _ in range(abs(step)):
            t = np.nextafter(t, np.float32(step * 100.0))
        rows.append(t)
    u = np.concatenate(rows)
    g = np.tile(g, 3)
    x = torch.zeros(g.size, 256)
    x[:, 5], x[:, 128 + 5] = torch.from_numpy(g), torch.from_numpy(u)
    _, s = quantize(plan, x.cuda(), g.size, 128, flags=dfx.DFX_QUANT_SWIGLU)
    v = g.astype(np.float64) / (1 + np.exp(-g.astype(np.float64))) * u.astype(np.float64)
    sure = np.abs(v - 1.75) > 1e-14
    assert np.array_equal(s[sure, 0], np.where(v > 1.75, 120, 119)[sure])


# ---------------------------------------------------------------- products

def operand(q, s, cols):
    """Rows and scales in buffers whose unused bytes are NaN values and NaN scales."""
    qb = torch.full((*q.shape[:-1], up(cols, 16)), 0x7F, dtype=torch.uint8)
    qb[..., :cols] = q.view(torch.uint8)
    sb = torch.full((*s.shape[:-1], up(s.shape[-1], 4)), 0xFF, dtype=torch.uint8)
    sb[..., : s.shape[-1]] = s
    return qb.cuda(), sb.cuda()


def product(plan, x, sx, w, sw, rows, cols, offsets=None, y_type=torch.float32, ld_y=None, status=0, fill=-7.0):
    """x: float8 [tokens, cols]; w: float8 [experts, rows, cols] (CPU); Y with its untouched elements."""
    tokens, experts = x.shape[0], w.shape[0]
    xb, sxb = operand(x, sx, cols)
    wb, swb = operand(w, sw, cols)
    y = torch.full((tokens, ld_y or rows), fill, dtype=y_type, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dfx.dfx_gemm_fp8(plan, xb, xb.shape[-1], sxb, sxb.shape[-1], tokens, wb, wb.shape[-1], swb, swb.shape[-1], rows, cols,
                     experts, off, y, dfx.DFX_F32 if y_type == torch.float32 else dfx.DFX_BF16, y.shape[1])
    assert dfx.dfx_device_status(plan) == status
    return y.cpu()


def scaled(q, s, block_rows):
    v = q.float().double()
    f = torch.exp2(s.double() - 127)
    f = f.repeat_interleave(block_rows, -2)[..., : v.shape[-2], :].repeat_interleave(128, -1)[..., : v.shape[-1]]
    return v * f


def grid_case(tokens, rows, cols, experts, seed):
    """Integers in -4..4 and scales 1/2, 1, 2: every sum is a multiple of 1/4 below 2^24 / 4."""
    g = torch.Generator().manual_seed(seed)
    blocks = -(-cols // 128)
    x = torch.randint(-4, 5, (tokens, cols), generator=g).float().to(torch.float8_e4m3fn)
    w = torch.randint(-4, 5, (experts, rows, cols), generator=g).float().to(torch.float8_e4m3fn)
    sx = torch.randint(126, 129, (tokens, blocks), generator=g).to(torch.uint8)
    sw = torch.randint(126, 129, (experts, -(-rows // 128), blocks), generator=g).to(torch.uint8)
    return x, sx, w, sw


def check(y, x, sx, w, sw, offsets, rows, exact, fill=-7.0):
    tokens = x.shape[0]
    xv, wv = scaled(x, sx, 1), scaled(w, sw, 128)
    edges = [0, tokens] if offsets is None else offsets
    used = torch.zeros(tokens, dtype=torch.bool)
    for e in range(w.shape[0]):
        a, b = edges[e], edges[e + 1]
        used[a:b] = True
        ref = xv[a:b] @ wv[e].T
        got = y[a:b, :rows]
        if exact:
            assert torch.equal(got, ref.to(y.dtype)), (e, (got.double() - ref).abs().max())
        else:
            # FP32 sums in any order (2^-23 a term, for an accumulator that truncates), rounded once
            room = x.shape[1] * 2.0 ** -23 * (xv[a:b].abs() @ wv[e].abs().T) + torch.finfo(y.dtype).eps / 2 * ref.abs()
            assert torch.all((got.double() - ref).abs() <= room + 1e-30)
    assert torch.all(y[~used] == fill) and torch.all(y[:, rows:] == fill), "elements outside Y were written"


DENSE = [(1, 128, 128), (1, 1, 16), (1, 4096, 1024), (16, 256, 512), (17, 130, 640), (33, 384, 128), (100, 200, 1000),
         (129, 128, 2048), (240, 100, 500), (241, 256, 256), (500, 700, 300), (1000, 1024, 1100), (3, 513, 4096),
         (32, 128, 8192), (7, 64, 1),
         # K split over a cluster of 2, 4 and 8; pairs of 240 and of 256 tokens
         (5, 5000, 1000), (9, 1000, 1300), (1, 1030, 2100), (70, 600, 1500), (480, 300, 260), (512, 600, 700), (1025, 300, 384)]


@pytest.mark.parametrize("tokens,rows,cols", DENSE)
@pytest.mark.parametrize("y_type", [torch.float32, torch.bfloat16])
def test_gemm_exact_on_integers(plan, tokens, rows, cols, y_type):
    x, sx, w, sw = grid_case(tokens, rows, cols, 1, tokens + rows + cols)
    y = product(plan, x, sx, w, sw, rows, cols, y_type=y_type, ld_y=rows + 3)
    check(y, x, sx, w, sw, None, rows, exact=True)


def gaussian_case(tokens, rows, cols, experts, seed):
    g = torch.Generator().manual_seed(seed)
    blocks = -(-cols // 128)

    def quant(v, block_rows):
        s, q = reference(v.double().numpy().reshape(-1, cols), block_rows)
        return torch.from_numpy(to_e4m3(q)).view(torch.float8_e4m3fn), torch.from_numpy(s)

    x, sx = quant(torch.randn(tokens, cols, generator=g), 1)
    ws, sws = zip(*[quant(torch.randn(rows, cols, generator=g) / math.sqrt(cols), 128) for _ in range(experts)])
    w, sw = torch.stack([v.view(torch.uint8) for v in ws]).view(torch.float8_e4m3fn), torch.stack(sws)
    assert sw.shape == (experts, -(-rows // 128), blocks)
    return x, sx, w, sw


@pytest.mark.parametrize("tokens,rows,cols", [(1, 512, 4096), (40, 300, 2000), (300, 256, 1024)])
@pytest.mark.parametrize("y_type", [torch.float32, torch.bfloat16])
def test_gemm_gaussian(plan, tokens, rows, cols, y_type):
    x, sx, w, sw = gaussian_case(tokens, rows, cols, 1, 5)
    check(product(plan, x, sx, w, sw, rows, cols, y_type=y_type), x, sx, w, sw, None, rows, exact=False)


GROUPED = [
    # tokens, rows, cols, offsets
    (5, 128, 256, [0, 5]),                              # one matrix with offsets
    (10, 130, 200, [0, 0, 10, 10]),                     # experts without tokens
    (64, 256, 384, [0, 1, 3, 3, 40, 64]),
    (64, 100, 128, [2, 10, 20, 50]),                    # rows in front and behind stay
    (300, 128, 512, [0, 250, 260, 299]),
    (700, 200, 300, [0, 1, 500, 500, 690]),
    (40, 128, 128, [0] * 41),                           # no expert has a token
    (200, 128, 160, list(range(0, 201))),               # 200 experts of one token each
    (900, 20, 130, [0] * 500 + list(range(0, 524)) + [880]),  # as many experts as there may be
    (260, 140, 256, [0, 129, 260]),                     # runs of an expert on both sides of a tile's cap
    (1500, 300, 256, [0, 700, 1480]),                   # pairs of CTAs
]


@pytest.mark.parametrize("tokens,rows,cols,offsets", GROUPED)
def test_gemm_experts_exact_on_integers(plan, tokens, rows, cols, offsets):
    x, sx, w, sw = grid_case(tokens, rows, cols, len(offsets) - 1, tokens)
    y = product(plan, x, sx, w, sw, rows, cols, offsets, y_type=torch.bfloat16)
    check(y, x, sx, w, sw, offsets, rows, exact=True)


def test_gemm_every_scale_byte_reaches_its_block(plan):
    """One value per row, block and token: Y shows the product of exactly two scales."""
    tokens, rows, cols = 250, 256, 1024
    g = torch.Generator().manual_seed(2)
    sx = torch.randint(100, 150, (tokens, 8), generator=g).to(torch.uint8)
    sw = torch.randint(100, 150, (1, 2, 8), generator=g).to(torch.uint8)
    w = torch.ones(1, rows, cols).to(torch.float8_e4m3fn)
    for block in range(8):
        x = torch.zeros(tokens, cols)
        x[:, 128 * block + (37 * block) % 128] = 1.0
        x = x.to(torch.float8_e4m3fn)
        y = product(plan, x, sx, w, sw, rows, cols)
        ref = torch.exp2(sx[:, block].double() + 0.0)[:, None] * torch.exp2(sw[0, :, block].double() - 254.0)[None, :]
        assert torch.equal(y.double(), ref.repeat_interleave(128, 1)), block


def test_gemm_nan_and_the_extreme_scales(plan):
    """NaN stays in its token's row; scales at both ends; neighbours of a NaN token are unharmed."""
    x, sx, w, sw = grid_case(20, 128, 256, 1, 7)
    clean = product(plan, x, sx, w, sw, 128, 256)
    xb = x.clone().view(torch.uint8)
    xb[3, 5] = 0x7F
    y = product(plan, xb.view(torch.float8_e4m3fn), sx, w, sw, 128, 256)
    assert torch.all(torch.isnan(y[3]))
    rest = torch.arange(20) != 3
    assert torch.equal(y[rest], clean[rest])
    x = torch.ones(4, 128).to(torch.float8_e4m3fn)
    w = torch.ones(1, 128, 128).to(torch.float8_e4m3fn)
    sx = torch.tensor([[0], [127], [200], [254]], dtype=torch.uint8)
    y = product(plan, x, sx, w, torch.tensor([[[127]]], dtype=torch.uint8), 128, 128)
    assert torch.equal(y[:3, 0].double(), torch.tensor([128 * 2.0 ** -127, 128.0, 128 * 2.0 ** 73], dtype=torch.float64))


def test_gemm_bad_offsets_set_the_status_and_stay_inside(plan):
    x, sx, w, sw = grid_case(50, 128, 128, 3, 1)
    for offsets in ([0, 20, 10, 50], [0, 20, 40, 51], [-1, 20, 30, 50], [0, 50, 0, 50], [50, 0, 50, 0]):
        product(plan, x, sx, w, sw, 128, 128, offsets, status=dfx.DFX_STATUS_INDEX)
    y = product(plan, x, sx, w, sw, 128, 128, [0, 20, 30, 50])
    check(y, x, sx, w, sw, [0, 20, 30, 50], 128, exact=True)


@pytest.mark.parametrize("tokens,rows,cols", [(20, 256, 512), (1, 128, 100), (100, 2000, 128), (300, 512, 640), (512, 300, 300)])
def test_gemm_wait_that_runs_out_is_reported(plan, tokens, rows, cols):
    """Tile copies that are left out: the status says so, and the next call is sound."""
    x, sx, w, sw = grid_case(tokens, rows, cols, 1, 3)
    dfx.dfx_debug_inject(dfx.DFX_INJECT_SKIP_TILE_COPY)
    try:
        product(plan, x, sx, w, sw, rows, cols, status=dfx.DFX_STATUS_TIMEOUT)
    finally:
        dfx.dfx_debug_inject(0)
    check(product(plan, x, sx, w, sw, rows, cols), x, sx, w, sw, None, rows, exact=True)


def test_nothing_to_do(plan):
    dfx.dfx_gemm_fp8(plan, None, 16, None, 4, 0, None, 16, None, 4, 128, 16, 1, None, None, dfx.DFX_F32, 128)
    dfx.dfx_gemm_fp8(plan, None, 16, None, 4, 5, None, 16, None, 4, 0, 16, 1, None, None, dfx.DFX_F32, 0)
    dfx.dfx_quantize_fp8(plan, None, dfx.DFX_F32, 16, 0, None, 0, 16, 1, 0, None, 16, None, 4)
    assert dfx.dfx_device_status(plan) == 0


# One to eight tokens, one matrix: rows spread over the SMs, two rows of scales in a tile, K's last
# block cut at several places of its 16 bytes, the most rows and blocks of one round of loads and more.
FEW = [(1, 1, 1), (2, 147, 15), (3, 149, 17), (8, 2500, 31), (5, 2368, 1000), (7, 2369, 300), (8, 500, 8192), (4, 130, 8193),
       (8, 4096, 4096), (6, 4737, 4100), (1, 18944, 100), (8, 18945, 130), (2, 18945, 128), (1, 7, 5000), (8, 16, 1024)]


@pytest.mark.parametrize("tokens,rows,cols", FEW)
@pytest.mark.parametrize("y_type", [torch.float32, torch.bfloat16])
def test_gemm_few_tokens_exact_on_integers(plan, tokens, rows, cols, y_type):
    x, sx, w, sw = grid_case(tokens, rows, cols, 1, rows)
    y = product(plan, x, sx, w, sw, rows, cols, y_type=y_type, ld_y=rows + 5)
    check(y, x, sx, w, sw, None, rows, exact=True)


@pytest.mark.parametrize("tokens,rows,cols", [(1, 1000, 4096), (8, 700, 2000), (3, 3000, 520)])
def test_gemm_few_tokens_gaussian(plan, tokens, rows, cols):
    x, sx, w, sw = gaussian_case(tokens, rows, cols, 1, 6)
    check(product(plan, x, sx, w, sw, rows, cols), x, sx, w, sw, None, rows, exact=False)


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9])
def test_gemm_few_tokens_scales_and_nan(plan, tokens):
    """Scale bytes of which only the product is in FP32's range, NaN scales, and a NaN value of W and of X."""
    rows, cols = 300, 640
    x = torch.ones(tokens, cols).to(torch.float8_e4m3fn)
    w = torch.ones(1, rows, cols).to(torch.float8_e4m3fn)
    sx = torch.tensor([[0, 254, 250, 2, 127]], dtype=torch.uint8).repeat(tokens, 1)
    sw = torch.tensor([[254, 0, 1, 254, 127]], dtype=torch.uint8).repeat(3, 1)[None].contiguous()
    want = 128 * (1 + 1 + 0.125 + 4 + 1)  # 128 products a block, times 2^(sx + sw - 254)
    assert torch.all(product(plan, x, sx, w, sw, rows, cols) == want)
    bad = sw.clone()
    bad[0, 1, 3] = 255
    y = product(plan, x, sx, w, bad, rows, cols)
    assert torch.all(torch.isnan(y[:, 128:256])) and torch.all(y[:, :128] == want) and torch.all(y[:, 256:] == want)
    bad = sx.clone()
    bad[tokens - 1, 0] = 255
    y = product(plan, x, bad, w, sw, rows, cols)
    assert torch.all(torch.isnan(y[tokens - 1])) and torch.all(y[: tokens - 1] == want)
    bad = w.clone().view(torch.uint8)
    bad[0, 200, 639] = 0xFF
    y = product(plan, x, sx, bad.view(torch.float8_e4m3fn), sw, rows, cols)
    assert torch.all(torch.isnan(y[:, 200])) and torch.all(y[:, :200] == want) and torch.all(y[:, 201:] == want)
    bad = x.clone().view(torch.uint8)
    bad[0, 0] = 0x7F
    y = product(plan, bad.view(torch.float8_e4m3fn), sx, w, sw, rows, cols)
    assert torch.all(torch.isnan(y[0])) and torch.all(y[1:] == want)
