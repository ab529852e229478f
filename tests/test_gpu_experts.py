"""A layer of experts with 8-bit weights through the tensor helpers: weights restored from their
containers, laid out in 8 bits, tokens routed, sent to their experts, multiplied, brought back."""
import numpy as np
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


def values(f: dfx.Fp8):
    """What an Fp8 stands for, in float64."""
    v = f.values[..., : f.cols].view(torch.float8_e4m3fn).double()
    s = torch.exp2(f.scales[..., : -(-f.cols // 128)].double() - 127)
    return v * s.repeat_interleave(f.block_rows, -2)[..., : v.shape[-2], :].repeat_interleave(128, -1)[..., : f.cols]


def layer(tokens, experts, width, inner, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, width, generator=g).to(dtype)
    logits = torch.randn(tokens, experts, generator=g) * 1.5
    w_in = (torch.randn(experts, 2 * inner, width, generator=g) / width ** 0.5).bfloat16()
    w_out = (torch.randn(experts, width, inner, generator=g) / inner ** 0.5).bfloat16()
    return x.cuda(), logits.cuda(), w_in.cuda(), w_out.cuda()


def restored(w):
    """A weight through its container and back."""
    back = dfx.decode(dfx.encode(w), w.numel()).reshape(w.shape)
    assert torch.equal(back.view(torch.int16), w.view(torch.int16))
    return back


CASES = [
    dict(tokens=1, experts=8, width=256, inner=128, topk=2),
    dict(tokens=37, experts=16, width=384, inner=200, topk=4, score="sigmoid", renormalize=True),
    dict(tokens=300, experts=4, width=512, inner=256, topk=2, renormalize=True),
    dict(tokens=130, experts=64, width=136, inner=72, topk=8, score="sigmoid", groups=8, top_groups=3, group_best=2,
         renormalize=True, scale=2.5),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_step_by_step(case, dtype):
    """Each step against its definition in 64 bits on the step before's actual output, and the
    layer's own call against the steps, bit for bit."""
    case = dict(case)
    sizes = [case.pop(k) for k in ("tokens", "experts", "width", "inner")]
    tokens, experts, width, inner = sizes
    topk = case.pop("topk")
    x, logits, w_in, w_out = layer(*sizes, seed=sum(sizes), dtype=dtype)
    logits[tokens // 3] = -torch.inf  # padding
    a, b = dfx.quantize_fp8(restored(w_in), block_rows=128), dfx.quantize_fp8(restored(w_out), block_rows=128)
    # a rounding to e4m3 is off by at most 2^-4 of the value, or 2^-10 of the scale among subnormals
    scale = torch.exp2(a.scales[..., : -(-width // 128)].double() - 127).repeat_interleave(128, -2)[:, : 2 * inner]
    scale = scale.repeat_interleave(128, -1)[..., :width]
    assert torch.all((values(a) - w_in.double()).abs() <= w_in.double().abs() * 2.0 ** -4 + scale * 2.0 ** -10)

    r = dfx.route(logits, topk, **case)
    offsets = r.offsets.tolist()
    used = offsets[-1]
    assert used == (r.ids >= 0).sum().item() and r.ids[tokens // 3].tolist() == [-1] * topk
    xq = dfx.quantize_fp8(x, index=r.rows)
    whole = dfx.quantize_fp8(x)
    sent = r.rows[:used].long()
    assert torch.equal(xq.values[:used, :width], whole.values[sent][:, :width])
    assert torch.equal(xq.scales[:used, : -(-width // 128)], whole.scales[sent][:, : -(-width // 128)])

    def product_is_right(y, q, w):
        v, wv = values(Fp8_rows(q, used)), values(w)
        for e in range(experts):
            lo, hi = offsets[e], offsets[e + 1]
            ref = v[lo:hi] @ wv[e].T
            # FP32 sums in any order (2^-23 a term), rounded once to BF16 (2^-8)
            room = q.cols * 2.0 ** -23 * (v[lo:hi].abs() @ wv[e].abs().T) + 2.0 ** -8 * ref.abs()
            assert torch.all((y[lo:hi].double() - ref).abs() <= room + 1e-30)

    h = dfx.gemm_fp8(xq, a, r.offsets)
    product_is_right(h, xq, a)
    hq = dfx.quantize_fp8(h, swiglu=True)
    gate, value = h[:used, :inner].double(), h[:used, inner:].double()
    act = gate / (1 + torch.exp(-gate)) * value
    got = values(Fp8_rows(hq, used))
    step = torch.exp2(hq.scales[:used, : -(-inner // 128)].double() - 127).repeat_interleave(128, -1)[:, :inner]
    assert torch.all((got - act).abs() <= act.abs() * (2.0 ** -4 + 2.0 ** -20) + step * 2.0 ** -10)
    z = dfx.gemm_fp8(hq, b, r.offsets)
    product_is_right(z, hq, b)
    y = dfx.combine(z, r.slots, r.weights, dtype=dtype)
    terms = torch.where(r.slots[..., None] >= 0, r.weights[..., None].double() * z[r.slots.long().clamp(min=0)].double(), 0.0)
    ref = terms.sum(1)
    room = topk * 2.0 ** -24 * terms.abs().sum(1) + torch.finfo(dtype).eps / 2 * ref.abs()
    assert torch.all((y.double() - ref).abs() <= room)
    assert torch.all(y[tokens // 3] == 0)
    assert torch.equal(dfx.experts_fp8(x, logits, a, b, topk, **case), y)


def Fp8_rows(f, n):
    return f._replace(values=f.values[:n], scales=f.scales[:n])


def test_captured_layer_follows_its_inputs():
    x, logits, w_in, w_out = layer(64, 8, 256, 128, seed=1)
    a, b = dfx.quantize_fp8(w_in, block_rows=128), dfx.quantize_fp8(w_out, block_rows=128)
    with dfx.dfx_plan(0) as plan:
        dfx.experts_fp8(x, logits, a, b, 2, plan=plan)  # loads the kernels
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = dfx.experts_fp8(x, logits, a, b, 2, plan=plan)
        for seed in (2, 3):
            x2, logits2, _, _ = layer(64, 8, 256, 128, seed)
            x.copy_(x2), logits.copy_(logits2)
            graph.replay()
            torch.cuda.synchronize()
            assert dfx.dfx_device_status(plan) == 0
            assert torch.equal(y, dfx.experts_fp8(x2, logits2, a, b, 2))


def test_two_streams_at_once():
    """Layers on two streams, each with its own buffers, do not disturb one another."""
    sets = [layer(200, 16, 256, 128, seed=s) for s in (1, 2)]
    w = [(dfx.quantize_fp8(s[2], block_rows=128), dfx.quantize_fp8(s[3], block_rows=128)) for s in sets]
    want = [dfx.experts_fp8(s[0], s[1], *q, 4) for s, q in zip(sets, w)]
    streams = [torch.cuda.Stream() for _ in sets]
    plans = [dfx.dfx_plan(0) for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (s, q) in enumerate(zip(sets, w)):
            got[i].append(dfx.experts_fp8(s[0], s[1], *q, 4, plan=plans[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert dfx.dfx_device_status(plans[i]) == 0
        assert all(torch.equal(g, want[i]) for g in got[i])
        plans[i].free()


def test_helpers_take_views_and_refuse_the_rest():
    x = torch.randn(40, 300, device="cuda").bfloat16()
    part = x[:, 3:260]  # neither aligned nor contiguous
    q, ref = dfx.quantize_fp8(part), dfx.quantize_fp8(part.contiguous())
    assert torch.equal(q.values[:, :257], ref.values[:, :257]) and torch.equal(q.scales[:, :3], ref.scales[:, :3])
    t = dfx.quantize_fp8(x.T)
    assert torch.equal(t.values[:, :40], dfx.quantize_fp8(x.T.contiguous()).values[:, :40])
    w = dfx.quantize_fp8(torch.randn(64, 257, device="cuda"), block_rows=128)
    y = dfx.gemm_fp8(q, w)
    out = torch.zeros(40, 80, device="cuda", dtype=torch.bfloat16)
    dfx.gemm_fp8(q, w, out=out[:, :64])
    assert torch.equal(out[:, :64], y) and torch.all(out[:, 64:] == 0)
    with pytest.raises(ValueError):
        dfx.gemm_fp8(q, q)                                  # 1 x 128 blocks on both sides
    with pytest.raises(ValueError):
        dfx.gemm_fp8(q, dfx.quantize_fp8(torch.randn(64, 256, device="cuda"), block_rows=128))
    with pytest.raises(ValueError):
        dfx.gemm_fp8(q, w, out=out[:1, :64].expand(40, 64))  # rows on top of one another
    with pytest.raises(ValueError):
        dfx.gemm_fp8(q._replace(scales=q.scales[:39]), w)
    with pytest.raises(ValueError):
        dfx.gemm_fp8(q, w._replace(values=w.values[:, :256]))
    with pytest.raises(ValueError):
        dfx.quantize_fp8(torch.zeros(4, 4))                 # not on a GPU
    with pytest.raises(TypeError):
        dfx.quantize_fp8(torch.zeros(4, 4, device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        dfx.quantize_fp8(x, index=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        dfx.route(torch.zeros(4, 8, device="cuda"), 2, score="relu")
    with pytest.raises(dfx.DfxError) as e:
        dfx.route(torch.zeros(4, 8, device="cuda"), 9)
    assert e.value.code == dfx.DFX_ERR_ARG
    with pytest.raises(dfx.DfxError) as e:                  # a row that x does not have
        dfx.quantize_fp8(x, index=torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    assert e.value.code == dfx.DFX_ERR_CORRUPT


def test_no_token():
    x, logits, w_in, w_out = layer(0, 8, 256, 128, seed=1)
    y = dfx.experts_fp8(x, logits, dfx.quantize_fp8(w_in, block_rows=128), dfx.quantize_fp8(w_out, block_rows=128), 2)
    assert y.shape == (0, 256)


@pytest.mark.parametrize("tokens", [1, 16, 300])
def test_results_do_not_depend_on_the_run(tokens):
    x, logits, w_in, w_out = layer(tokens, 32, 512, 256, seed=6)
    a, b = dfx.quantize_fp8(w_in, block_rows=128), dfx.quantize_fp8(w_out, block_rows=128)
    first = dfx.experts_fp8(x, logits, a, b, 8)
    for _ in range(5):
        assert torch.equal(dfx.experts_fp8(x, logits, a, b, 8), first)
