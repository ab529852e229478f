"""dfx_route and dfx_combine against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import lossless_entropy_coded_exponent_b200 as dfx
from lossless_entropy_coded_exponent_b200 import build as dfx_build

pytestmark = pytest.mark.gpu

FILL = -77


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfx_build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    dfx.lib()


@pytest.fixture(scope="module")
def plan():
    with dfx.dfx_plan(0) as p:
        yield p


def route(plan, logits, topk, sigmoid=False, bias=None, groups=0, top_groups=0, best=0, renorm=False, scale=0.0,
          ld=None, lists=True, experts=None):
    tokens, e = logits.shape[0], experts or logits.shape[1]
    params = dfx.dfx_route_params(score=dfx.DFX_SCORE_SIGMOID if sigmoid else dfx.DFX_SCORE_SOFTMAX, topk=topk,
                                  groups=groups, top_groups=top_groups, group_best=best, renormalize=int(renorm),
                                  scale=scale)
    ints = lambda *s: torch.full(s, FILL, dtype=torch.int32, device="cuda")  # noqa: E731
    ids, weights = ints(tokens, topk), torch.full((tokens, topk), math.nan, device="cuda")
    offsets, rows, slots = ints(e + 1), ints(tokens * topk), ints(tokens, topk)
    ws = torch.empty(dfx.dfx_route_workspace(tokens, e, params), dtype=torch.uint8, device="cuda")
    extra = (offsets, rows, slots, ws, ws.numel()) if lists else ()
    dfx.dfx_route(plan, logits.cuda(), dfx.DFX_BF16 if logits.dtype == torch.bfloat16 else dfx.DFX_F32,
                  ld or logits.shape[1], tokens, e, None if bias is None else bias.cuda(), params, ids, weights, *extra)
    assert dfx.dfx_device_status(plan) == 0
    return [v.cpu().numpy() for v in (ids, weights, offsets, rows, slots)]


def reference(logits, topk, sigmoid=False, bias=None, groups=0, top_groups=0, best=0, renorm=False, scale=0.0):
    x = logits.double().numpy()
    b = None if bias is None else bias.double().numpy()
    tokens, experts = x.shape
    best = best or 1
    ids = np.full((tokens, topk), -1)
    weights = np.zeros((tokens, topk))
    for t in range(tokens):
        open_ = x[t] > -np.inf
        if b is not None:
            closed_by_bias = ~(b > -np.inf)
        score = np.zeros(experts)
        if open_.any():
            if sigmoid:
                with np.errstate(over="ignore"):
                    score[open_] = 1.0 / (1.0 + np.exp(-x[t, open_]))
            else:
                m = x[t, open_].max()
                with np.errstate(invalid="ignore"):
                    e = np.where(x[t, open_] == m, 1.0, np.exp(x[t, open_] - m))
                score[open_] = e / e.sum()
        by_score = b is not None or (groups > 1 and best == 2)
        choice = (score + (0 if b is None else b)) if by_score else x[t].copy()
        choice[~open_] = -np.inf
        if b is not None:
            choice[closed_by_bias] = -np.inf
        if groups > 1:
            per = experts // groups
            worth = []
            for g in range(groups):
                top = np.sort(choice[g * per:(g + 1) * per])[::-1][:best]
                worth.append(-np.inf if top[0] == -np.inf else top[top > -np.inf].sum())
            kept = np.argsort(-np.array(worth), kind="stable")[:top_groups]
            for g in range(groups):
                if g not in kept:
                    choice[g * per:(g + 1) * per] = -np.inf
        order = np.argsort(-choice, kind="stable")[:topk]
        order = order[choice[order] > -np.inf]
        ids[t, : order.size] = order
        w = score[order]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        weights[t, : order.size] = w * (scale or 1.0)
    return ids, weights


def check_lists(ids, offsets, rows, slots, experts):
    tokens, topk = ids.shape
    flat = ids.reshape(-1)
    kept = np.nonzero(flat >= 0)[0]
    order = kept[np.argsort(flat[kept], kind="stable")]
    counts = np.bincount(flat[kept], minlength=experts)
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(counts)]))
    want_rows = np.full(tokens * topk, -1)
    want_rows[: order.size] = order // topk
    want_slots = np.full(tokens * topk, -1)
    want_slots[order] = np.arange(order.size)
    assert np.array_equal(rows, want_rows)
    assert np.array_equal(slots.reshape(-1), want_slots)


def check(plan, logits, topk, **kw):
    ids, weights, offsets, rows, slots = route(plan, logits, topk, **kw)
    want, w = reference(logits, topk, **kw)
    assert np.array_equal(ids, want)
    # chosen scores are formed in FP64 and rounded once (2^-24); a softmax over all logits divides
    # by an FP32 sum of exponentials: 2^-22 each, at most 16 + 5 additions of 2^-24
    assert np.all(np.abs(weights - w) <= np.abs(w) * (8 + 21 + 1) * 2.0 ** -24 + 2.0 ** -149)
    check_lists(ids, offsets, rows, slots, logits.shape[1])


def logits_of(tokens, experts, dtype=torch.float32, seed=0, spread=1.5):
    return (torch.randn(tokens, experts, generator=torch.Generator().manual_seed(seed)) * spread).to(dtype)


SIZES = [(1, 1, 1), (1, 8, 2), (2, 33, 5), (63, 64, 6), (64, 64, 6), (65, 60, 8), (100, 128, 8), (300, 256, 8),
         (7, 257, 16), (1000, 512, 32), (500, 512, 1), (3, 32, 32), (5000, 96, 4), (513, 5, 5)]


@pytest.mark.parametrize("tokens,experts,topk", SIZES)
@pytest.mark.parametrize("sigmoid,bias,renorm", [(False, False, False), (False, False, True), (True, False, True),
                                                 (True, True, True), (False, True, False)])
def test_route(plan, tokens, experts, topk, sigmoid, bias, renorm):
    x = logits_of(tokens, experts, seed=tokens + experts)
    b = 0.2 * torch.randn(experts, generator=torch.Generator().manual_seed(1)) if bias else None
    check(plan, x, topk, sigmoid=sigmoid, bias=b, renorm=renorm, scale=2.5 if renorm else 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("experts,groups,top_groups,topk", [(64, 8, 3, 6), (256, 8, 4, 8), (60, 4, 2, 5), (512, 32, 1, 16),
                                                            (96, 32, 32, 8), (6, 3, 2, 4), (8, 8, 3, 3)])
@pytest.mark.parametrize("best,bias", [(1, False), (2, False), (1, True), (2, True)])
def test_groups(plan, dtype, experts, groups, top_groups, topk, best, bias):
    x = logits_of(150, experts, dtype, seed=experts)
    x[3:6] = -math.inf
    x[6, ::2] = -math.inf
    b = 0.2 * torch.randn(experts, generator=torch.Generator().manual_seed(1)) if bias else None
    check(plan, x, topk, sigmoid=True, bias=b, groups=groups, top_groups=top_groups, best=best, renorm=True)
    check(plan, x, topk, bias=b, groups=groups, top_groups=top_groups, best=best)


@pytest.mark.parametrize("tokens", [40, 200])
def test_ties_go_to_the_lowest_index(plan, tokens):
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-1, 2, (tokens, 64), generator=g).float()
    x[0] = 0.0
    x[1, ::2], x[1, 1::2] = 0.0, -0.0  # the same value
    check(plan, x, 9)
    check(plan, x.bfloat16(), 9, sigmoid=True, bias=torch.zeros(64), renorm=True)
    check(plan, x, 6, sigmoid=True, bias=torch.zeros(64), groups=8, top_groups=3, best=2)
    check(plan, x, 6, groups=8, top_groups=3, best=1)


@pytest.mark.parametrize("tokens", [30, 333])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_masked_rows_and_extreme_logits(plan, tokens, sigmoid, bias):
    x = logits_of(tokens, 40, seed=8)
    low = torch.finfo(torch.float32).min
    x[0] = -math.inf                       # padding
    x[1, 3:] = -math.inf                   # three experts open
    x[2] = low                             # the lowest value is no mask: all equal
    x[3, :20] = low
    x[4, 7] = math.inf
    x[5, [2, 9]] = math.inf
    x[6] = math.nan
    x[7, 5] = math.nan
    x[8] = -1000.0                         # scores of zero
    x[9] = 1000.0
    x[10, 1:] = -math.inf
    x[11:20, ::3] = -math.inf
    x[-1] = -math.inf
    b = None
    if bias:
        b = 0.1 * torch.randn(40, generator=torch.Generator().manual_seed(1))
        b[4], b[11] = -math.inf, math.nan
    for renorm in (False, True):
        check(plan, x, 8, sigmoid=sigmoid, bias=b, renorm=renorm)


def test_near_scores_keep_their_order(plan):
    """Choices nearer than FP32's rounding come in the order of their exact values."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(400, 32, generator=g)
    s = 1 / (1 + torch.exp(-x[:1].double()))
    x[:] = x[:1]
    b = (1.0 - s[0]).float()  # every score + bias is 1 within FP32's rounding
    check(plan, x, 12, sigmoid=True, bias=b, renorm=True)


def test_no_token_and_every_token_masked(plan):
    ids, weights, offsets, rows, slots = route(plan, torch.zeros(0, 16), 2)
    assert np.all(offsets == 0)
    for tokens in (5, 100):
        ids, weights, offsets, rows, slots = route(plan, torch.full((tokens, 16), -math.inf), 2)
        assert np.all(ids == -1) and np.all(weights == 0) and np.all(offsets == 0)
        assert np.all(rows == -1) and np.all(slots == -1)


@pytest.mark.parametrize("tokens", [10, 200])
def test_strided_logits_and_no_lists(plan, tokens):
    x = logits_of(tokens, 70, seed=2)
    ids, weights, offsets, rows, slots = route(plan, x, 4, experts=64, lists=False)
    want, w = reference(x[:, :64], 4)
    assert np.array_equal(ids, want)
    assert np.all(offsets == FILL) and np.all(rows == FILL) and np.all(slots == FILL)


def test_one_expert_takes_every_token(plan):
    x = torch.zeros(70_000, 3)
    x[:, 1] = 5.0
    ids, weights, offsets, rows, slots = route(plan, x, 1)
    assert np.all(ids == 1) and offsets.tolist() == [0, 0, 70_000, 70_000]
    assert np.array_equal(rows, np.arange(70_000)) and np.array_equal(slots[:, 0], np.arange(70_000))


# ---------------------------------------------------------------- the way back

def combine(plan, z, slots, weights, cols, y_type, ld_y=None, z_rows=None, status=0):
    tokens, topk = slots.shape
    y = torch.full((tokens, ld_y or cols), 5.0, dtype=y_type, device="cuda")
    kind = lambda t: dfx.DFX_BF16 if t == torch.bfloat16 else dfx.DFX_F32  # noqa: E731
    dfx.dfx_combine(plan, z.cuda(), kind(z.dtype), z.shape[1], z_rows or z.shape[0], cols, slots.cuda(), weights.cuda(),
                    tokens, topk, y, kind(y_type), y.shape[1])
    assert dfx.dfx_device_status(plan) == status
    y = y.cpu()
    assert torch.all(y[:, cols:] == 5.0)
    return y[:, :cols]


@pytest.mark.parametrize("tokens,topk,cols,ld_z,ld_y", [(1, 1, 1, 1, 1), (1, 8, 4096, 4096, 4096), (33, 2, 100, 104, 101),
                                                        (130, 8, 256, 256, 264), (20, 17, 64, 64, 64), (9, 32, 7, 9, 8),
                                                        (700, 6, 1000, 1000, 1000)])
@pytest.mark.parametrize("z_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("y_type", [torch.bfloat16, torch.float32])
def test_combine(plan, tokens, topk, cols, ld_z, ld_y, z_type, y_type):
    g = torch.Generator().manual_seed(tokens + cols)
    z = torch.randn(tokens * topk + 3, ld_z, generator=g).to(z_type)
    z[1] = math.nan  # a row that nobody has
    slots = torch.randperm(tokens * topk, generator=g).to(torch.int32).reshape(tokens, topk) + 3
    weights = torch.randn(tokens, topk, generator=g)
    gone = torch.rand(tokens, topk, generator=g) < 0.2
    gone[tokens // 2] = True  # a token without a row
    slots[gone] = -1
    weights[gone] = math.nan
    y = combine(plan, z, slots, weights, cols, y_type, ld_y)
    w = torch.where(gone, 0.0, weights.double())
    rows = z[slots.long().clamp(min=0) * ~gone + 3 * gone][..., :cols].double()
    terms = w[:, :, None] * rows
    ref = terms.sum(1)
    # topk fused additions of FP32 (2^-24 each), rounded once
    room = topk * 2.0 ** -24 * terms.abs().sum(1) + torch.finfo(y_type).eps / 2 * ref.abs()
    assert torch.all((y.double() - ref).abs() <= room)
    assert torch.all(y[tokens // 2] == 0)


def test_combine_slot_outside_sets_the_status(plan):
    z = torch.ones(4, 64)
    y = combine(plan, z, torch.tensor([[0, 4], [1, 2]], dtype=torch.int32), torch.ones(2, 2), 64, torch.float32,
                status=dfx.DFX_STATUS_INDEX)
    assert torch.all(y[0] == 1) and torch.all(y[1] == 2)
