"""The operators of a mixture-of-experts layer with 8-bit weights, as cases to be timed and checked.

  route     dfx_route:        gate logits -> experts, weights, and the assignments sorted by expert
  quantize  dfx_quantize_fp8: BF16 -> e4m3 with a power-of-two scale for each 1x128 or 128x128 block
  gemm      dfx_gemm_fp8:     y = x w^T on such operands, with one matrix or one per expert
  combine   dfx_combine:      the weighted sum of a token's rows over the experts it went to

Where `own` is false, `run` computes them with elementary torch operations.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a small batch: latency is all that counts
        dict(name="route_step", op="route", tokens=4, experts=64, topk=6, score="softmax", bias=False, groups=1,
             top_groups=1, best=1, renorm=False, bf16=True, masked=0.0),
        # a prefill batch, grouped sigmoid gate with a balance bias, an eighth of the rows padding
        dict(name="route_grouped", op="route", tokens=4096, experts=256, topk=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renorm=True, bf16=False, masked=0.125),
        # the largest batch, plain softmax gate, a ragged number of tokens
        dict(name="route_long", op="route", tokens=32749, experts=128, topk=8, score="softmax", bias=False, groups=1,
             top_groups=1, best=1, renorm=True, bf16=True, masked=0.0),
        # activations of one decoding step in front of a 4096-wide projection
        dict(name="quantize_step", op="quantize", rows=16, cols=4096, blocks=1, swiglu=False, gather=False),
        # the gate projection of the 8B-shaped layer, restored from its container and laid out once
        dict(name="quantize_weights", op="quantize", rows=14336, cols=4096, blocks=128, swiglu=False, gather=False),
        # between an expert layer's two products: SwiGLU and its quantization, an odd width
        dict(name="quantize_swiglu", op="quantize", rows=8195, cols=14320, blocks=1, swiglu=True, gather=False),
        # one token through the gate projection: every weight is read for two operations
        dict(name="gemm_token", op="gemm", tokens=1, rows=14336, cols=4096, experts=1, fp32=False),
        # a decoding step over experts: 16 tokens x 8, most experts with a few tokens, some with none
        dict(name="gemm_experts_step", op="gemm", tokens=128, rows=2048, cols=4096, experts=128, fp32=False),
        # a prefill chunk over experts, ragged, rows past the last one unused; FP32 output
        dict(name="gemm_experts", op="gemm", tokens=16384, rows=4096, cols=2048, experts=32, fp32=True),
        # a long prefill through the gate projection: the tensor cores bound it
        dict(name="gemm_prefill", op="gemm", tokens=8192, rows=14336, cols=4096, experts=1, fp32=False),
        # the way back, one decoding step
        dict(name="combine_step", op="combine", tokens=16, topk=8, cols=4096, fp32=False, missing=0.0),
        # the way back of a prefill chunk, some assignments dropped
        dict(name="combine_long", op="combine", tokens=8191, topk=8, cols=4096, fp32=False, missing=0.05),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "quantize", "gemm", "gemm", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = log(4, 512 // groups)
        experts = groups * per
        top_groups = rng.randint(1, groups)
        topk = rng.randint(1, min(16, top_groups * per))
        return dict(op=op, tokens=log(1, 32749), experts=experts, topk=topk, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, best=rng.choice([1, 2]),
                    renorm=rng.random() < 0.5, bf16=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1, 0.3]))
    if op == "quantize":
        swiglu = rng.random() < 0.33
        blocks = 1 if swiglu else rng.choice([1, 128])
        return dict(op=op, rows=log(1, 8195), cols=log(64, 14320), blocks=blocks, swiglu=swiglu,
                    gather=blocks == 1 and not swiglu and rng.random() < 0.5)
    if op == "gemm":
        experts = rng.choice([1, 1, log(2, 64)])
        most = 8192 if experts == 1 else 4096
        rows, cols = log(100, most), log(100, most)
        return dict(op=op, tokens=log(1, 8192), rows=rows, cols=cols, experts=experts, fp32=rng.random() < 0.3)
    return dict(op=op, tokens=log(1, 8191), topk=rng.randint(1, 8), cols=log(64, 4096), fp32=rng.random() < 0.5,
                missing=rng.choice([0.0, 0.05, 0.5]))


# ---------------------------------------------------------------- sizes

def up(x, to):
    return -(-x // to) * to


def expert_counts(case):
    """Rows of each expert, most first: a skewed share of all but a thirty-second of the rows, which stay unused."""
    total, experts = case["tokens"], case["experts"]
    if experts == 1:
        return [total]
    used = total - total // 32
    share = [(i + 1.0) ** -0.7 for i in range(experts)]
    edge, counts, before = 0.0, [], 0
    for s in share:
        edge += s
        now = int(used * (edge / sum(share)) + 0.5)
        counts.append(now - before)
        before = now
    return counts


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + (4 * e if case["bias"] else 0) + 16 * t * k + 4 * (e + 1),
                "flops": 4 * t * e}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["blocks"]) * -(-case["cols"] // BLOCK)
        return {"bytes": n * (4 if case["swiglu"] else 2) + n + scales, "flops": (8 if case["swiglu"] else 3) * n}
    if op == "gemm":
        counts = expert_counts(case)
        used, hit, r, c = sum(counts), sum(n > 0 for n in counts), case["rows"], case["cols"]
        scales = used * -(-c // BLOCK) + hit * -(-r // BLOCK) * -(-c // BLOCK)
        return {"bytes": used * c + hit * r * c + scales + used * r * (4 if case["fp32"] else 2),
                "flops": 2 * used * r * c}
    t, k, c = case["tokens"], case["topk"], case["cols"]
    kept = t * k * (1 - case["missing"])
    return {"bytes": int(kept * c * 2) + t * c * (4 if case["fp32"] else 2) + 8 * t * k, "flops": int(2 * kept * c)}


# ---------------------------------------------------------------- inputs

def power_of_two(e):
    """2^e in 64 bits, built from its exponent's bits (pow and exp2 are rounded)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def quantized(x, block_rows):
    """e4m3 values and e8m0 scale bytes of x [..., rows, cols]: per block the smallest power of two that brings the
    largest finite magnitude to 448 or below."""
    rows, cols = x.shape[-2:]
    padded = torch.nn.functional.pad(x, (0, up(cols, BLOCK) - cols, 0, up(rows, block_rows) - rows))
    blocks = padded.reshape(*x.shape[:-2], -1, block_rows, up(cols, BLOCK) // BLOCK, BLOCK)
    amax = torch.where(torch.isfinite(blocks), blocks, 0.0).abs().amax(dim=(-3, -1))
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax == 0, 0, torch.clamp(exponent - 9 + (mantissa > 0.875).int(), -127, 127))
    q = blocks * power_of_two(-e)[..., :, None, :, None].to(x.dtype)
    q = q.reshape(padded.shape)[..., :rows, :cols].to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def strided(x, to):
    """x [..., n] in rows padded with bytes of no meaning to a multiple of `to`."""
    room = torch.full((*x.shape[:-1], up(x.shape[-1], to)), 0x7F, dtype=torch.uint8, device=x.device)
    room[..., :x.shape[-1]] = x.view(torch.uint8)
    return room


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    op = case["op"]
    st = dict(case)
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        # a gate's logits: each token its own, some experts liked by most
        logits = 1.5 * normal(t, e) + 0.5 * normal(1, e)
        if case["masked"]:
            logits[uniform(t) < case["masked"]] = -math.inf         # padding
            logits[uniform(t, e) < 0.25 * case["masked"]] = -math.inf  # experts closed to a token
        st["logits"] = logits.to(torch.bfloat16 if case["bf16"] else torch.float32)
        st["bias"] = 0.1 * normal(e) if case["bias"] else None
    elif op == "quantize":
        r, c = case["rows"], case["cols"]
        if case["blocks"] == 1:
            # activations: a few channels far larger than the others
            x = normal(r, 2 * c if case["swiglu"] else c) * torch.exp(0.5 * normal(1, 2 * c if case["swiglu"] else c))
        else:
            # weights: N(0, 1/cols) with rare large ones
            x = normal(r, c) / math.sqrt(c)
            x = torch.where(uniform(r, c) < 5e-4, 0.5 * normal(r, c), x)
        st["x"] = x.to(torch.bfloat16)
        # rows in the order of the experts they go to; the last slots of a batch may be unused
        st["index"] = torch.randint(0, r, (r,), generator=gen, device=DEV, dtype=torch.int32) if case["gather"] else None
    elif op == "gemm":
        t, r, c, e = case["tokens"], case["rows"], case["cols"], case["experts"]
        xq, sx = quantized(normal(t, c) * torch.exp(0.5 * normal(1, c)), 1)
        wq, sw = quantized(normal(e, r, c) / math.sqrt(c), BLOCK)
        st["x"], st["sx"], st["w"], st["sw"] = strided(xq, 16), strided(sx, 4), strided(wq, 16), strided(sw, 4)
        counts = torch.tensor(expert_counts(case), device=DEV)[torch.randperm(e, generator=gen, device=DEV)]
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32) if e > 1 else None
        st["most"] = max(expert_counts(case))  # a bound that a caller has: no expert gets more rows
        # rows that no expert has stay as they are
        st["y"] = torch.zeros(t, r, device=DEV, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
    else:
        t, k, c = case["tokens"], case["topk"], case["cols"]
        st["z"] = normal(t * k, c).to(torch.bfloat16)
        st["weights"] = torch.softmax(normal(t, k), dim=1)
        slots = torch.randperm(t * k, generator=gen, device=DEV).to(torch.int32).reshape(t, k)
        st["slots"] = torch.where(uniform(t, k) < case["missing"], -1, slots)
    if own:
        prepare_own(st)
    return st


def prepare_own(st):
    """The plan and the buffers that a program keeps beside its inputs."""
    import lossless_entropy_coded_exponent_b200 as dfx

    def ints(*shape):
        return torch.empty(*shape, device=DEV, dtype=torch.int32)

    op = st["op"]
    st["dfx"] = dfx
    st["plan"] = dfx.dfx_plan(0)
    if op == "route":
        t, e, k = st["tokens"], st["experts"], st["topk"]
        st["params"] = dfx.dfx_route_params(
            score=dfx.DFX_SCORE_SOFTMAX if st["score"] == "softmax" else dfx.DFX_SCORE_SIGMOID, topk=k,
            groups=st["groups"], top_groups=st["top_groups"], group_best=st["best"], renormalize=int(st["renorm"]),
            scale=1.0)
        st["out"] = [ints(t, k), torch.empty(t, k, device=DEV), ints(e + 1), ints(t * k), ints(t, k)]
        st["workspace"] = torch.empty(dfx.dfx_route_workspace(t, e, st["params"]), device=DEV, dtype=torch.uint8)
    elif op == "quantize":
        r, c = st["rows"], st["cols"]
        q = torch.empty(r, up(c, 16), device=DEV, dtype=torch.uint8)
        s = torch.empty(-(-r // st["blocks"]), up(-(-c // BLOCK), 4), device=DEV, dtype=torch.uint8)
        st["out"] = [q, s]
        st["values"] = [q[:, :c].view(torch.float8_e4m3fn), s[:, :-(-c // BLOCK)].view(torch.float8_e8m0fnu)]
    elif op == "combine":
        st["y"] = torch.empty(st["tokens"], st["cols"], device=DEV, dtype=torch.float32 if st["fp32"] else torch.bfloat16)


# ---------------------------------------------------------------- one pass

def run(st):
    if own:
        return run_own(st)
    return {"route": route, "quantize": quantize, "gemm": gemm, "combine": combine}[st["op"]](st)


def run_own(st):
    dfx, plan, op = st["dfx"], st["plan"], st["op"]
    if op == "route":
        x = st["logits"]
        dfx.dfx_route(plan, x, dfx.DFX_BF16 if st["bf16"] else dfx.DFX_F32, st["experts"], st["tokens"], st["experts"],
                      st["bias"], st["params"], *st["out"], st["workspace"], st["workspace"].numel())
        return st["out"]
    if op == "quantize":
        q, s = st["out"]
        x = st["x"]
        dfx.dfx_quantize_fp8(plan, x, dfx.DFX_BF16, x.shape[1], x.shape[0], st["index"], st["rows"], st["cols"],
                             st["blocks"], dfx.DFX_QUANT_SWIGLU if st["swiglu"] else 0, q, q.shape[1], s, s.shape[1])
        return st["values"]
    if op == "gemm":
        x, sx, w, sw, y = st["x"], st["sx"], st["w"], st["sw"], st["y"]
        dfx.dfx_gemm_fp8(plan, x, x.shape[-1], sx, sx.shape[-1], st["tokens"], w, w.shape[-1], sw, sw.shape[-1],
                         st["rows"], st["cols"], st["experts"], st["offsets"], y, dfx.DFX_F32 if st["fp32"] else dfx.DFX_BF16,
                         st["rows"])
        return y
    z, y = st["z"], st["y"]
    dfx.dfx_combine(plan, z, dfx.DFX_BF16, st["cols"], z.shape[0], st["cols"], st["slots"], st["weights"], st["tokens"],
                    st["topk"], y, dfx.DFX_F32 if st["fp32"] else dfx.DFX_BF16, st["cols"])
    return y


def route(st):
    e, k, groups = st["experts"], st["topk"], st["groups"]
    logits = st["logits"].double()  # the order of near scores would change in 32 bits
    t = logits.shape[0]
    lowest = -math.inf
    open_ = logits > lowest
    if st["score"] == "softmax":
        shifted = torch.where(open_, logits - torch.where(open_, logits, lowest).amax(1, keepdim=True), lowest)
        scores = torch.exp(shifted)
        scores = torch.where(open_, scores / scores.sum(1, keepdim=True), 0.0)
    else:
        scores = torch.where(open_, 1.0 / (1.0 + torch.exp(-logits)), 0.0)
    by_score = st["bias"] is not None or (groups > 1 and st["best"] == 2)
    choice = scores + (st["bias"].double() if st["bias"] is not None else 0.0) if by_score else logits
    choice = torch.where(open_, choice, lowest)
    if groups > 1:
        # a group's score: its best choices summed, of a group with fewer those that it has
        best = torch.sort(choice.reshape(t, groups, -1), dim=2, descending=True).values[:, :, :st["best"]]
        none = best[:, :, 0] == lowest
        group = torch.where(none, lowest, torch.where(best == lowest, 0.0, best).sum(2))
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :st["top_groups"]]
        inside = torch.zeros(t, groups, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        choice = torch.where(inside.repeat_interleave(e // groups, 1), choice, lowest)
    order = torch.sort(choice, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] > lowest, order.indices[:, :k], -1)
    weights = torch.where(ids >= 0, torch.gather(scores, 1, ids.clamp(min=0)), 0.0)
    if st["renorm"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0.0)
    # the assignments by expert, then by token
    flat = torch.where(ids >= 0, ids, e).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(e + 1, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts[:e].cumsum(0)])
    place = torch.arange(t * k, device=DEV)
    slots = torch.empty_like(order).scatter_(0, order, place)
    slots = torch.where(flat < e, slots, -1).reshape(t, k)
    rows = torch.where(place < offsets[e], order // k, -1)
    return [ids.int(), weights.float(), offsets.int(), rows.int(), slots.int()]


def quantize(st):
    x = st["x"].float() if st["index"] is None else st["x"][st["index"].long()].float()
    if st["swiglu"]:
        # in 64 bits: a block's largest value may stand next to a power of two's border
        gate, value = x[:, :st["cols"]].double(), x[:, st["cols"]:].double()
        x = gate / (1.0 + torch.exp(-gate)) * value
    q, scales = quantized(x, st["blocks"])
    return [q, scales.view(torch.float8_e8m0fnu)]


def dequantized(q, scales, cols, block_rows):
    rows = q.shape[-2]
    values = q[..., :cols].view(torch.float8_e4m3fn).float()
    s = power_of_two(scales[..., :-(-cols // BLOCK)].int() - 127).float()
    return values * s.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def gemm(st):
    r, c, e, most = st["rows"], st["cols"], st["experts"], st["most"]
    x = dequantized(st["x"], st["sx"], c, 1)
    w = dequantized(st["w"], st["sw"], c, BLOCK)
    if e == 1:
        return (x @ w[0].T).to(st["y"].dtype)
    # each expert's rows beside one another, short ones filled up with a row of zeros
    begin, end = st["offsets"][:-1].long(), st["offsets"][1:].long()
    at = begin[:, None] + torch.arange(most, device=DEV)
    at = torch.where(at < end[:, None], at, st["tokens"])
    x = torch.cat([x, x.new_zeros(1, c)])
    z = torch.bmm(x[at], w.transpose(1, 2))
    y = torch.zeros(st["tokens"] + 1, r, device=DEV)
    y[at.reshape(-1)] = z.reshape(-1, r)
    return y[:-1].to(st["y"].dtype)


def combine(st):
    slots = st["slots"].long()
    weights = torch.where(slots >= 0, st["weights"], 0.0)
    z = st["z"][slots.clamp(min=0)].float()
    y = (weights[:, :, None] * z).sum(1)
    return y.to(torch.float32 if st["fp32"] else torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"route": exact_route, "quantize": exact_quantize, "gemm": exact_gemm, "combine": exact_combine}[case["op"]](st)


def exact_route(st):
    """The weights by the definition, at the experts that sorting its scores gives."""
    e, k, g = st["experts"], st["topk"], st["groups"]
    x = st["logits"].to(torch.float64)
    t = x.shape[0]
    closed = torch.isneginf(x)
    score = torch.softmax(x, 1).nan_to_num(0.0) if st["score"] == "softmax" else torch.sigmoid(x)
    score[closed] = 0.0
    key = x.clone()
    if st["bias"] is not None or (g > 1 and st["best"] == 2):
        key = score + (0 if st["bias"] is None else st["bias"].to(torch.float64))
        key[closed] = -math.inf
    if g > 1:
        top = key.view(t, g, e // g).topk(min(st["best"], e // g), dim=2).values
        worth = top[:, :, 0].clone()
        if st["best"] == 2 and e // g > 1:
            worth += top[:, :, 1].clamp(min=-1e300).where(~torch.isneginf(top[:, :, 1]), torch.zeros(()).double().to(DEV))
        rank = torch.argsort(torch.argsort(-worth, dim=1, stable=True), dim=1, stable=True)
        key[(rank >= st["top_groups"]).repeat_interleave(e // g, 1)] = -math.inf
    picked = torch.argsort(-key, dim=1, stable=True)[:, :k]
    weight = torch.gather(score, 1, picked) * (~torch.isneginf(torch.gather(key, 1, picked)))
    if st["renorm"]:
        weight = (weight / weight.sum(1, keepdim=True)).nan_to_num(0.0)
    return [None, weight, None, None, None]


def exact_quantize(st):
    """The scaled values before they are rounded, and the scales."""
    x = st["x"].to(torch.float64)
    if st["index"] is not None:
        x = x.index_select(0, st["index"])
    c, b = st["cols"], st["blocks"]
    if st["swiglu"]:
        x = torch.nn.functional.silu(x[:, :c]) * x[:, c:]
    tall, wide = up(x.shape[0], b), up(c, BLOCK)
    full = torch.zeros(tall, wide, dtype=torch.float64, device=DEV)
    full[:x.shape[0], :c] = x
    full = full.view(tall // b, b, wide // BLOCK, BLOCK)
    peak = full.abs().amax(3).amax(1)
    peak = torch.where(peak > 0, peak, E4M3_MAX)
    e = torch.round(torch.log2(peak / E4M3_MAX)) - 1
    for _ in range(2):  # the logarithm is rounded: the border itself is compared
        e += E4M3_MAX * power_of_two(e) < peak
    scale = power_of_two(e)
    values = (full / scale[:, None, :, None]).view(tall, wide)[:x.shape[0], :c]
    return [values, scale]


def exact_gemm(st):
    c, e = st["cols"], st["experts"]

    def values(q, s, tall):
        v = q[..., :c].view(torch.float8_e4m3fn).to(torch.float64)
        factor = power_of_two(s.to(torch.int64) - 127)
        i = torch.arange(v.shape[-2], device=DEV) // tall
        j = torch.arange(c, device=DEV) // BLOCK
        return v * factor[..., i, :][..., j]

    x = values(st["x"], st["sx"], 1)
    y = torch.zeros(st["tokens"], st["rows"], dtype=torch.float64, device=DEV)
    edges = [0, st["tokens"]] if e == 1 else st["offsets"].tolist()
    for i in range(e):
        if edges[i + 1] > edges[i]:
            y[edges[i]:edges[i + 1]] = x[edges[i]:edges[i + 1]] @ values(st["w"][i], st["sw"][i], BLOCK).T
    return y


def exact_combine(st):
    y = torch.zeros(st["tokens"], st["cols"], dtype=torch.float64, device=DEV)
    for k in range(st["topk"]):
        slot = st["slots"][:, k]
        here = (slot >= 0).nonzero()[:, 0]
        y[here] += st["weights"][here, k].to(torch.float64)[:, None] * st["z"][slot[here].long()].to(torch.float64)
    return y
