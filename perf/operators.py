"""The operators around the grouped expert products, as cases to be timed and compared.

Kinds of case:

* ``route``        router logits -> expert ids, weights, group sizes and packed rows (softmax or
                   sigmoid scores, balance bias, expert groups, renormalisation)
* ``route_bwd``    gradient of the weights -> gradient of the logits
* ``dispatch``     token rows -> packed rows sorted by expert
* ``combine``      packed rows -> weighted token rows
* ``combine_bwd``  gradient of the token rows -> gradients of the packed rows and of the weights
* ``mxfp4``        bf16 rows -> 4-bit microscaled rows -> the values they stand for
* ``product4``     4-bit rows x 4-bit expert weights -> bf16
* ``ffn4``         bf16 tokens -> 4-bit packed rows -> up (SiLU-GLU) -> 4 bits -> down -> weighted tokens

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of
``expert_ffn_ragged_gb300``.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32                      # elements that share one scale
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # magnitudes of a 4-bit (E2M1) code
SOFTMAX, SIGMOID = 0, 1


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding token of a 128-expert layer: the smallest call, its latency
        dict(name="route 1x128 top8", kind="route", tokens=1, experts=128, topk=8, score=SOFTMAX,
             bias=False, groups=1, topk_groups=1, renorm=True, dtype="bf16", masked=0.0),
        # a prompt batch with padding tokens through a grouped, bias-balanced sigmoid router
        dict(name="route 32771x256 grouped", kind="route", tokens=32771, experts=256, topk=8,
             score=SIGMOID, bias=True, groups=8, topk_groups=4, renorm=True, dtype="f32",
             masked=0.03),
        # training step of a 128-expert router: probabilities of all experts take a gradient
        dict(name="route_bwd 65536x128 soft", kind="route_bwd", tokens=65536, experts=128, topk=8,
             score=SOFTMAX, renorm=False, dtype="f32"),
        # small fine-tuning batch, bf16 logits, renormalised sigmoid weights
        dict(name="route_bwd 509x256 sigm", kind="route_bwd", tokens=509, experts=256, topk=8,
             score=SIGMOID, renorm=True, dtype="bf16"),
        # the 225280-row packed buffer filled from its tokens
        dict(name="dispatch 28160x4096 top8", kind="dispatch", tokens=28160, experts=64, topk=8,
             hidden=4096),
        # a decoding batch of 16 tokens put together again
        dict(name="combine 16x4096 top8", kind="combine", tokens=16, experts=128, topk=8,
             hidden=4096, weighted=True),
        # a prompt's tokens after a top-2 layer
        dict(name="combine 16384x4096 top2", kind="combine", tokens=16384, experts=8, topk=2,
             hidden=4096, weighted=True),
        # training step over 126152 packed rows
        dict(name="combine_bwd 15769x4096 top8", kind="combine_bwd", tokens=15769, experts=64,
             topk=8, hidden=4096),
        # activations of a prompt to 4 bits and back
        dict(name="mxfp4 16381x4096", kind="mxfp4", rows=16381, width=4096),
        # one decoding token through a 128-expert layer in 4 bits: latency and 8 experts' weights
        dict(name="ffn4 1 token", kind="ffn4", tokens=1, experts=128, topk=8, hidden=4096, inner=768),
        # a decoding batch: almost every expert's weights are read
        dict(name="ffn4 256 tokens", kind="ffn4", tokens=256, experts=128, topk=8, hidden=4096,
             inner=768),
        # a prompt through one product of a top-2-of-8 layer: bound by the tensor cores
        dict(name="product4 32768x4096x14336", kind="product4", tokens=16384, experts=8, topk=2,
             width=4096, cols=14336),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; multiples of 3 move up by one, so
    that odd sizes and sizes that no tile divides are common."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n % 3 == 0)


def draw(rng):
    kind = rng.choice(["route", "route_bwd", "dispatch", "combine", "combine_bwd", "mxfp4",
                       "product4", "ffn4"])
    experts = rng.choice([8, 16, 64, 96, 128, 160, 256])
    topk = rng.randint(1, 8)
    tokens = _spread(rng, 1, 15000)
    hidden = 8 * _spread(rng, 8, 512)
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        topk_groups = rng.randint((groups + 1) // 2, groups)
        return dict(kind=kind, tokens=_spread(rng, 1, 30000), experts=experts,
                    topk=min(topk, experts // groups * topk_groups), score=rng.randint(0, 1),
                    bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups,
                    renorm=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]),
                    masked=rng.choice([0.0, 0.05]))
    if kind == "route_bwd":
        return dict(kind=kind, tokens=_spread(rng, 1, 30000), experts=experts, topk=topk,
                    score=rng.randint(0, 1), renorm=rng.random() < 0.5,
                    dtype=rng.choice(["f32", "bf16"]))
    if kind == "dispatch":
        return dict(kind=kind, tokens=tokens, experts=experts, topk=topk, hidden=hidden)
    if kind == "combine":
        return dict(kind=kind, tokens=tokens, experts=experts, topk=topk, hidden=hidden,
                    weighted=rng.random() < 0.7)
    if kind == "combine_bwd":
        return dict(kind=kind, tokens=tokens, experts=experts, topk=topk, hidden=hidden)
    if kind == "mxfp4":
        return dict(kind=kind, rows=tokens, width=32 * _spread(rng, 1, 128))
    if kind == "product4":
        return dict(kind=kind, tokens=_spread(rng, 1, 8192), experts=rng.choice([8, 16, 32]),
                    topk=rng.randint(1, 4), width=32 * _spread(rng, 4, 128),
                    cols=8 * _spread(rng, 8, 512))
    return dict(kind=kind, tokens=_spread(rng, 1, 2048), experts=rng.choice([8, 32, 64]), topk=topk,
                hidden=32 * _spread(rng, 4, 128), inner=32 * _spread(rng, 2, 40))


# ------------------------------------------------------------------------------------------ work
def _scales_width(k):
    """Bytes of one row's scales: one for each 32 elements, rounded up to 16."""
    return (k // BLOCK + 15) // 16 * 16


def work(case):
    c = case
    kind = c["kind"]
    if kind == "route":
        el = 4 if c["dtype"] == "f32" else 2
        n = c["tokens"] * c["topk"]
        return {"bytes": c["tokens"] * c["experts"] * el + 12 * n + 4 * c["experts"] + 4
                + (4 * c["experts"] if c["bias"] else 0), "flops": 4 * c["tokens"] * c["experts"]}
    if kind == "route_bwd":
        el = 4 if c["dtype"] == "f32" else 2
        n = c["tokens"] * c["topk"]
        dense = c["score"] == SOFTMAX and not c["renorm"]
        read = c["tokens"] * c["experts"] * el if dense else n * el
        return {"bytes": read + c["tokens"] * c["experts"] * el + 8 * n,
                "flops": 4 * c["tokens"] * c["experts"]}
    if kind in ("dispatch", "combine"):
        n = c["tokens"] * c["topk"]
        w = 4 * n if c.get("weighted") else 0
        return {"bytes": (c["tokens"] + n) * c["hidden"] * 2 + 4 * n + w,
                "flops": 2 * n * c["hidden"] if kind == "combine" else 0}
    if kind == "combine_bwd":
        n = c["tokens"] * c["topk"]
        return {"bytes": (c["tokens"] + 2 * n) * c["hidden"] * 2 + 12 * n, "flops": 3 * n * c["hidden"]}
    if kind == "mxfp4":
        # the bf16 rows in, the 4-bit rows out and in again, their values out
        n = c["rows"] * c["width"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // BLOCK), "flops": 2 * n}
    live = min(c["experts"], c["tokens"] * c["topk"])
    m = c["tokens"] * c["topk"]
    per = 0.5 + 1 / BLOCK
    if kind == "product4":
        return {"bytes": (m * c["width"] + live * c["width"] * c["cols"]) * per + m * c["cols"] * 2,
                "flops": 2 * m * c["width"] * c["cols"]}
    weights = live * 3 * c["hidden"] * c["inner"]
    return {"bytes": weights * per + 2 * c["tokens"] * c["hidden"] * 2 + 8 * m,
            "flops": 6 * m * c["hidden"] * c["inner"]}


# ------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _plan(g, tokens, experts, topk):
    """A router's choice with a mild preference for some experts, and the packed rows it gives."""
    logits = _normal(g, tokens, experts) + 0.5 * _normal(g, experts)
    ids = torch.topk(logits, topk, dim=1).indices.to(torch.int32)
    sizes, pos, rows = _sorted_rows(ids, experts)
    weights = torch.softmax(torch.gather(logits, 1, ids.long()), 1)
    return dict(ids=ids, group_sizes=sizes, pos=pos, rows=rows, weights=weights,
                most=int(sizes.max()))


def _weights4(g, experts, cols, width):
    """Expert weights [experts, cols, width] of variance 1 / width, packed to 4 bits."""
    q = torch.empty(experts, cols, width // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(experts, cols, _scales_width(width), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        codes, scales = _quantized(_normal(g, cols, width) / math.sqrt(width))
        q[e] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        s[e, :, : width // BLOCK] = scales
    return q, s


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    kind = c["kind"]
    if kind in ("route", "route_bwd"):
        t, e = c["tokens"], c["experts"]
        logits = 1.5 * _normal(g, t, e) + 0.5 * _normal(g, e)
        if c.get("masked"):
            # padding tokens have no expert at all; here and there an expert is switched off
            u = torch.rand(t, generator=g, device="cuda")
            logits[u < c["masked"]] = float("-inf")
            off = torch.rand(t, e, generator=g, device="cuda") < c["masked"] / 4
            logits[off] = float("-inf")
        c["logits"] = logits.to(torch.float32 if c["dtype"] == "f32" else torch.bfloat16)
        c["bias_t"] = 0.05 * _normal(g, e) if c.get("bias") else None
        if kind == "route_bwd":
            c["ids"] = torch.topk(c["logits"].float(), c["topk"], dim=1).indices.to(torch.int32)
            c["d_weights"] = _normal(g, t, c["topk"])
        return c
    if kind == "mxfp4":
        # rows of different size and a few outlying columns, as activations have
        x = _normal(g, c["rows"], c["width"]) * torch.exp(0.5 * _normal(g, c["rows"], 1))
        x = x * torch.where(torch.rand(c["width"], generator=g, device="cuda") < 0.01, 20.0, 1.0)
        c["x"] = x.to(torch.bfloat16)
        return c
    c.update(_plan(g, c["tokens"], c["experts"], c["topk"]))
    n = c["tokens"] * c["topk"]
    if kind == "dispatch":
        c["x"] = _normal(g, c["tokens"], c["hidden"]).to(torch.bfloat16)
    elif kind == "combine":
        c["y"] = _normal(g, n, c["hidden"]).to(torch.bfloat16)
    elif kind == "combine_bwd":
        c["y"] = _normal(g, n, c["hidden"]).to(torch.bfloat16)
        c["d_out"] = _normal(g, c["tokens"], c["hidden"]).to(torch.bfloat16)
    elif kind == "product4":
        codes, scales = _quantized(_normal(g, n, c["width"]))
        c["a_q"] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        c["a_s"] = torch.zeros(n, _scales_width(c["width"]), dtype=torch.uint8, device="cuda")
        c["a_s"][:, : c["width"] // BLOCK] = scales
        c["w_q"], c["w_s"] = _weights4(g, c["experts"], c["cols"], c["width"])
    else:
        c["x"] = _normal(g, c["tokens"], c["hidden"]).to(torch.bfloat16)
        c["up_q"], c["up_s"] = _weights4(g, c["experts"], 2 * c["inner"], c["hidden"])
        c["down_q"], c["down_s"] = _weights4(g, c["experts"], c["hidden"], c["inner"])
    return c


# ------------------------------------------------------------------------------------------ plain forms
def _chosen(logits, bias, topk, score, groups, topk_groups):
    """Expert ids of the chosen slots, best first, ties to the lowest index; -1 where none is left."""
    t, e = logits.shape
    none = torch.isnan(logits) | (logits == float("-inf"))
    key = logits if score == SOFTMAX else 1.0 / (1.0 + torch.exp(-logits))
    if bias is not None:
        key = key + bias
    low = torch.full((), float("-inf"), device=logits.device)
    key = torch.where(none, low, key)
    if groups > 1:
        by = torch.sort(key.view(t, groups, e // groups), dim=2, descending=True).values
        best = by[:, :, 0]
        if score == SIGMOID and e // groups > 1:
            second = by[:, :, 1]
            best = best + torch.where(second == low, torch.zeros_like(second), second)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        kept = torch.zeros(t, groups, dtype=torch.bool, device=logits.device).scatter(1, order, True)
        key = torch.where(kept.repeat_interleave(e // groups, 1), key, low)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(key[:, :topk] == low, -1, ids[:, :topk])


def _shares(logits, ids, score, renorm):
    """What each chosen expert gets: its score, or its share of the chosen scores. And 1 / their sum."""
    there = ids >= 0
    at = torch.gather(logits, 1, ids.clamp(min=0))
    zero = torch.zeros_like(at)
    if score == SOFTMAX:
        over = torch.where(there, at, float("-inf")) if renorm else \
            torch.where(torch.isnan(logits), float("-inf"), logits)
        top = over.amax(1, keepdim=True)
        top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
        total = torch.exp(over - top).sum(1, keepdim=True)
        part = torch.where(there, torch.exp(at - top), zero)
    else:
        part = torch.where(there, 1.0 / (1.0 + torch.exp(-at)), zero)
        total = part.sum(1, keepdim=True) if renorm else torch.ones_like(part[:, :1])
    inverse = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    return part, torch.where(total > 0, part / total, zero), inverse


def _sorted_rows(ids, experts):
    """Group sizes, the packed row of each slot (by expert, then by slot) and the number of rows."""
    flat = ids.reshape(-1).long()
    there = flat >= 0
    order = torch.argsort(torch.where(there, flat, experts), stable=True)
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(flat.numel(), device=flat.device)
    pos = torch.where(there, pos, -1).view(ids.shape).to(torch.int32)
    sizes = torch.zeros(experts, dtype=torch.int32, device=flat.device)
    sizes.index_add_(0, flat.clamp(min=0), there.to(torch.int32))
    return sizes, pos, there.sum().view(1).to(torch.int32)


def _route(s):
    logits = s["logits"].float()
    ids = _chosen(logits, s["bias_t"], s["topk"], s["score"], s["groups"], s["topk_groups"])
    weights = _shares(logits, ids, s["score"], s["renorm"])[1]
    sizes, pos, rows = _sorted_rows(ids, s["experts"])
    return [ids.to(torch.int32), weights, sizes, pos, rows]


def _route_bwd(s):
    logits, ids, d = s["logits"].float(), s["ids"].long(), s["d_weights"]
    part, share, inverse = _shares(logits, ids, s["score"], s["renorm"])
    mean = (share * d).sum(1, keepdim=True)
    if s["score"] == SOFTMAX and not s["renorm"]:
        top = logits.amax(1, keepdim=True)
        p = torch.exp(logits - top) * inverse
        out = (-p * mean).scatter_add(1, ids, share * d)
    else:
        if s["score"] == SOFTMAX:
            at = share * (d - mean)
        else:
            at = ((d - mean) * inverse if s["renorm"] else d) * part * (1.0 - part)
        out = torch.zeros_like(logits).scatter(1, ids, at)
    return out.to(s["logits"].dtype)


def _power(biased):
    """2^(biased - 127) as f32, exactly (built from its bits), for biased from 0 to 254."""
    bits = biased.to(torch.int32) << 23
    return torch.where(biased == 0, 0x00400000, bits).to(torch.int32).view(torch.float32)


def _quantized(x):
    """4-bit codes (one to a byte) and scale bytes of f32 rows, in blocks of 32 along the last axis."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    bits = blocks.abs().amax(-1, keepdim=True).view(torch.int32)
    exponent = ((bits >> 23) - 2).clamp(min=0)
    bad = ~torch.isfinite(blocks).all(-1, keepdim=True)
    exponent = torch.where(bad, 255, exponent)
    # x / 2^(exponent - 127), exactly: the factor is a power of two
    v = blocks * _power(254 - exponent.clamp(max=254))
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = torch.where(bad, 0, code | (torch.signbit(v).to(torch.uint8) << 3)).to(torch.uint8)
    return code.reshape(x.shape), exponent.squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """The f32 values of codes (one to a byte) and their blocks' scale bytes."""
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    factor = torch.where(scales == 255, float("nan"), _power(scales))
    v = table[codes.to(torch.int32)].view(*scales.shape, BLOCK) * factor.unsqueeze(-1)
    return v.reshape(codes.shape)


def _unpacked(q, s):
    codes = torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], 2 * q.shape[-1])
    return _values(codes, s[..., : codes.shape[-1] // BLOCK])


def _grouped(a, w, sizes, most):
    """Packed rows a times their own expert's w^T: each expert's rows padded to the longest group."""
    start = torch.cumsum(sizes, 0) - sizes
    lane = torch.arange(most, device=a.device)
    row = start.unsqueeze(1) + lane
    there = lane < sizes.unsqueeze(1)
    padded = a[torch.where(there, row, 0).long()] * there.unsqueeze(-1)
    out = torch.bmm(padded, w.transpose(1, 2))
    group = torch.repeat_interleave(torch.arange(sizes.numel(), device=a.device), sizes,
                                    output_size=a.shape[0])
    return out[group, torch.arange(a.shape[0], device=a.device) - start[group]]


def _combined(y, pos, weights):
    rows = y.float()[pos.long()]
    return (rows if weights is None else rows * weights.unsqueeze(-1)).sum(1)


def _plain(s):
    kind = s["kind"]
    if kind == "route":
        return _route(s)
    if kind == "route_bwd":
        return _route_bwd(s)
    if kind == "dispatch":
        out = torch.empty(s["pos"].numel(), s["hidden"], dtype=torch.bfloat16, device="cuda")
        out[s["pos"].long()] = s["x"].unsqueeze(1).expand(-1, s["topk"], -1)
        return out
    if kind == "combine":
        return _combined(s["y"], s["pos"], s["weights"] if s["weighted"] else None).to(torch.bfloat16)
    if kind == "combine_bwd":
        d, pos = s["d_out"].float(), s["pos"].long()
        d_y = torch.empty_like(s["y"])
        d_y[pos] = (d.unsqueeze(1) * s["weights"].unsqueeze(-1)).to(torch.bfloat16)
        return [d_y, (d.unsqueeze(1) * s["y"].float()[pos]).sum(-1)]
    if kind == "mxfp4":
        return _values(*_quantized(s["x"].float())).to(torch.bfloat16)
    if kind == "product4":
        out = _grouped(_unpacked(s["a_q"], s["a_s"]), _unpacked(s["w_q"], s["w_s"]),
                       s["group_sizes"], s["most"])
        return out.to(torch.bfloat16)
    x = _values(*_quantized(s["x"].float()))
    packed = torch.empty(s["pos"].numel(), s["hidden"], device="cuda")
    packed[s["pos"].long()] = x.unsqueeze(1).expand(-1, s["topk"], -1)
    fused = _grouped(packed, _unpacked(s["up_q"], s["up_s"]), s["group_sizes"], s["most"])
    gate, up = fused[:, : s["inner"]], fused[:, s["inner"]:]
    h = _values(*_quantized(gate / (1.0 + torch.exp(-gate)) * up))
    y = _grouped(h, _unpacked(s["down_q"], s["down_s"]), s["group_sizes"], s["most"])
    # the experts' rows are bf16, as every product of the framework leaves them
    return _combined(y.to(torch.bfloat16), s["pos"], s["weights"]).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if not own:
        return _plain(s)
    import expert_ffn_ragged_gb300 as rd

    kind = s["kind"]
    if kind == "route":
        r = rd.route(s["logits"], s["topk"], score=s["score"], bias=s["bias_t"], groups=s["groups"],
                     topk_groups=s["topk_groups"], renormalize=s["renorm"])
        return [r.ids, r.weights, r.group_sizes, r.pos, r.rows]
    if kind == "route_bwd":
        return rd.route_bwd(s["logits"], s["ids"], s["d_weights"], score=s["score"],
                            renormalize=s["renorm"])
    if kind == "dispatch":
        return rd.dispatch_rows(s["x"], s["pos"])
    if kind == "combine":
        return rd.combine_rows(s["y"], s["pos"], s["weights"] if s["weighted"] else None)
    if kind == "combine_bwd":
        return list(rd.combine_rows_bwd(s["d_out"], s["y"], s["pos"], s["weights"]))
    if kind == "mxfp4":
        return rd.mxfp4_dequantize(*rd.mxfp4_quantize(s["x"]))
    if kind == "product4":
        return rd.ragged_dot_mxfp4(s["a_q"], s["a_s"], s["w_q"], s["w_s"], s["group_sizes"])
    q, scales = rd.mxfp4_quantize(s["x"], pos=s["pos"])
    h, h_scales = rd.ragged_dot_mxfp4(q, scales, s["up_q"], s["up_s"], s["group_sizes"],
                                      epilogue=rd.EPI_SILU_GLU_MXFP4)
    y = rd.ragged_dot_mxfp4(h, h_scales, s["down_q"], s["down_s"], s["group_sizes"])
    return rd.combine_rows(y, s["pos"], s["weights"])


# ------------------------------------------------------------------------------------------ 64 bits
def _exact_values(x):
    """The values that f64 rows stand for once held in 4 bits, as a 64-bit array."""
    grid = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    blocks = x.reshape(-1, BLOCK)
    most = blocks.abs().amax(1, keepdim=True)
    exponent = torch.frexp(torch.where(most > 0, most, torch.ones_like(most))).exponent - 3
    scale = ((exponent.long() + 1023) << 52).view(torch.float64)
    v = blocks.abs() / scale
    # the nearest level; of two equally near ones, that with the even code
    far = (v.unsqueeze(-1) - grid).abs()
    odd = torch.arange(8, device=x.device) % 2
    code = torch.argmin(far + 1e-12 * odd, -1)
    return (torch.sign(blocks) * grid[code] * scale).reshape(x.shape)


def _exact_unpacked(q, s, width):
    grid = torch.tensor(LEVELS, dtype=torch.float64, device=q.device)
    out = torch.empty(*q.shape[:-1], width, dtype=torch.float64, device=q.device)
    for half in range(2):
        nibble = (q.long() >> (4 * half)) & 15
        out[..., half::2] = grid[nibble % 8] * (1 - 2 * (nibble // 8))
    exponent = s[..., : width // BLOCK].double() - 127
    return out * torch.exp2(exponent).repeat_interleave(BLOCK, -1)


def _exact_product(a, q, s, sizes, width):
    parts, at = [], 0
    for e, n in enumerate(sizes.tolist()):
        parts.append(a[at:at + n] @ _exact_unpacked(q[e], s[e], width).T)
        at += n
    return torch.cat(parts)


def _exact_shares(logits, ids, score, renorm):
    """f64 weights of the chosen experts of each token (rows of numpy arrays)."""
    there = ids >= 0
    at = np.take_along_axis(logits, np.maximum(ids, 0), 1)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == SOFTMAX:
            base = np.where(there, at, -np.inf) if renorm else logits
            top = base.max(1, keepdims=True)
            top = np.where(np.isfinite(top), top, 0.0)
            part = np.where(there, np.exp(at - top), 0.0)
            total = np.exp(base - top).sum(1, keepdims=True)
        else:
            part = np.where(there, 1 / (1 + np.exp(-at)), 0.0)
            total = part.sum(1, keepdims=True) if renorm else np.ones((len(at), 1))
        return part, np.where(total > 0, part / total, 0.0), total


def _exact_route(s):
    logits = s["logits"].double().cpu().numpy()
    t, e = logits.shape
    key = logits if s["score"] == SOFTMAX else 1 / (1 + np.exp(-logits))
    if s["bias_t"] is not None:
        key = key + s["bias_t"].double().cpu().numpy()
    key = np.where(np.isneginf(logits), -np.inf, key)
    size = e // s["groups"]
    if s["groups"] > 1:
        by = -np.sort(-key.reshape(t, s["groups"], size), axis=2)
        best = by[..., 0]
        if s["score"] == SIGMOID and size > 1:
            best = best + np.where(np.isneginf(by[..., 1]), 0.0, by[..., 1])
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat(rank < s["topk_groups"], size, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, : s["topk"]]
    ids = np.where(np.isneginf(np.take_along_axis(key, ids, 1)), -1, ids)
    weights = _exact_shares(logits, ids, s["score"], s["renorm"])[1]
    return [None, weights, None, None, None]


def _exact_route_bwd(s):
    logits, ids = s["logits"].double().cpu().numpy(), s["ids"].long().cpu().numpy()
    d = s["d_weights"].double().cpu().numpy()
    part, share, total = _exact_shares(logits, ids, s["score"], s["renorm"])
    out = np.zeros_like(logits)
    if s["score"] == SOFTMAX:
        # the Jacobian of a softmax over all experts, or over the chosen ones
        mean = (share * d).sum(1, keepdims=True)
        if not s["renorm"]:
            p = np.exp(logits - logits.max(1, keepdims=True))
            out -= p / p.sum(1, keepdims=True) * mean
            np.put_along_axis(out, ids, np.take_along_axis(out, ids, 1) + share * d, 1)
        else:
            np.put_along_axis(out, ids, share * (d - mean), 1)
    else:
        slope = part * (1 - part)
        if s["renorm"]:
            d = d / total - (part * d).sum(1, keepdims=True) / total ** 2
        np.put_along_axis(out, ids, d * slope, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "route":
        return _exact_route(s)
    if kind == "route_bwd":
        return _exact_route_bwd(s)
    if kind == "mxfp4":
        return torch.cat([_exact_values(x.double()) for x in s["x"].split(1024)])
    pos = s["pos"].long()
    if kind == "dispatch":
        out = torch.empty(pos.numel(), s["hidden"], dtype=torch.float64, device="cuda")
        for k in range(s["topk"]):
            out[pos[:, k]] = s["x"].double()
        return out
    if kind == "combine":
        out = torch.zeros(s["tokens"], s["hidden"], dtype=torch.float64, device="cuda")
        for k in range(s["topk"]):
            w = s["weights"][:, k:k + 1].double() if s["weighted"] else 1.0
            out += s["y"][pos[:, k]].double() * w
        return out
    if kind == "combine_bwd":
        d = s["d_out"].double()
        d_y = torch.empty(pos.numel(), s["hidden"], dtype=torch.float64, device="cuda")
        d_w = torch.empty(s["tokens"], s["topk"], dtype=torch.float64, device="cuda")
        for k in range(s["topk"]):
            d_y[pos[:, k]] = d * s["weights"][:, k:k + 1].double()
            d_w[:, k] = torch.einsum("th,th->t", d, s["y"][pos[:, k]].double())
        return [d_y, d_w]
    if kind == "product4":
        a = _exact_unpacked(s["a_q"], s["a_s"], s["width"])
        return _exact_product(a, s["w_q"], s["w_s"], s["group_sizes"], s["width"])
    tokens = torch.arange(s["tokens"], device="cuda").repeat_interleave(s["topk"])
    packed = torch.empty(pos.numel(), s["hidden"], dtype=torch.float64, device="cuda")
    packed[pos.reshape(-1)] = _exact_values(s["x"].double())[tokens]
    fused = _exact_product(packed, s["up_q"], s["up_s"], s["group_sizes"], s["hidden"])
    gate, up = fused.split(s["inner"], 1)
    h = _exact_values(gate * torch.sigmoid(gate) * up)
    y = _exact_product(h, s["down_q"], s["down_s"], s["group_sizes"], s["inner"])
    return (y[pos] * s["weights"].double().unsqueeze(-1)).sum(1)
