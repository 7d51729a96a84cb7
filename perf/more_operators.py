"""The rest of a feed-forward block around the experts, as cases to be timed and compared.

Kinds of case:

* ``norm``         layer norm of token rows, with or without the statistics that training keeps
* ``norm_bwd``     gradients of the rows, of the weight and of the bias
* ``linear``       rows x weights + bias -> activation -> + residual, dense or grouped by expert; training
                   also keeps the rows before the activation
* ``linear_bwd``   gradient of the output -> gradient before the activation, gradient of the bias
* ``dropout``      dropout by a counter-based generator, added to the residual; its gradient is the same
                   call without a residual

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the calls of
``expert_ffn_ragged_gb300``.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")     # by the number that the framework gives them
EPS = 1e-5
VEC = 8                          # elements that one call of the generator decides
STEPS = 65536                    # drop probabilities are multiples of 1 / STEPS
CUBIC = 0.044715                 # of the tanh form of gelu


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding token in front of its layer: the smallest call, its latency
        dict(name="norm 1x4096", kind="norm", rows=1, hidden=4096, dtype="bf16", out="bf16",
             stats=False, bias=True),
        # a training batch's residual stream, kept in f32, into bf16 products
        dict(name="norm 28157x4096 f32", kind="norm", rows=28157, hidden=4096, dtype="f32", out="bf16",
             stats=True, bias=True),
        # a small fine-tuning batch
        dict(name="norm_bwd 509x4096", kind="norm_bwd", rows=509, hidden=4096, dtype="bf16", out="bf16",
             bias=True),
        # the training batch's way back
        dict(name="norm_bwd 28157x4096 f32", kind="norm_bwd", rows=28157, hidden=4096, dtype="f32",
             out="bf16", bias=True),
        # one decoding token through the up projection of a dense feed-forward: weights at full speed
        dict(name="linear 1x4096x14336 gelu", kind="linear", rows=1, width=4096, cols=14336, experts=0,
             act="gelu", bias=True, residual=False, pre=False, out="bf16"),
        # a decoding batch through its down projection, onto the residual stream
        dict(name="linear 64x14336x4096 residual", kind="linear", rows=64, width=14336, cols=4096,
             experts=0, act="none", bias=True, residual=True, pre=False, out="bf16"),
        # a prompt batch's router logits in f32: few columns, bound by the tokens' bytes
        dict(name="linear 16381x4096x128 f32", kind="linear", rows=16381, width=4096, cols=128, experts=0,
             act="none", bias=True, residual=False, pre=False, out="f32"),
        # a training step's up projection of a top-2-of-8 layer with biases: bound by the tensor cores
        dict(name="linear 32768x4096x14336 g8 silu", kind="linear", rows=32768, width=4096, cols=14336,
             experts=8, act="silu", bias=True, residual=False, pre=True, out="bf16"),
        # the biases' and the activation's gradients of a small batch over many experts
        dict(name="linear_bwd 2048x1024 g64", kind="linear_bwd", rows=2048, cols=1024, experts=64,
             act="gelu_tanh", out="bf16"),
        # the same of a training step's dense feed-forward
        dict(name="linear_bwd 16384x14336 gelu", kind="linear_bwd", rows=16384, cols=14336, experts=0,
             act="gelu", out="bf16"),
        # a small batch's branch added to its residual
        dict(name="dropout 16x4096", kind="dropout", rows=16, hidden=4096, dtype="bf16", out="bf16", p=0.1,
             residual=True),
        # a training batch's branch added to the f32 residual stream
        dict(name="dropout 28157x4096 f32", kind="dropout", rows=28157, hidden=4096, dtype="bf16",
             out="f32", p=0.1, residual=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; multiples of 3 move up by one, so
    that odd sizes and sizes that no tile divides are common."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n % 3 == 0)


def draw(rng):
    kind = rng.choice(["norm", "norm_bwd", "linear", "linear", "linear_bwd", "dropout"])
    rows = _spread(rng, 1, 20000)
    hidden = 8 * _spread(rng, 8, 700)
    dtype, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if kind == "norm":
        return dict(kind=kind, rows=rows, hidden=hidden, dtype=dtype, out=out, stats=rng.random() < 0.5,
                    bias=rng.random() < 0.7)
    if kind == "norm_bwd":
        return dict(kind=kind, rows=rows, hidden=hidden, dtype=dtype, out=out, bias=rng.random() < 0.7)
    if kind == "dropout":
        return dict(kind=kind, rows=rows, hidden=hidden, dtype=dtype, out=out,
                    p=rng.choice([0.0, 0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.6)
    experts = rng.choice([0, 0, 4, 16, 64])
    act = rng.choice(ACTS)
    if kind == "linear_bwd":
        return dict(kind=kind, rows=rows, cols=hidden, experts=experts, act=act, out=out)
    return dict(kind=kind, rows=_spread(rng, 1, 12000), width=8 * _spread(rng, 8, 512),
                cols=8 * _spread(rng, 1, 512), experts=experts, act=act, bias=rng.random() < 0.8,
                residual=rng.random() < 0.4, pre=rng.random() < 0.4, out=out)


# ------------------------------------------------------------------------------------------ work
def work(case):
    c = case
    kind = c["kind"]
    out = SIZE[c["out"]]
    if kind in ("norm", "norm_bwd", "dropout"):
        n, el = c["rows"] * c["hidden"], SIZE[c["dtype"]]
        if kind == "norm":
            return {"bytes": n * (el + out) + 4 * c["hidden"] * (1 + c["bias"])
                    + (8 * c["rows"] if c["stats"] else 0), "flops": 8 * n}
        if kind == "norm_bwd":
            return {"bytes": n * (2 * el + out) + 4 * c["hidden"] * (2 + c["bias"]) + 8 * c["rows"],
                    "flops": 16 * n}
        return {"bytes": n * (el + out * (1 + c["residual"])), "flops": 3 * n}
    sizes = max(c["experts"], 1)
    n = c["rows"] * c["cols"]
    if kind == "linear_bwd":
        pre = 0 if c["act"] == "none" else 2
        return {"bytes": n * (out + pre + 2) + 4 * sizes * c["cols"], "flops": 10 * n}
    live = min(sizes, c["rows"])
    return {"bytes": 2 * c["rows"] * c["width"] + 2 * live * c["width"] * c["cols"]
            + (4 * live * c["cols"] if c["bias"] else 0)
            + n * (out * (1 + c["residual"]) + (2 if c["pre"] else 0)),
            "flops": 2 * n * c["width"]}


# ------------------------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, rows, hidden):
    """Rows of a residual stream: of different size, off zero, with a few outlying columns."""
    x = _normal(g, rows, hidden) * torch.exp(0.5 * _normal(g, rows, 1)) + 0.3 * _normal(g, rows, 1)
    return x * torch.where(torch.rand(hidden, generator=g, device="cuda") < 0.01, 10.0, 1.0)


def _sizes(g, rows, experts):
    """Rows of each expert as a router with mild preferences fills them (they add up to rows)."""
    if not experts:
        return None
    share = torch.softmax(0.5 * _normal(g, experts), 0)
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    return torch.bincount(pick, minlength=experts).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    kind = c["kind"]
    if kind in ("norm", "norm_bwd"):
        x = _stream(g, c["rows"], c["hidden"])
        c["x"] = x.to(TYPES[c["dtype"]])
        c["weight"] = 1.0 + 0.1 * _normal(g, c["hidden"])
        c["bias_t"] = 0.1 * _normal(g, c["hidden"]) if c["bias"] else None
        if kind == "norm_bwd":
            wide = c["x"].double()
            var, mean = torch.var_mean(wide, 1, correction=0)
            c["mean"], c["rstd"] = mean.float(), (1.0 / torch.sqrt(var + EPS)).float()
            c["d_out"] = _normal(g, c["rows"], c["hidden"]).to(TYPES[c["out"]])
        return c
    if kind == "dropout":
        c["x"] = _normal(g, c["rows"], c["hidden"]).to(TYPES[c["dtype"]])
        c["res"] = _stream(g, c["rows"], c["hidden"]).to(TYPES[c["out"]]) if c["residual"] else None
        c["rng"] = torch.randint(-2 ** 63, 2 ** 63 - 1, (2,), generator=g, device="cuda")
        return c
    rows, cols, experts = c["rows"], c["cols"], c["experts"]
    c["group_sizes"] = _sizes(g, rows, experts)
    c["most"] = int(c["group_sizes"].max()) if experts else rows
    if kind == "linear_bwd":
        c["d_out"] = _normal(g, rows, cols).to(TYPES[c["out"]])
        c["pre_t"] = None if c["act"] == "none" else (1.2 * _normal(g, rows, cols)).to(torch.bfloat16)
        return c
    width = c["width"]
    lead = (experts,) if experts else ()
    c["x"] = _normal(g, rows, width).to(torch.bfloat16)
    c["w"] = (_normal(g, *lead, width, cols) / math.sqrt(width)).to(torch.bfloat16)
    c["bias_t"] = 0.2 * _normal(g, *lead, cols) if c["bias"] else None
    c["res"] = _stream(g, rows, cols).to(TYPES[c["out"]]) if c["residual"] else None
    return c


# ------------------------------------------------------------------------------------------ plain forms
def _norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    off = x - mean
    rstd = 1.0 / torch.sqrt((off * off).mean(1, keepdim=True) + EPS)
    out = off * rstd * s["weight"]
    if s["bias_t"] is not None:
        out = out + s["bias_t"]
    out = out.to(TYPES[s["out"]])
    return [out, mean.squeeze(1), rstd.squeeze(1)] if s["stats"] else [out]


def _norm_bwd(s):
    d, rstd = s["d_out"].float(), s["rstd"].unsqueeze(1)
    at = (s["x"].float() - s["mean"].unsqueeze(1)) * rstd
    g = d * s["weight"]
    d_x = rstd * (g - g.mean(1, keepdim=True) - at * (g * at).mean(1, keepdim=True))
    grads = [d_x.to(s["x"].dtype), (d * at).sum(0)]
    return grads + [d.sum(0)] if s["bias"] else grads


def _logistic(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _activated(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return z * _logistic(2.0 * math.sqrt(2.0 / math.pi) * (z + CUBIC * z * z * z))
    return z * _logistic(z)


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        bell = torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * bell
    if act == "gelu_tanh":
        a = 2.0 * math.sqrt(2.0 / math.pi)
        sig = _logistic(a * (z + CUBIC * z * z * z))
        return sig + z * sig * (1.0 - sig) * a * (1.0 + 3.0 * CUBIC * z * z)
    sig = _logistic(z)
    return sig * (1.0 + z * (1.0 - sig))


def _group_of(sizes, rows):
    return torch.repeat_interleave(torch.arange(sizes.numel(), device=sizes.device), sizes, output_size=rows)


def _padded(a, sizes, most):
    """[groups, most, width]: each group's rows, the rest zero."""
    start = torch.cumsum(sizes, 0) - sizes
    lane = torch.arange(most, device=a.device)
    there = lane < sizes.unsqueeze(1)
    return a[torch.where(there, start.unsqueeze(1) + lane, 0).long()] * there.unsqueeze(-1)


def _linear(s):
    x, w, sizes = s["x"].float(), s["w"].float(), s["group_sizes"]
    if sizes is None:
        z = x @ w
        if s["bias_t"] is not None:
            z = z + s["bias_t"]
    else:
        z = torch.bmm(_padded(x, sizes, s["most"]), w)
        if s["bias_t"] is not None:
            z = z + s["bias_t"].unsqueeze(1)
        group = _group_of(sizes, x.shape[0])
        start = torch.cumsum(sizes, 0) - sizes
        z = z[group, torch.arange(x.shape[0], device=x.device) - start[group]]
    out = _activated(z, s["act"])
    if s["res"] is not None:
        out = out + s["res"].float()
    out = out.to(TYPES[s["out"]])
    return [out, z.to(torch.bfloat16)] if s["pre"] else [out]


def _linear_bwd(s):
    d = s["d_out"].float()
    if s["act"] != "none":
        d = d * _slope(s["pre_t"].float(), s["act"])
    if s["group_sizes"] is None:
        total = d.sum(0)
    else:
        total = _padded(d, s["group_sizes"], s["most"]).sum(1)
    return [d.to(torch.bfloat16), total]


def _high_low(a, b):
    """The high and low 32 bits of the product of 32-bit numbers held in int64 (b: a number)."""
    low = (a & 0xFFFF) * b                                   # below 2^48
    top = (a >> 16) * b + (low >> 16)                        # below 2^49
    return top >> 16, ((top & 0xFFFF) << 16) | (low & 0xFFFF)


def _words(rng, vectors):
    """The four 32-bit words that the generator (Philox 4x32 in ten rounds; Salmon et al., 2011) gives
    for each vector of elements: key = the seed, counter = the vector's index and the offset."""
    mask = 0xFFFFFFFF
    index = torch.arange(vectors, device=rng.device)
    c0, c1 = index & mask, index >> 32
    c2, c3 = (rng[1] & mask).expand_as(c0), ((rng[1] >> 32) & mask).expand_as(c0)
    k0, k1 = rng[0] & mask, (rng[0] >> 32) & mask
    for _ in range(10):
        h0, l0 = _high_low(c0, 0xD2511F53)
        h1, l1 = _high_low(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    return torch.stack((c0, c1, c2, c3), 1)


def _dropout(s):
    x = s["x"].float()
    least = int(math.floor(s["p"] * STEPS + 0.5))
    words = _words(s["rng"], x.numel() // VEC)
    draws = torch.stack((words & 0xFFFF, words >> 16), 2).view(x.shape)
    scale = STEPS / (STEPS - least) if least < STEPS else 0.0
    out = torch.where(draws >= least, x * scale, torch.zeros_like(x))
    if s["res"] is not None:
        out = out + s["res"].float()
    return [out.to(TYPES[s["out"]])]


def _plain(s):
    return {"norm": _norm, "norm_bwd": _norm_bwd, "linear": _linear, "linear_bwd": _linear_bwd,
            "dropout": _dropout}[s["kind"]](s)


# ------------------------------------------------------------------------------------------ one pass
def run(state):
    s = state
    if not own:
        return _plain(s)
    import expert_ffn_ragged_gb300 as rd

    kind = s["kind"]
    out = TYPES[s["out"]]
    if kind == "norm":
        r = rd.layer_norm_fwd(s["x"], s["weight"], s["bias_t"], eps=EPS, out_dtype=out, stats=s["stats"])
        return [r.out, r.mean, r.rstd] if s["stats"] else [r.out]
    if kind == "norm_bwd":
        d_x, d_weight, d_bias = rd.layer_norm_bwd(s["d_out"], s["x"], s["weight"], s["mean"], s["rstd"],
                                                  need_bias=s["bias"])
        return [d_x, d_weight, d_bias] if s["bias"] else [d_x, d_weight]
    if kind == "dropout":
        return [rd.dropout_rows(s["x"], s["rng"], s["p"], residual=s["res"], out_dtype=out)]
    act = ACTS.index(s["act"])
    if kind == "linear_bwd":
        return list(rd.linear_act_bwd(s["d_out"], s["pre_t"], act, group_sizes=s["group_sizes"]))
    r = rd.linear(s["x"], s["w"], s["bias_t"], residual=s["res"], act=act, group_sizes=s["group_sizes"],
                  out_dtype=out, save_pre=s["pre"])
    return list(r) if s["pre"] else [r]


# ------------------------------------------------------------------------------------------ 64 bits
def _exact_act(z, act):
    if act == "relu":
        return torch.relu(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + CUBIC * z ** 3)))
    return z * torch.sigmoid(z) if act == "silu" else z


def _exact_slope(z, act):
    """The derivative of the activation, by automatic differentiation of its definition."""
    at = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(_exact_act(at, act).sum(), at)[0]


def _bounds(sizes, rows):
    ends = [rows] if sizes is None else np.cumsum(sizes.cpu().numpy()).tolist()
    return list(zip([0] + ends[:-1], ends))


def _exact_words(seed, offset, lo, hi):
    """Words of the vectors [lo, hi), with numpy's 64-bit products."""
    u = np.uint64
    low, shift = u(0xFFFFFFFF), u(32)
    index = np.arange(lo, hi, dtype=np.uint64)
    c = [index & low, index >> shift, np.full_like(index, offset & 0xFFFFFFFF), np.full_like(index, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = u(0xD2511F53) * c[0], u(0xCD9E8D57) * c[2]
        c = [(b >> shift) ^ c[1] ^ u(k[0]), b & low, (a >> shift) ^ c[3] ^ u(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, 1).astype(np.uint32)


def _exact_dropout(s):
    seed, offset = (int(v) % 2 ** 64 for v in s["rng"].tolist())
    least = int(math.floor(s["p"] * STEPS + 0.5))
    out = torch.empty(s["rows"], s["hidden"], dtype=torch.float64, device="cuda")
    per = s["hidden"] // VEC
    for r in range(0, s["rows"], 4096):
        part = s["x"][r:r + 4096].double()
        words = _exact_words(seed, offset, r * per, r * per + part.numel() // VEC)
        kept = words.astype("<u4").view("<u2") >= least
        kept = torch.from_numpy(kept.reshape(part.shape)).to("cuda")
        part = part * kept * (STEPS / (STEPS - least))
        out[r:r + 4096] = part if s["res"] is None else part + s["res"][r:r + 4096].double()
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "dropout":
        return _exact_dropout(s)
    if kind == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        out = (x - mean) / torch.sqrt(var + EPS) * s["weight"].double()
        if s["bias_t"] is not None:
            out += s["bias_t"].double()
        return [out, mean.squeeze(1), (var + EPS).rsqrt().squeeze(1)] if s["stats"] else [out]
    if kind == "norm_bwd":
        # the Jacobian of a normalised row takes out its components along 1 and along the row itself
        d, r = s["d_out"].double(), s["rstd"].double().unsqueeze(1)
        at = (s["x"].double() - s["mean"].double().unsqueeze(1)) * r
        g = d * s["weight"].double()
        dots = torch.einsum("rh,rh->r", g, at).unsqueeze(1)
        d_x = (g * s["hidden"] - g.sum(1, keepdim=True) - at * dots) * r / s["hidden"]
        both = [d_x, torch.einsum("rh,rh->h", d, at)]
        return both + [torch.einsum("rh->h", d)] if s["bias"] else both
    spans = _bounds(s["group_sizes"], s["rows"])
    if kind == "linear_bwd":
        d = s["d_out"].double()
        if s["act"] != "none":
            d = d * _exact_slope(s["pre_t"].double(), s["act"])
        total = torch.stack([d[lo:hi].sum(0) for lo, hi in spans])
        return [d, total if s["experts"] else total[0]]
    parts = []
    for j, (lo, hi) in enumerate(spans):
        w, b = (s["w"], s["bias_t"]) if not s["experts"] else (s["w"][j], None if s["bias_t"] is None else s["bias_t"][j])
        z = s["x"][lo:hi].double() @ w.double()
        parts.append(z if b is None else z + b.double())
    z = torch.cat(parts)
    out = _exact_act(z, s["act"])
    if s["res"] is not None:
        out = out + s["res"].double()
    return [out, z] if s["pre"] else [out]
