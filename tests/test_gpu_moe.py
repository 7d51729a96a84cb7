"""Routing, sorting, dispatch / combine on the GPU against the float64 oracle.

Tolerances (fixed from the arithmetic, u = 2^-24):

* ids, group sizes, positions: exact.  Logits lie on a grid of 1/8 and biases on one of 1/4, so that
  softmax keys are exact in f32; sigmoid keys are f32 values within 2^-22 of the float64 ones, so
  there the chosen keys must be the best ones within that margin, in order.
* weights: the argument of exp is off by u |l - max|, exp itself by 2 ulp, the sums of at most 42
  roundings, the quotient and the scale by one each: relative 2^-23 (48 + 2 max|l|).
* gradients: the same factor on scale (|d_j| + sum_k |q_k d_k|) times what multiplies it, and for
  1 - s an absolute u more; bf16 output adds half an ulp, 2^-8 relative.
* combine: (topk + 1) u sum|w y| and the bf16 rounding, 2^-8 relative.
* d_y: bit for bit; d_w: gamma_n sum|d y| for n products in any order.
"""
import numpy as np
import pytest

from oracle import bf16 as obf
from oracle import moe, unsort

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _grid_logits(rng, tokens, experts, masked, dtype):
    l = np.round(rng.normal(size=(tokens, experts)) * 1.5 * 8) / 8
    if masked:
        l[rng.random((tokens, experts)) < 0.15] = -np.inf
        l[rng.random((tokens, experts)) < 0.02] = np.nan
        l[rng.random(tokens) < 0.1] = -np.inf          # tokens without any expert
    return torch.from_numpy(l.astype(np.float32)).to(dtype)


def _check_weights(got, l, ids, score, renorm, scale):
    for t in range(len(ids)):
        ref = moe.route_weights(l[t], ids[t], score, renorm, scale)
        finite = l[t][np.isfinite(l[t])]
        big = np.abs(finite).max() if finite.size else 0.0
        assert np.all(np.abs(got[t] - ref) <= 2.0 ** -23 * (48 + 2 * big) * np.abs(ref) + 1e-30), t


CASES = [  # tokens, experts, topk, score, bias, groups, topk_groups, renorm, dtype, masked
    (1, 128, 8, 0, False, 1, 1, True, "bf16", False),
    (3, 1, 1, 0, False, 1, 1, False, "f32", True),
    (17, 8, 8, 1, True, 1, 1, True, "f32", True),
    (33, 31, 5, 0, True, 1, 1, False, "bf16", True),
    (40, 64, 6, 1, True, 8, 3, True, "f32", True),       # groups of whole lanes
    (29, 96, 4, 0, True, 8, 2, True, "f32", True),       # groups across lanes
    (29, 160, 8, 1, False, 32, 5, False, "bf16", True),
    (64, 256, 8, 1, True, 8, 4, True, "f32", True),
    (9, 257, 32, 0, False, 1, 1, True, "f32", False),    # rows off the vector boundaries
    (7, 1000, 32, 1, True, 10, 3, False, "bf16", True),
    (5, 1024, 16, 0, True, 16, 16, True, "f32", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}s{c[3]}g{c[5]}")
def test_route(rd_lib, case):
    tokens, experts, topk, score, with_bias, groups, topk_groups, renorm, dt, masked = case
    rng = np.random.default_rng(tokens * 1000 + experts)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    logits = _grid_logits(rng, tokens, experts, masked, dtype)
    bias = np.round(rng.normal(size=experts) * 4) / 4 * 0.25 if with_bias else None
    r = rd_lib.route(logits.to(DEV), topk, score=score, groups=groups, topk_groups=topk_groups,
                     bias=None if bias is None else torch.tensor(bias, dtype=torch.float32, device=DEV),
                     renormalize=renorm, scale=2.5)
    ids, l = r.ids.cpu().numpy(), logits.double().numpy()
    for t in range(tokens):
        want = moe.route_choose(l[t], bias, topk, score, groups, topk_groups)
        if score == moe.SOFTMAX:
            assert ids[t].tolist() == want, t
            continue
        live = [e for e in ids[t] if e >= 0]
        assert len(set(live)) == len(live) == sum(e >= 0 for e in want)
        assert all(e == -1 for e in ids[t][len(live):])
        if groups == 1:
            key = moe.route_keys(l[t], bias, score)
            got = key[live]
            assert np.all(np.abs(got - key[want[:len(live)]]) <= 2.0 ** -22)
            for a, b in zip(live, live[1:]):       # equal inputs keep the order of their indices
                if l[t][a] == l[t][b] and (bias is None or bias[a] == bias[b]):
                    assert a < b
        else:
            # within the grid of the inputs distinct sums of sigmoids are rarely closer than the margin
            assert set(live) == set(want[:len(live)]) or _near_tie(l[t], bias, topk, groups, topk_groups)
    _check_weights(r.weights.double().cpu().numpy(), l, ids, score, renorm, 2.5)
    sizes, pos, rows = moe.sort_rows(ids, experts)
    assert r.group_sizes.cpu().tolist() == sizes.tolist() and int(r.rows) == rows
    np.testing.assert_array_equal(r.pos.cpu().numpy(), pos)


def _near_tie(l, bias, topk, groups, topk_groups):
    """Whether two keys or two group scores of the token are within the keys' f32 error."""
    key = moe.route_keys(l, bias, moe.SIGMOID)
    size = len(key) // groups
    by = -np.sort(-key.reshape(groups, size), axis=1)
    scores = by[:, 0] + (np.where(np.isneginf(by[:, 1]), 0, by[:, 1]) if size > 1 else 0)
    for v in (np.sort(scores[np.isfinite(scores)]), np.sort(key[np.isfinite(key)])):
        d = np.diff(v)
        if np.any(d <= 2.0 ** -21):
            return True
    return False


def test_route_extreme_logits(rd_lib):
    """Saturated sigmoids tie (lowest index first), at 1 and, where exp(-l) overflows f32, at 0; +inf wins."""
    l = torch.tensor([[100.0, 200.0, 90.0, -3.0, 150.0, -200.0, -90.0, -88.0],
                      [-100.0, -87.0, -86.5, -120.0, -1e30, -103.0, -95.0, -89.5]], device=DEV)
    r = rd_lib.route(l, 4, score=rd_lib.SCORE_SIGMOID, renormalize=False)
    assert r.ids[0].tolist() == [0, 1, 2, 4]
    ref = moe.sigmoid(l[1].double().cpu().numpy())
    assert r.ids[1].tolist() == [2, 1, 0, 3]
    got = r.weights[1].double().cpu().numpy()
    # f32 subnormals: half a unit of 2^-149 on top of the relative error of exp and the reciprocal
    assert np.all(np.abs(got[:2] - ref[[2, 1]]) <= 2.0 ** -148 + 2.0 ** -15 * ref[[2, 1]])
    assert got[2:].tolist() == [0, 0]
    l = torch.tensor([[float("inf"), 1.0, 2.0, float("nan")]], device=DEV)
    r = rd_lib.route(l, 3, score=rd_lib.SCORE_SOFTMAX)
    assert r.ids[0].tolist() == [0, 2, 1] and bool(r.weights[0].isnan().all())
    # the lowest finite value is not a mask
    low = torch.finfo(torch.float32).min
    r = rd_lib.route(torch.full((1, 4), low, device=DEV), 2)
    assert r.ids[0].tolist() == [0, 1] and r.weights[0].tolist() == [0.5, 0.5]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,topk,dt", [(1, 128, 8, "f32"), (37, 64, 6, "bf16"), (19, 257, 5, "f32"),
                                                    (6, 1024, 32, "bf16"), (300, 8, 2, "f32")])
def test_route_bwd(rd_lib, tokens, experts, topk, dt, score, renorm):
    rng = np.random.default_rng(experts + 7 * topk)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    logits = _grid_logits(rng, tokens, experts, True, dtype)
    l = logits.double().numpy()
    ids = np.array([moe.route_choose(l[t], None, topk, score) for t in range(tokens)])
    d = rng.normal(size=(tokens, topk)).astype(np.float32)
    out = rd_lib.route_bwd(logits.to(DEV), _i32(ids), torch.from_numpy(d).to(DEV), score=score,
                           renormalize=renorm, scale=1.5)
    assert out.dtype == dtype
    got = out.double().cpu().numpy()
    for t in range(tokens):
        ref = moe.route_loss_grad(l[t], ids[t], d[t], score, renorm, 1.5)
        q = moe.route_weights(l[t], ids[t], score, renorm)
        live = np.isfinite(l[t])
        big = np.abs(l[t][live]).max() if live.any() else 0.0
        spread = np.abs(q * d[t]).sum() + np.abs(d[t]).max()
        if score == moe.SOFTMAX and not renorm:
            factor = np.zeros(experts)
            if live.any():
                factor[live] = np.exp(l[t][live] - l[t][live].max())
                factor /= factor.sum()
        else:
            factor = np.zeros(experts)
            total = sum(moe.sigmoid(l[t][e]) for e in ids[t] if e >= 0)
            for k, e in enumerate(ids[t]):
                if e >= 0:
                    s = moe.sigmoid(l[t][e])
                    factor[e] = q[k] if score == moe.SOFTMAX else (s / total if renorm else s)
        tol = 2.0 ** -23 * (64 + 4 * big) * 1.5 * factor * spread + 1e-30
        if dt == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(got[t] - ref) <= tol), t


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 8, 128), (5, 3, 7), (1000, 8, 256), (2049, 6, 512),
                                                 (1500, 8, 1024), (30000, 8, 64), (50000, 7, 513)])
def test_sort_rows(rd_lib, tokens, topk, experts):
    """Repeated experts in a token, ids outside the range, one and several batches of every warp."""
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, experts + 1, (tokens, topk))
    sizes, pos, rows = rd_lib.sort_rows(_i32(ids), experts)
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(live, flat, experts), kind="stable")
    want = np.empty(flat.size, np.int64)
    want[order] = np.arange(flat.size)
    want[~live] = -1
    np.testing.assert_array_equal(pos.cpu().numpy().reshape(-1), want)
    np.testing.assert_array_equal(sizes.cpu().numpy(), np.bincount(flat[live], minlength=experts))
    assert int(rows) == live.sum()
    if tokens * topk < 5000:
        o = moe.sort_rows(ids, experts)
        np.testing.assert_array_equal(o[1], pos.cpu().numpy())


def test_sort_of_no_slots(rd_lib):
    sizes, pos, rows = rd_lib.sort_rows(torch.empty((0, 4), dtype=torch.int32, device=DEV), 9)
    assert sizes.tolist() == [0] * 9 and int(rows) == 0 and pos.shape == (0, 4)
    sizes, pos, rows = rd_lib.sort_rows(torch.full((6, 2), -1, dtype=torch.int32, device=DEV), 3)
    assert sizes.tolist() == [0] * 3 and int(rows) == 0 and bool((pos == -1).all())


def test_token_limit(rd_lib):
    """Tokens at or past the device-side limit are neither read nor written and have no row."""
    rng = np.random.default_rng(2)
    tokens, experts, topk, hidden = 50, 16, 4, 72
    logits = _grid_logits(rng, tokens, experts, False, torch.float32).to(DEV)
    for lim in (-3, 0, 1, 33, 50, 99):
        L = max(0, min(lim, tokens))
        limit = _i32([lim])
        bad = logits.clone()
        bad[L:] = float("nan")
        out = rd_lib.Routing(*[torch.full(s, 77, dtype=d, device=DEV) for s, d in (
            ((tokens, topk), torch.int32), ((tokens, topk), torch.float32), ((experts,), torch.int32),
            ((tokens, topk), torch.int32), ((1,), torch.int32))])
        rd_lib.route(bad, topk, limit=limit, out=out)
        for x in (out.ids, out.weights, out.pos):
            assert bool((x[L:] == 77).all())
        assert int(out.rows) == int(out.group_sizes.sum()) == L * topk
        x = torch.randn(tokens, hidden, device=DEV).to(torch.bfloat16)
        packed = rd_lib.dispatch_rows(x, out.pos, limit=limit, out=torch.full(
            (tokens * topk, hidden), 5.0, dtype=torch.bfloat16, device=DEV))
        assert bool((packed[L * topk:] == 5.0).all())
        for t in range(0, L, 7):
            assert bool((packed[out.pos[t].long()] == x[t]).all())
        back = rd_lib.combine_rows(packed, out.pos, out.weights, limit=limit,
                                   out=torch.full((tokens, hidden), 9.0, dtype=torch.bfloat16, device=DEV))
        assert bool((back[L:] == 9.0).all())
        d_y, d_w = rd_lib.combine_rows_bwd(x, packed, out.pos, out.weights, limit=limit,
                                           d_y=torch.full_like(packed, 3.0),
                                           d_w=torch.full((tokens, topk), 4.0, device=DEV))
        assert bool((d_w[L:] == 4.0).all()) and bool((d_y[L * topk:] == 3.0).all())
        g = rd_lib.route_bwd(bad, out.ids, torch.ones(tokens, topk, device=DEV), limit=limit,
                             out=torch.full((tokens, experts), 6.0, device=DEV))
        assert bool((g[L:] == 6.0).all()) and bool(g[:L].isfinite().all())


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_of_a_constant_weight(rd_lib, score, dtype):
    """One expert a token, renormalised: its weight is the scale whatever the logits are, so the gradient is zero."""
    rng = np.random.default_rng(21)
    logits = torch.from_numpy(4 * rng.normal(size=(777, 24)).astype(np.float32)).to(dtype).to(DEV)
    r = rd_lib.route(logits, 1, score=score, scale=2.5)
    assert bool((r.weights == 2.5).all())
    d_w = torch.from_numpy(rng.normal(size=(777, 1)).astype(np.float32)).to(DEV)
    assert not rd_lib.route_bwd(logits, r.ids, d_w, score=score, scale=2.5).any()


def _slots(rng, tokens, topk, rows):
    """Positions of some slots, without repeats; others have no row (-1 or far outside)."""
    pos = np.full(tokens * topk, -1)
    n = min(rows, tokens * topk)
    at = rng.choice(tokens * topk, n, replace=False)
    pos[at] = rng.choice(rows, n, replace=False)
    drop = rng.random(tokens * topk) < 0.1
    pos[drop] = rng.choice([-1, -2 ** 31, rows, 2 ** 31 - 1], drop.sum())
    return pos.reshape(tokens, topk)


@pytest.mark.parametrize("tokens,topk,hidden,rows", [(1, 1, 8, 1), (1, 8, 4096, 8), (7, 3, 264, 25), (33, 32, 1016, 900),
                                                     (500, 2, 4104, 1000), (3000, 8, 512, 24000)])
def test_dispatch_combine(rd_lib, tokens, topk, hidden, rows):
    rng = np.random.default_rng(tokens + hidden)
    pos = _slots(rng, tokens, topk, rows)
    x = torch.from_numpy(rng.normal(size=(tokens, hidden)).astype(np.float32)).to(torch.bfloat16)
    buf = torch.full((rows + 2, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    rd_lib.dispatch_rows(x.to(DEV), _i32(pos), out_rows=rows, out=buf[:rows])
    want = torch.full((rows + 2, hidden), 7.0, dtype=torch.bfloat16)
    for t, k in np.argwhere((pos >= 0) & (pos < rows)):
        want[pos[t, k]] = x[t]
    assert torch.equal(buf.cpu().view(torch.int16), want.view(torch.int16))

    y = torch.from_numpy(rng.normal(size=(rows, hidden)).astype(np.float32)).to(torch.bfloat16)
    w = rng.normal(size=(tokens, topk)).astype(np.float32)
    w[(pos < 0) | (pos >= rows)] = np.nan           # the weight of a slot without a row is not used
    y64 = y.double().numpy()
    for weights in (w, None):
        got = rd_lib.combine_rows(y.to(DEV), _i32(pos), None if weights is None else torch.from_numpy(w).to(DEV))
        ref, mag = moe.combine_rows(y64, pos, weights)
        tol = (topk + 1) * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(ref) + 1e-38
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)

    d_out = torch.from_numpy(rng.normal(size=(tokens, hidden)).astype(np.float32)).to(torch.bfloat16)
    d_y = torch.full((rows, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    _, d_w = rd_lib.combine_rows_bwd(d_out.to(DEV), y.to(DEV), _i32(pos), torch.from_numpy(w).to(DEV), d_y=d_y)
    d_w = d_w.double().cpu().numpy()
    bits = np.full((rows, hidden), obf.round_f32_to_bf16_bits(np.float32(7.0)), np.uint16)
    d32 = d_out.float().numpy()
    for t, k in np.argwhere((pos >= 0) & (pos < rows)):
        p = pos[t, k]
        bits[p] = obf.round_f32_to_bf16_bits(d32[t] * w[t, k])
        ref = float((d32[t].astype(np.float64) * y64[p]).sum())
        assert abs(d_w[t, k] - ref) <= unsort.dot_tolerance(d32[t:t + 1], y64[p:p + 1])[0]
    np.testing.assert_array_equal(obf.torch_bf16_bits(d_y), bits)
    assert np.all(d_w[(pos < 0) | (pos >= rows)] == 0)


def test_combine_gradient_is_the_formulas(rd_lib):
    """d_y and d_w of a scalar loss against differences of the oracle's combine."""
    rng = np.random.default_rng(11)
    tokens, topk, hidden = 6, 3, 16
    ids = np.array([rng.permutation(5)[:topk] for _ in range(tokens)])
    _, pos, _ = moe.sort_rows(ids, 5)
    y = torch.from_numpy(rng.normal(size=(tokens * topk, hidden)).astype(np.float32)).to(torch.bfloat16)
    w = rng.normal(size=(tokens, topk)).astype(np.float32)
    d = torch.from_numpy(rng.normal(size=(tokens, hidden)).astype(np.float32)).to(torch.bfloat16)
    d_y, d_w = rd_lib.combine_rows_bwd(d.to(DEV), y.to(DEV), _i32(pos), torch.from_numpy(w).to(DEV))
    d64, y64 = d.double().numpy(), y.double().numpy()

    def loss(yy, ww):
        return float((d64 * moe.combine_rows(yy, pos, ww)[0]).sum())

    h = 1e-3          # the loss is linear in y and in w: differences are exact up to rounding, 1e-12 / h
    for t, k in ((0, 0), (2, 1), (5, 2)):
        w1 = w.astype(np.float64).copy()
        w1[t, k] += h
        ref = (loss(y64, w1) - loss(y64, w.astype(np.float64))) / h
        assert abs(ref - float(d_w[t, k])) < 1e-5
        p = pos[t, k]
        y1 = y64.copy()
        y1[p, 3] += h
        ref = (loss(y1, w) - loss(y64, w)) / h
        assert abs(ref - float(d_y[p, 3])) <= 2.0 ** -8 * abs(ref) + 1e-8


def test_offsets_past_32_bits(rd_lib):
    """Rows whose element offsets pass 2^31: 600001 packed rows of 4096 (4.9 GB)."""
    rows, hidden = 600001, 4096
    far = [rows - 1, rows - 2, 524288, 0]
    y = torch.zeros((rows, hidden), dtype=torch.bfloat16, device=DEV)
    x = torch.randn(2, hidden, device=DEV).to(torch.bfloat16)
    pos = _i32([[far[0], far[3]], [far[1], far[2]]])
    rd_lib.dispatch_rows(x, pos, out_rows=rows, out=y)
    for t in range(2):
        for p in pos[t].tolist():
            assert torch.equal(y[p], x[t])
    w = torch.tensor([[0.5, 0.25], [2.0, -1.0]], device=DEV)
    got = rd_lib.combine_rows(y, pos, w)
    assert torch.equal(got, (x.float() * w.sum(1, keepdim=True)).to(torch.bfloat16))
    d_y = torch.zeros_like(y)
    rd_lib.combine_rows_bwd(x, y, pos, w, d_y=d_y)
    assert torch.equal(d_y[far[0]], (x[0].float() * 0.5).to(torch.bfloat16))
    q = rd_lib.Mxfp4(torch.zeros((rows, hidden // 2), dtype=torch.uint8, device=DEV),
                     torch.zeros((rows, 128), dtype=torch.uint8, device=DEV))
    rd_lib.mxfp4_quantize(x, pos=pos, out_rows=rows, out=q)
    one = rd_lib.mxfp4_quantize(x)
    assert torch.equal(q.q[far[0]], one.q[0]) and torch.equal(q.scales[far[1]], one.scales[1])


def test_other_streams_graph_and_repeats(rd_lib):
    """The chain on a side stream, then in a CUDA graph replayed after the inputs changed on the
    device: the same bits as the eager calls, every time."""
    rng = np.random.default_rng(4)
    tokens, experts, topk, hidden = 300, 32, 4, 256
    logits = torch.from_numpy(rng.normal(size=(tokens, experts)).astype(np.float32)).to(DEV)
    x = torch.randn(tokens, hidden, device=DEV).to(torch.bfloat16)
    limit = _i32([tokens])

    def chain(stream=None):
        r = rd_lib.route(logits, topk, limit=limit, stream=stream)
        packed = rd_lib.dispatch_rows(x, r.pos, limit=limit, stream=stream)
        return r, packed, rd_lib.combine_rows(packed, r.pos, r.weights, limit=limit, stream=stream)

    want = [chain()[2].clone() for _ in range(2)]
    assert torch.equal(want[0], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = chain()[2]
    side.synchronize()
    assert torch.equal(on_side, want[0])
    side.wait_stream(torch.cuda.current_stream())
    given = chain(side)[2]            # the stream as an argument
    side.synchronize()
    assert torch.equal(given, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, packed, out = chain()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    logits.copy_(torch.from_numpy(rng.normal(size=(tokens, experts)).astype(np.float32)))
    limit.fill_(123)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert int(r.rows) == 123 * topk
    assert torch.equal(out[:123], chain()[2][:123]) and bool((out[123:] == 0).all())


def test_binding_refusals(rd_lib):
    l = torch.zeros(4, 16, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    rows = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    for call in (lambda: rd_lib.route(l[:, ::2], 2), lambda: rd_lib.route(l.double(), 2),
                 lambda: rd_lib.route(l, 2, bias=torch.zeros(15, device=DEV)),
                 lambda: rd_lib.route(l, 2, bias=torch.zeros(16)),
                 lambda: rd_lib.route(l, 2, limit=torch.zeros(2, dtype=torch.int32, device=DEV)),
                 lambda: rd_lib.route_bwd(l, ids[:3], w), lambda: rd_lib.route_bwd(l, ids.long(), w),
                 lambda: rd_lib.route_bwd(l, ids, w.half()), lambda: rd_lib.sort_rows(ids.t(), 4),
                 lambda: rd_lib.dispatch_rows(rows, ids), lambda: rd_lib.dispatch_rows(rows[:4].float(), ids),
                 lambda: rd_lib.dispatch_rows(rows[:4], ids, out=rows[:, :32]),
                 lambda: rd_lib.combine_rows(rows.t(), ids), lambda: rd_lib.combine_rows(rows, ids, w[:2]),
                 lambda: rd_lib.combine_rows_bwd(rows[:4], rows[:, :32].contiguous(), ids, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rd_lib.route(l, 17), lambda: rd_lib.route(l, 2, groups=3),
                 lambda: rd_lib.route(l, 2, groups=4, topk_groups=5), lambda: rd_lib.route(l, 2, score=9),
                 lambda: rd_lib.sort_rows(ids, 2000), lambda: rd_lib.sort_rows(ids, 0),
                 lambda: rd_lib.combine_rows(rows[:, :60].contiguous(), ids)):
        with pytest.raises(rd_lib.RdError):
            call()
