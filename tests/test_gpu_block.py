"""Layer norm, products with bias / activation / residual, and dropout on the GPU against the float64
oracle.

Tolerances (fixed from the arithmetic, u = 2^-24; ROUND is half a step of the output's type, 2^-8 for
bf16 and u for f32, relative to the value):

* row sums: at most 128 roundings on any path from an element to its sum (eight elements of up to
  four vectors in a thread, five steps in a warp, 32 warps), so 128 u of the sum of magnitudes.
* norm: a centred element is off by u of itself and by the error of the mean, which is taken out of the
  centred elements a second time, so 128 u of their mean magnitude (at most the deviation); 1 / deviation by
  half of 128 u and a few u.  With y the normalised element: 140 u (|y| + 1) |w| + 2 u |out| + ROUND.
* norm's gradients: y is off by 2 u, the two row means by 130 u of the mean magnitudes of their terms, the
  rest by 8 u; the columns' sums by (rows + 64) u of the sum of magnitudes.
* products: f32 accumulation of k exact products, a rounding (or truncation, 2 u) for each of them and for
  each of up to 16 in one step: 2^-22 (k + 16) sum|x w|, plus 2 u of bias and residual; activations
  have slopes below 1.2.
* activations and slopes: hardware exp and reciprocal, 2 ulp each, and the rounding of exp's
  argument a: relative 2^-18 + 2^-21 |a| of the terms s and z b of a slope (s z of a value).
* dropout: two roundings, and ROUND; what is kept is exact.
"""
import math

import numpy as np
import pytest

from oracle import block, group_bounds
from parity_util import assert_close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ROUND = {"f32": U, "bf16": 2.0 ** -8}
SENT = 0x3C3C
EXTRA = 3                 # rows behind the output that must stay as they are


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _rows(rng, shape, dtype, scale=1.0, shift=0.0):
    return (torch.from_numpy(rng.normal(size=shape) * scale + shift)).to(TYPES[dtype])


def _f64(t):
    return t.double().cpu().numpy()


def _buffer(rows, cols, dtype):
    buf = torch.empty(rows + EXTRA, cols, dtype=TYPES[dtype], device=DEV)
    buf.view(torch.int16).fill_(SENT)
    return buf


def _untouched(buf, first):
    return bool((buf[first:].contiguous().view(torch.int16) == SENT).all())


def _poisoned(x, limit):
    y = x.clone()
    if limit is not None:
        y[max(limit, 0):] = float("nan")
    return y.to(DEV)


def _live(rows, limit):
    return rows if limit is None else min(max(limit, 0), rows)


# ---------------------------------------------------------------------------- layer norm
def _check_norm(rd, rows, hidden, dt, ot, weight=True, bias=True, limit=None, shift=0.0, scale=1.0, eps=1e-5, seed=0):
    rng = np.random.default_rng(seed + rows * 7 + hidden)
    x = _rows(rng, (rows, hidden), dt, scale, shift)
    w = _rows(rng, hidden, "f32") if weight else None
    b = _rows(rng, hidden, "f32") if bias else None
    buf = _buffer(rows, hidden, ot)
    stats = torch.full((2, rows + EXTRA), 7.0, device=DEV)
    out = rd.LayerNorm(buf[:rows], stats[0, :rows], stats[1, :rows])
    rd.layer_norm_fwd(_poisoned(x, limit), None if w is None else w.to(DEV), None if b is None else b.to(DEV), eps=eps,
                      limit=None if limit is None else _i32([limit]), out=out)
    L = _live(rows, limit)
    assert _untouched(buf, L) and bool((stats[:, L:] == 7.0).all())
    if L == 0:
        return
    w64 = np.ones(hidden) if w is None else _f64(w)
    b64 = np.zeros(hidden) if b is None else _f64(b)
    x64 = _f64(x)[:L]
    ref, mean, rstd = block.layer_norm(x64, w64, b64, float(np.float32(eps)))
    y = (x64 - mean[:, None]) * rstd[:, None]
    tol = 140 * U * (np.abs(y) + 1) * np.abs(w64) + 2 * U * np.abs(ref) + ROUND[ot] * np.abs(ref) + 1e-37
    assert_close(_f64(out.out)[:L], ref, tol, "norm")
    assert_close(_f64(out.mean)[:L], mean, 2 * U * np.abs(mean) + 130 * U / rstd, "mean")
    assert_close(_f64(out.rstd)[:L], rstd, 140 * U * rstd, "rstd")


NORM_WIDTHS = [8, 64, 248, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392,
               32768, 32776, 40008]


@pytest.mark.parametrize("hidden", NORM_WIDTHS)
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm(rd_lib, hidden, dt, ot):
    _check_norm(rd_lib, 13, hidden, dt, ot)


@pytest.mark.parametrize("rows", [0, 1, 2, 7, 8, 9, 700, 2500])
@pytest.mark.parametrize("hidden", [64, 520, 4096])
def test_norm_rows(rd_lib, rows, hidden):
    _check_norm(rd_lib, rows, hidden, "bf16", "f32", limit=None)


@pytest.mark.parametrize("limit", [-3, 0, 1, 5, 17, 40])
@pytest.mark.parametrize("hidden", [248, 4096, 33000])
def test_norm_limit(rd_lib, limit, hidden):
    _check_norm(rd_lib, 17, hidden, "f32", "bf16", limit=limit)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("hidden", [64, 4096, 12288, 33000])
def test_norm_without_parameters(rd_lib, weight, bias, hidden):
    _check_norm(rd_lib, 5, hidden, "bf16", "f32", weight, bias)


@pytest.mark.parametrize("hidden", [64, 1000, 4096, 16384, 33000])
@pytest.mark.parametrize("shift,scale", [(1e4, 1.0), (-3e5, 0.5), (0.0, 1e-18), (0.0, 1e15), (1.0, 0.0)])
def test_norm_far_from_zero(rd_lib, hidden, shift, scale):
    """Rows far from zero keep their variance; tiny and large ones their scale; constant ones give the bias."""
    _check_norm(rd_lib, 6, hidden, "f32", "f32", shift=shift, scale=scale)


def test_norm_special_rows(rd_lib):
    """A row with an infinity or a NaN is NaN throughout, and its neighbours are not."""
    for hidden in (64, 4096, 33000):
        x = torch.randn(24, hidden, generator=torch.Generator().manual_seed(hidden))
        clean = rd_lib.layer_norm_fwd(x.to(DEV), stats=True)
        x[3, 5], x[9, hidden - 1], x[17, 0] = float("inf"), float("nan"), float("-inf")
        got = rd_lib.layer_norm_fwd(x.to(DEV), stats=True)
        bad = [3, 9, 17]
        good = [r for r in range(24) if r not in bad]
        assert bool(torch.isnan(got.out[bad]).all()) and bool(torch.isnan(got.rstd[bad]).all())
        assert torch.equal(got.out[good], clean.out[good]) and torch.equal(got.rstd[good], clean.rstd[good])


def _check_norm_bwd(rd, rows, hidden, dt, ot, weight=True, limit=None, need=(True, True), seed=0):
    rng = np.random.default_rng(seed + rows * 5 + hidden)
    x, d = _rows(rng, (rows, hidden), dt, 1.5, 0.3), _rows(rng, (rows, hidden), ot)
    w = _rows(rng, hidden, "f32") if weight else None
    _, mean, rstd = block.layer_norm(_f64(x), eps=1e-5)
    mean, rstd = torch.from_numpy(mean).float(), torch.from_numpy(rstd).float()
    L = _live(rows, limit)
    buf = _buffer(rows, hidden, dt)
    ws = torch.full((rd.layer_norm_bwd_workspace_bytes(rows, hidden) + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    d_x, d_w, d_b = rd.layer_norm_bwd(_poisoned(d, limit), _poisoned(x, limit), None if w is None else w.to(DEV),
                                      _poisoned(mean, limit), _poisoned(rstd, limit),
                                      limit=None if limit is None else _i32([limit]), need_weight=need[0],
                                      need_bias=need[1], d_x=buf[:rows], workspace=ws[:-64])
    assert _untouched(buf, L) and bool((ws[-64:] == 0xFF).all())
    assert (d_w is not None, d_b is not None) == need
    w64 = np.ones(hidden) if w is None else _f64(w)
    x64, d64, mean, rstd = _f64(x)[:L], _f64(d)[:L], _f64(mean)[:L], _f64(rstd)[:L]
    ref, ref_w, ref_b = block.layer_norm_bwd(d64, x64, w64, mean, rstd)
    y, g, r = (x64 - mean[:, None]) * rstd[:, None], d64 * w64, rstd[:, None]
    p, q = np.abs(g).mean(1, keepdims=True), np.abs(g * y).mean(1, keepdims=True)
    if L:
        tol = r * U * (8 * np.abs(g) + 140 * p + 140 * np.abs(y) * q) + ROUND[dt] * np.abs(ref) + 1e-37
        assert_close(_f64(d_x)[:L], ref, tol, "d_x")
    if need[0]:
        assert_close(_f64(d_w), ref_w, (L + 64) * U * np.abs(d64 * y).sum(0), "d_weight")
    if need[1]:
        assert_close(_f64(d_b), ref_b, (L + 64) * U * np.abs(d64).sum(0), "d_bias")


@pytest.mark.parametrize("hidden", [8, 64, 248, 256, 264, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392,
                                    20000, 32776, 65536, 65544])
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm_bwd(rd_lib, hidden, dt, ot):
    _check_norm_bwd(rd_lib, 37, hidden, dt, ot)


@pytest.mark.parametrize("hidden", [8, 248, 264, 1024, 1032, 2048, 2056, 4096, 4104, 8192])
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_norm_bwd_many_rows(rd_lib, hidden, dt, ot):
    _check_norm_bwd(rd_lib, 1061, hidden, dt, ot)


@pytest.mark.parametrize("limit", [-1, 0, 1, 700, 1299, 2000])
@pytest.mark.parametrize("hidden", [248, 4096])
def test_norm_bwd_many_rows_limit(rd_lib, limit, hidden):
    _check_norm_bwd(rd_lib, 1300, hidden, "f32", "bf16", limit=limit)


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
def test_norm_bwd_many_rows_parts_left_out(rd_lib, need):
    _check_norm_bwd(rd_lib, 1030, 1032, "bf16", "f32", weight=False, need=need)


@pytest.mark.parametrize("rows", [0, 1, 3, 8, 9, 600, 1024, 1025, 3001])
@pytest.mark.parametrize("hidden", [64, 1032, 4096, 8192, 12000])
def test_norm_bwd_rows(rd_lib, rows, hidden):
    _check_norm_bwd(rd_lib, rows, hidden, "bf16", "bf16")


@pytest.mark.parametrize("limit", [-1, 0, 1, 20, 33, 50])
@pytest.mark.parametrize("hidden", [248, 4096, 9000, 70000])
def test_norm_bwd_limit(rd_lib, limit, hidden):
    _check_norm_bwd(rd_lib, 33, hidden, "f32", "bf16", limit=limit)


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("hidden", [64, 2048, 9000, 70000])
def test_norm_bwd_parts_left_out(rd_lib, need, hidden):
    _check_norm_bwd(rd_lib, 21, hidden, "bf16", "f32", weight=False, need=need)


# ---------------------------------------------------------------------------- activations' error
def _exp_argument(z, kind):
    z = np.asarray(z, np.float64)
    if kind == block.GELU:
        return z * z / 2
    if kind == block.GELU_TANH:
        return np.abs(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return np.abs(z) if kind == block.SILU else np.zeros_like(z)


def _act_tol(z, kind):
    if kind in (block.NONE, block.RELU):
        return np.zeros_like(z)
    return (2.0 ** -18 + 2.0 ** -21 * np.minimum(_exp_argument(z, kind), 120)) * np.abs(block.act(z, kind)) + 1e-37


def _slope_tol(z, kind):
    if kind in (block.NONE, block.RELU):
        return np.zeros_like(z)
    s, b = block.slope_terms(z, kind)
    return (2.0 ** -18 + 2.0 ** -21 * np.minimum(_exp_argument(z, kind), 120)) * (np.abs(s) + np.abs(b)) + 1e-37


# ---------------------------------------------------------------------------- products
def _check_linear(rd, m, k, n, kind=0, bias=True, residual=False, pre=False, ot="bf16", limit=None, sizes=None, off=0,
                  gl=None, seed=0):
    rng = np.random.default_rng(seed + m * 3 + k * 5 + n)
    gl = None if sizes is None else (len(sizes) - off if gl is None else gl)
    lead = () if sizes is None else (gl,)
    x = _rows(rng, (m, k), "bf16")
    w = _rows(rng, lead + (k, n), "bf16", 1.5 / math.sqrt(max(k, 1)))
    b = _rows(rng, lead + (n,), "f32", 0.5) if bias else None
    res = _rows(rng, (m, n), ot) if residual else None
    buf, pbuf = _buffer(m, n, ot), _buffer(m, n, "bf16")
    status = _i32([0])
    bounds, L = group_bounds([m] if sizes is None else sizes, m, limit)
    got = rd.linear(_poisoned(x, L), w.to(DEV), None if b is None else b.to(DEV),
                    residual=None if res is None else _poisoned(res, L), act=kind,
                    group_sizes=None if sizes is None else _i32(sizes), group_offset=off,
                    limit=None if limit is None else _i32([limit]), out=buf[:m], pre=pbuf[:m] if pre else None,
                    status=status)
    assert isinstance(got, tuple) == pre
    assert _untouched(buf, L) and _untouched(pbuf, L if pre else 0)
    assert int(status.item()) == 0
    x64, w64 = _f64(x), _f64(w)
    b64 = None if b is None else _f64(b)
    r64 = None if res is None else _f64(res)
    ref, z = block.linear(x64, w64, b64, r64, kind, sizes, off, limit)
    mass, _ = block.linear(np.abs(x64), np.abs(w64), None, None, 0, sizes, off, limit)
    ztol = 2.0 ** -22 * (k + 16) * mass + 2 * U * np.abs(z) + 2 * U * (0 if b is None else np.abs(b64).max())
    lo, hi = (0, L) if sizes is None else (bounds[off], bounds[off + gl])
    tol = 1.2 * ztol + _act_tol(z, kind) + 2 * U * (0 if res is None else np.abs(r64)) + (ROUND[ot] + U) * np.abs(ref) + 1e-37
    o64 = _f64(buf[:m])
    assert_close(o64[lo:hi], ref[lo:hi], tol[lo:hi], "out")
    zero = buf[:m].view(torch.int16 if ot == "bf16" else torch.int32)
    assert bool((zero[:lo] == 0).all()) and bool((zero[hi:L] == 0).all())
    if pre:
        assert_close(_f64(pbuf[:m])[lo:hi], z[lo:hi], (ztol + 2.0 ** -8 * np.abs(z) + 1e-37)[lo:hi], "pre")
        pz = pbuf[:m].view(torch.int16)
        assert bool((pz[:lo] == 0).all()) and bool((pz[hi:L] == 0).all())


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 16, 31, 63, 64, 65, 127, 128, 129, 200, 257])
@pytest.mark.parametrize("k,n", [(8, 8), (64, 64), (520, 72), (1032, 200), (4096, 136)])
def test_linear_few_rows(rd_lib, m, k, n):
    """One weight, few output tiles: k shared out over clusters, odd widths, rows off every tile."""
    kind = (m + n) % 5
    _check_linear(rd_lib, m, k, n, kind, residual=m % 2 == 0, pre=m % 3 == 0, ot="f32" if m % 4 == 1 else "bf16")


def test_linear_f32_output_is_as_exact_as_f32(rd_lib):
    """Router logits: the tensor core cuts its sums off (by less than an ulp, 2^-23) at each of 32 steps, then a
    rounded sum takes over, whatever k is: at most 32 ulp of the result's norm.  On few tiles and on many."""
    for m, k, n in ((300, 8192, 136), (2500, 4096, 128), (9, 16384, 72), (130, 4096, 14336), (3000, 8192, 2056)):
        rng = np.random.default_rng(m)
        x, w = _rows(rng, (m, k), "bf16"), _rows(rng, (k, n), "bf16", 1 / math.sqrt(k))
        got = rd_lib.linear(x.to(DEV), w.to(DEV), out_dtype=torch.float32)
        ref = x.to(DEV).double() @ w.to(DEV).double()
        assert float((got.double() - ref).norm() / ref.norm()) <= 32 * 2.0 ** -23, (m, k, n)
        for v in (rd_lib.VARIANT_SINGLE, rd_lib.VARIANT_PAIR):
            with rd_lib.tuning(variant=v):
                one = rd_lib.linear(x.to(DEV), w.to(DEV).unsqueeze(0), group_sizes=_i32([m]), out_dtype=torch.float32)
            assert float((one.double() - ref).norm() / ref.norm()) <= 32 * 2.0 ** -23, (m, k, n, v)


@pytest.mark.parametrize("m,k,n", [(16381, 72, 128), (2047, 136, 1000), (19000, 64, 64), (700, 200, 2000)])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_linear_low_tiles(rd_lib, m, k, n, ot):
    """One weight, tiles for most SMs and for a little more than all."""
    _check_linear(rd_lib, m, k, n, block.GELU, residual=True, pre=True, ot=ot, limit=m - 5)


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(5, 1000), (100, 264), (3000, 520)])
def test_linear_activations(rd_lib, kind, ot, m, n):
    for bias, residual, pre in ((True, False, True), (False, True, False), (True, True, True)):
        _check_linear(rd_lib, m, 136, n, kind, bias, residual, pre, ot)


@pytest.mark.parametrize("m", [0, 1, 40, 700])
def test_linear_without_contraction(rd_lib, m):
    _check_linear(rd_lib, m, 0, 72, block.GELU, residual=True, pre=True)


@pytest.mark.parametrize("limit", [-2, 0, 1, 7, 8, 64, 65, 130, 500])
@pytest.mark.parametrize("m,n", [(70, 72), (300, 136), (5000, 1032)])
def test_linear_limit(rd_lib, limit, m, n):
    _check_linear(rd_lib, m, 200, n, block.SILU, residual=True, pre=True, limit=min(limit, m + 3), ot="f32")


@pytest.mark.parametrize("variant", ["single", "pair"])
@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,off,gl,limit", [
    ([0, 1, 127, 128, 129, 0, 255, 3], 0, None, None),
    ([0, 1, 127, 128, 129, 0, 255, 3], 2, 4, None),
    ([0, 1, 127, 128, 129, 0, 255, 3], 1, 5, 300),
    ([5, 0, 300, 20], 1, 2, 100),
    ([0, 0, 0], 0, None, None),
    ([643, 0], 0, 1, 0),
])
def test_linear_by_expert(rd_lib, variant, ot, sizes, off, gl, limit):
    v = rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE
    with rd_lib.tuning(variant=v):
        for i, (kind, residual, pre) in enumerate(((block.GELU, False, True), (block.GELU_TANH, True, False),
                                                   (block.NONE, True, True), (block.RELU, False, False))):
            _check_linear(rd_lib, 643 + 20 * (i % 2), 200, 264 + 32 * i, kind, True, residual, pre, ot, limit, sizes, off, gl)


@pytest.mark.parametrize("ot", ["bf16", "f32"])
def test_most_groups(rd_lib, ot):
    """1024 groups, most of them short and some empty."""
    sizes = [(7 * i) % 11 for i in range(1024)]
    sizes[500] = 700
    _check_linear(rd_lib, 5900, 584, 40, block.GELU, True, True, True, ot, 5800, sizes, 3, 1000)
    _check_act_bwd(rd_lib, 5900, 72, block.GELU, ot, sizes, 3, 1000, 5800)
    _check_act_bwd(rd_lib, 2000, 72, block.SILU, ot, [s % 3 for s in sizes], 0, 1024, None)


@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("m,sizes,off,gl,limit", [
    (1, [0, 0, 1, 0], 0, None, None),
    (1, [0, 0, 1, 0], 1, 1, None),                        # no row of the local groups: zeros alone
    (4, [1, 0, 2, 1], 0, None, None),
    (17, [3, 0, 0, 9, 5, 0], 1, 4, None),
    (17, [3, 0, 0, 9, 5, 0], 1, 4, 10),
    (60, [1] * 40 + [0] * 60, 3, 90, None),               # rows behind the groups
    (130, [129, 0, 1], 0, None, 130),
    (130, [130], 0, None, -1),
    (257, [127, 1, 128, 1], 0, 3, None),
    (300, [0, 300, 0, 0, 0, 0, 0, 0], 0, None, 299),      # all rows in one group of eight
    (40, [0] * 1000 + [7] + [0] * 20 + [30] + [0] * 2, 500, 523, None),
])
def test_linear_by_expert_few_rows(rd_lib, m, sizes, off, gl, limit, ot):
    """Few tiles: k shared out over clusters, tiles as high as the groups ask for."""
    cases = ((200, 72), (1032, 40)) if len(sizes) > 100 else ((0, 64), (200, 72), (1032, 136), (2056, 520))
    for i, (k, n) in enumerate(cases):
        _check_linear(rd_lib, m, k, n, (i + m) % 5, i != 2, i % 2 == 0, i < 2, ot, limit, sizes, off, gl)


def test_linear_by_expert_bad_sizes_are_reported(rd_lib):
    """Negative sizes count as none, sizes past m are cut, and the status word says so."""
    x = torch.randn(30, 200, device=DEV).bfloat16()
    w = torch.randn(3, 200, 72, device=DEV).bfloat16()
    for sizes, same in (([10, -5, 9], [10, 0, 9]), ([10, 15, 9], [10, 15, 5]), ([40, -1, 3], [30, 0, 0])):
        status, clean = _i32([0]), _i32([0])
        got = rd_lib.linear(x, w, group_sizes=_i32(sizes), status=status)
        want = rd_lib.linear(x, w, group_sizes=_i32(same), status=clean)
        bits = (rd_lib.STATUS_NEG_SIZE if min(sizes) < 0 else 0) | (rd_lib.STATUS_OVERFLOW if sum(v for v in sizes if v > 0) > 30 else 0)
        assert int(status.item()) == bits and int(clean.item()) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("variant", ["single", "pair"])
def test_linear_f32_by_expert_of_long_rows(rd_lib, variant):
    """k of three stretches of f32 sums and a part of one, so that the accumulators' turns go on from tile to tile."""
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE):
        _check_linear(rd_lib, 26000, 1608, 520, block.SILU, True, True, True, "f32", None, [9000, 0, 300, 1, 16600], 0, 4)


def test_linear_one_weight_equals_one_group(rd_lib):
    """The kernel for few tiles and the persistent one, both variants, agree within one rounding of bf16."""
    rng = np.random.default_rng(5)
    x, w = _rows(rng, (130, 520), "bf16").to(DEV), _rows(rng, (520, 264), "bf16", 0.05).to(DEV)
    b = _rows(rng, 264, "f32").to(DEV)
    a = rd_lib.linear(x, w, b, act=block.SILU)
    for v in (rd_lib.VARIANT_SINGLE, rd_lib.VARIANT_PAIR):
        with rd_lib.tuning(variant=v):
            c = rd_lib.linear(x, w.unsqueeze(0), b.unsqueeze(0), act=block.SILU, group_sizes=_i32([130]))
        assert float((a.double() - c.double()).abs().max()) <= 2.0 ** -7 * float(a.double().abs().max())


def test_linear_special_values(rd_lib):
    """Infinities and NaN of a row stay in it; the activations' limits at infinite sums."""
    for m in (6, 1200):
        x = torch.zeros(m, 64, dtype=torch.bfloat16)
        x[:, 0] = 1.0
        x[2, 0], x[3, 0], x[4, 0] = float("inf"), float("-inf"), float("nan")
        w = torch.zeros(64, 136, dtype=torch.bfloat16)
        w[0] = 1.0
        for kind, up in ((block.RELU, 0.0), (block.GELU, float("nan")), (block.SILU, float("nan")), (block.NONE, float("-inf"))):
            out = rd_lib.linear(x.to(DEV), w.to(DEV), act=kind, out_dtype=torch.float32).cpu()
            assert bool(torch.isinf(out[2]).all()) and bool(torch.isnan(out[4]).all())
            assert bool((torch.isnan(out[3]) if math.isnan(up) else out[3] == up).all())
            want = float(block.act(np.ones(1), kind)[0])
            rest = torch.cat([out[:2], out[5:]])
            assert float((rest - want).abs().max()) <= 2.0 ** -17


def test_linear_large_arguments(rd_lib):
    """Values over the whole range of f32 exponents: the tails keep their relative precision."""
    vals = np.concatenate([np.linspace(-13, 13, 1001), [-80.0, -30.0, 30.0, 80.0, 1e4, -1e4, 1e19, -1e19]])
    z = torch.from_numpy(np.resize(vals, (16, 72))).to(torch.bfloat16)
    x = torch.eye(16, dtype=torch.bfloat16)
    for kind in block.ACTS[1:]:
        out = _f64(rd_lib.linear(x.to(DEV), z.to(DEV), act=kind, out_dtype=torch.float32))
        z64 = _f64(z)
        with np.errstate(over="ignore"):
            ref = block.act(z64, kind)
        assert_close(out, ref, _act_tol(z64, kind) + 2 * U * np.abs(ref) + 1e-37, f"act {kind}")


# ---------------------------------------------------------------------------- activation and bias gradients
def _check_act_bwd(rd, m, n, kind, ot="bf16", sizes=None, off=0, gl=None, limit=None, need=(True, True), seed=0):
    rng = np.random.default_rng(seed + m * 3 + n)
    d = _rows(rng, (m, n), ot)
    pre = None if kind == block.NONE else _rows(rng, (m, n), "bf16", 2.0)
    bounds, L = group_bounds([m] if sizes is None else sizes, m, limit)
    g_local = 1 if sizes is None else (len(sizes) - off if gl is None else gl)
    buf = _buffer(m, n, "bf16")
    ws = torch.full((rd.linear_act_bwd_workspace_bytes(m, n, g_local) + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    status = _i32([0])
    d_pre, d_bias = rd.linear_act_bwd(_poisoned(d, L), None if pre is None else _poisoned(pre, L), kind,
                                      group_sizes=None if sizes is None else _i32(sizes), group_offset=off, g_local=gl,
                                      limit=None if limit is None else _i32([limit]), need_pre=need[0], need_bias=need[1],
                                      d_pre=buf[:m] if need[0] else None, workspace=ws[:-64], status=status)
    assert int(status.item()) == 0 and bool((ws[-64:] == 0xFF).all())
    assert _untouched(buf, L if need[0] else 0)
    d64, p64 = _f64(d), None if pre is None else _f64(pre)
    ref, ref_b = block.linear_act_bwd(d64, p64, kind, sizes, off, g_local, limit)
    err = np.zeros_like(d64) if kind == block.NONE else np.abs(d64) * _slope_tol(p64, kind)
    lo, hi = (0, L) if sizes is None else (bounds[off], bounds[off + g_local])
    if need[0]:
        assert_close(_f64(d_pre)[lo:hi], ref[lo:hi], (err + (2.0 ** -8 + U) * np.abs(ref) + 1e-37)[lo:hi], "d_pre")
        bits = buf[:m].view(torch.int16)
        assert bool((bits[:lo] == 0).all()) and bool((bits[hi:L] == 0).all())
    if need[1]:
        got = _f64(d_bias).reshape(g_local, n)
        for j in range(g_local):
            a, b = bounds[off + j] if sizes is not None else 0, bounds[off + j + 1] if sizes is not None else L
            tol = err[a:b].sum(0) + (b - a + 64) * U * np.abs(ref[a:b]).sum(0) + 1e-37
            assert_close(got[j], ref_b[j], tol, f"d_bias {j}")


@pytest.mark.parametrize("kind", block.ACTS)
@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 8), (37, 64), (509, 136), (2049, 72), (4500, 264)])
def test_act_bwd(rd_lib, kind, ot, m, n):
    _check_act_bwd(rd_lib, m, n, kind, ot)


@pytest.mark.parametrize("m", [643, 2300])
@pytest.mark.parametrize("sizes,off,gl,limit", [
    ([0, 1, 127, 128, 129, 0, 255, 3], 0, None, None),
    ([0, 1, 127, 128, 129, 0, 255, 3], 2, 4, None),
    ([0, 1, 127, 128, 129, 0, 255, 3], 1, 5, 300),
    ([0, 0, 0], 0, None, None),
    ([643, 0], 0, 2, 0),
    ([1] * 300 + [0] * 300 + [1] * 43, 100, 520, None),
    ([3] * 200, 20, 170, 500),
    ([0, 643] + [0] * 400, 1, 350, None),
])
def test_act_bwd_by_expert(rd_lib, m, sizes, off, gl, limit):
    _check_act_bwd(rd_lib, m, 136, block.SILU, "bf16", sizes, off, gl, limit)
    _check_act_bwd(rd_lib, m, 40, block.NONE, "f32", sizes, off, gl, limit)


@pytest.mark.parametrize("ot", ["bf16", "f32"])
@pytest.mark.parametrize("m,sizes", [
    (65, None), (200, None), (256, None), (257, None), (500, [0, 500]), (513, [500, 13]), (700, [100, 0, 599, 1]),
    (1024, [1, 1000, 23, 0, 0]), (1025, [500, 0, 25, 500]),
])
def test_act_bwd_whole_groups(rd_lib, m, sizes, ot):
    """Around the sizes where a block takes a whole group, and of both widths that it may have then."""
    for n in (8, 72, 1000, 4104):
        _check_act_bwd(rd_lib, m, n, block.GELU if n % 16 else block.NONE, ot, sizes)


@pytest.mark.parametrize("limit", [-1, 0, 1, 63, 64, 65, 2999, 4000])
def test_act_bwd_limit(rd_lib, limit):
    for m in (90, 3000):
        _check_act_bwd(rd_lib, m, 264, block.GELU, "f32", limit=min(limit, m))


@pytest.mark.parametrize("need", [(True, False), (False, True)])
def test_act_bwd_parts_left_out(rd_lib, need):
    for m in (0, 90, 3000):
        _check_act_bwd(rd_lib, m, 72, block.GELU_TANH, "bf16", need=need)
    _check_act_bwd(rd_lib, 300, 72, block.RELU, "bf16", sizes=[100, 50, 150], off=1, gl=1, need=need)


def test_act_bwd_limits_of_the_slopes(rd_lib):
    z = torch.tensor([[float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 1e30, -1e30, 300.0]] * 2, dtype=torch.bfloat16)
    d = torch.ones(2, 8)
    for kind in block.ACTS[1:]:
        got = rd_lib.linear_act_bwd(d.to(DEV), z.to(DEV), kind)[0][0].float().cpu().tolist()
        zero = 0.0 if kind == block.RELU else 0.5
        assert got[:2] == [1.0, 0.0] and math.isnan(got[2]) and got[3:5] == [zero, zero] and got[5:] == [1.0, 0.0, 1.0], kind


def test_act_bwd_bad_sizes_are_reported(rd_lib):
    """Negative sizes count as none, sizes past m are cut, and the status word says so."""
    d = torch.ones(10, 8, device=DEV)
    for sizes, bits, want in (([4, -3, 4], 1, [4, 0, 4]), ([4, 4, 100], 2, [4, 4, 2]), ([-1, 2 ** 31 - 1, 5], 3, [0, 10, 0])):
        status = _i32([0])
        _, d_bias = rd_lib.linear_act_bwd(d, None, 0, group_sizes=_i32(sizes), status=status)
        assert int(status.item()) == bits
        assert d_bias[:, 0].tolist() == want
        status = _i32([0])
        out = rd_lib.linear(torch.ones(10, 8, dtype=torch.bfloat16, device=DEV),
                            torch.ones(3, 8, 8, dtype=torch.bfloat16, device=DEV), group_sizes=_i32(sizes), status=status)
        assert int(status.item()) == bits
        assert out[:, 0].tolist() == [8.0] * sum(want) + [0.0] * (10 - sum(want))


# ---------------------------------------------------------------------------- dropout
def _check_dropout(rd, rows, hidden, dt, ot, p, residual, limit=None, words=(1234567890123, -5), seed=0):
    rng = np.random.default_rng(seed + rows + hidden)
    x = _rows(rng, (rows, hidden), dt)
    x[x == 0] = 1.0
    res = _rows(rng, (rows, hidden), ot) if residual else None
    L = _live(rows, limit)
    buf = _buffer(rows, hidden, ot)
    rd.dropout_rows(_poisoned(x, limit), torch.tensor(words, device=DEV), p,
                    residual=None if res is None else _poisoned(res, limit),
                    limit=None if limit is None else _i32([limit]), out=buf[:rows])
    assert _untouched(buf, L)
    r64 = None if res is None else _f64(res)
    ref, kept = block.dropout(_f64(x), words[0], words[1], p, r64)
    got = _f64(buf[:rows])[:L]
    size = np.abs(ref) + (0 if res is None else np.abs(r64))
    assert_close(got, ref[:L], (4 * U * (size + np.abs(_f64(x)) * 3) + ROUND[ot] * np.abs(ref))[:L], "dropout")
    if not residual:
        assert np.array_equal(got != 0, kept[:L])


@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 64), (17, 520), (200, 4096), (0, 64), (5, 40000)])
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(rd_lib, rows, hidden, dt, ot, residual):
    for p in (0.1, 0.5):
        _check_dropout(rd_lib, rows, hidden, dt, ot, p, residual)


@pytest.mark.parametrize("p", [0.0, 1e-6, 2.0 ** -17, 0.25, 0.9999, 1.0 - 2.0 ** -18, 1.0])
def test_dropout_probabilities(rd_lib, p):
    _check_dropout(rd_lib, 9, 1024, "f32", "f32", p, False, words=(-1, 2 ** 62 + 3))


@pytest.mark.parametrize("limit", [-1, 0, 1, 11, 30])
def test_dropout_limit(rd_lib, limit):
    _check_dropout(rd_lib, 11, 264, "bf16", "f32", 0.3, True, limit=limit)


def test_dropout_of_special_values(rd_lib):
    """A dropped infinity or NaN is 0; a kept one stays."""
    x = torch.full((8, 64), float("inf"))
    x[:, ::2] = float("nan")
    words = torch.tensor([3, 4], device=DEV)
    got = rd_lib.dropout_rows(x.to(DEV), words, 0.5).cpu()
    kept = torch.from_numpy(block.dropout(np.ones((8, 64)), 3, 4, 0.5)[1])
    assert bool((got[~kept] == 0).all()) and not bool(torch.isfinite(got[kept]).any())


def test_dropout_gradient_draws_the_same(rd_lib):
    x = torch.randn(50, 520, device=DEV)
    words = torch.tensor([99, 7], device=DEV)
    out = rd_lib.dropout_rows(x, words, 0.4)
    grad = rd_lib.dropout_rows(torch.ones_like(x, dtype=torch.bfloat16), words, 0.4, out_dtype=torch.float32)
    assert torch.equal(out, x * grad)


# ---------------------------------------------------------------------------- how the calls are made
def _calls(rd, g):
    """One call of each entry point: name -> function of a stream that gives tensors."""
    def n(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    x, w, b = n(300, 520), n(520, 264), n(264, dtype=torch.float32)
    gain, words, limit = n(520, dtype=torch.float32), torch.tensor([5, 6], device=DEV), _i32([250])
    big, wg, bg, sizes = n(2600, 520), n(3, 520, 264), n(3, 264, dtype=torch.float32), _i32([700, 0, 1900])
    d, pre = n(2600, 264), n(2600, 264)
    f, wide, few = rd.layer_norm_fwd(x, gain), n(90, 20000), _i32([7, 0, 20])
    fw = rd.layer_norm_fwd(wide)
    return {
        "norm": lambda **kw: rd.layer_norm_fwd(x, gain, gain, out_dtype=torch.float32, **kw),
        "norm_bwd": lambda **kw: rd.layer_norm_bwd(x, x, gain, f.mean, f.rstd, **kw),
        "norm_bwd_wide": lambda **kw: rd.layer_norm_bwd(wide, wide, None, fw.mean, fw.rstd, **kw),
        "split": lambda **kw: (rd.linear(x, w, b, act=2, **kw),),
        "linear": lambda **kw: rd.linear(big, wg, bg, act=4, group_sizes=sizes, save_pre=True, **kw),
        "experts": lambda **kw: rd.linear(big[:30], wg, bg, act=2, group_sizes=few, save_pre=True, **kw),
        "act_bwd": lambda **kw: rd.linear_act_bwd(d, pre, 3, group_sizes=sizes, **kw),
        "act_bwd_few": lambda **kw: rd.linear_act_bwd(d[:100], pre[:100], 3, **kw),
        "dropout": lambda **kw: (rd.dropout_rows(x, words, 0.2, residual=x, **kw),),
    }, (words, limit, x, sizes)


def test_streams_repeats_and_graphs(rd_lib):
    """Each call on the current stream, a side stream and a stream argument, twice, and from a graph whose
    inputs and device words change between replays: the same bits every time."""
    calls, (words, limit, x, sizes) = _calls(rd_lib, torch.Generator().manual_seed(1))
    side = torch.cuda.Stream()
    graphs = {}
    for name, call in calls.items():
        first = [t.clone() for t in call()]
        for _ in range(3):
            assert all(torch.equal(a, c) for a, c in zip(first, call())), name
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = call()
        given = call(stream=side)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, other)), name
        assert all(torch.equal(a, c) for a, c in zip(first, given)), name
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = call()
        graphs[name] = (graph, captured)
    words.copy_(torch.tensor([77, 78]))
    x.mul_(0.5)
    sizes.copy_(_i32([1000, 600, 900]))
    for name, (graph, captured) in graphs.items():
        graph.replay()
    torch.cuda.synchronize()
    for name, (graph, captured) in graphs.items():
        want = calls[name]()
        assert all(torch.equal(a, c) for a, c in zip(captured, want)), name


def test_graphs_that_run_at_once_keep_their_own_workspaces(rd_lib):
    """Two captured gradients replayed on two streams at the same time."""
    g = torch.Generator().manual_seed(3)
    sets = []
    for i in range(2):
        x = torch.randn(3000, 1024, generator=g).to(DEV)
        f = rd_lib.layer_norm_fwd(x)
        want = [t.clone() for t in rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)]
        pre = torch.randn(3000, 264, generator=g).to(torch.bfloat16).to(DEV)
        want2 = [t.clone() for t in rd_lib.linear_act_bwd(pre, pre, 2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)
            got2 = rd_lib.linear_act_bwd(pre, pre, 2)
        sets.append((graph, torch.cuda.Stream(), list(got) + list(got2), want + want2, x, f, pre))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in sets:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, *_ in sets:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals(rd_lib):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(64, 72, dtype=torch.bfloat16, device=DEV)
    v, many = torch.zeros(64, device=DEV), torch.zeros(1000, 64, dtype=torch.bfloat16, device=DEV)
    words = torch.zeros(2, dtype=torch.int64, device=DEV)
    st = torch.zeros(4, device=DEV)
    gs = _i32([4])
    bad = [
        lambda: rd_lib.layer_norm_fwd(x.t(), None), lambda: rd_lib.layer_norm_fwd(x.half()),
        lambda: rd_lib.layer_norm_fwd(x.cpu()), lambda: rd_lib.layer_norm_fwd(x, v.bfloat16()),
        lambda: rd_lib.layer_norm_fwd(x, v[:8]), lambda: rd_lib.layer_norm_fwd(x, out_dtype=torch.float16),
        lambda: rd_lib.layer_norm_fwd(x, out=rd_lib.LayerNorm(x.clone(), st, None)),
        lambda: rd_lib.layer_norm_bwd(x[:2], x, None, st, st), lambda: rd_lib.layer_norm_bwd(x, x, None, st[:2], st),
        lambda: rd_lib.linear(x, w[:8]), lambda: rd_lib.linear(x.float(), w), lambda: rd_lib.linear(x, w, v),
        lambda: rd_lib.linear(x, w.unsqueeze(0)), lambda: rd_lib.linear(x, w, group_sizes=gs),
        lambda: rd_lib.linear(x, w, group_offset=1), lambda: rd_lib.linear(x, w, residual=torch.zeros(4, 72, device=DEV)),
        lambda: rd_lib.linear(x, w.unsqueeze(0), group_sizes=gs.long()),
        lambda: rd_lib.linear_act_bwd(x, x.float(), 1), lambda: rd_lib.linear_act_bwd(x.half(), x, 1),
        lambda: rd_lib.dropout_rows(x, words.int(), 0.1), lambda: rd_lib.dropout_rows(x, words[:1], 0.1),
        lambda: rd_lib.dropout_rows(x, words, 0.1, residual=x.float(), out_dtype=torch.bfloat16),
        lambda: rd_lib.dropout_rows(x, words, 0.1, limit=torch.zeros(2, dtype=torch.int32, device=DEV)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    for call in (lambda: rd_lib.layer_norm_fwd(x, eps=-1.0), lambda: rd_lib.linear(x, w, act=9),
                 lambda: rd_lib.linear_act_bwd(x, x, 0), lambda: rd_lib.linear_act_bwd(x, None, 2),
                 lambda: rd_lib.dropout_rows(x, words, 1.5), lambda: rd_lib.dropout_rows(x, words, 0.1, out=x),
                 lambda: rd_lib.linear_act_bwd(many, many, 1, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
                 lambda: rd_lib.layer_norm_fwd(torch.zeros(4, 12, device=DEV)),
                 lambda: rd_lib.layer_norm_fwd(torch.zeros(4 * 64 + 4, device=DEV)[4:].view(4, 64))):
        with pytest.raises(rd_lib.RdError):
            call()


# ---------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["split", "single", "pair"])
def test_timeout_unwinds_and_reports(rd_lib, which, ot):
    """With a bound of 1 ns every wait that its first tries (of a microsecond each) do not end gives up: the
    call reports it and the next one is right.  The waits of the kernel for few tiles, and those of f32 outputs
    for each 512 of k, can be shorter than the tries when nothing else runs, so there a call that reports nothing has to be
    right itself."""
    rng = np.random.default_rng(2)
    m, k, n = (40, 16384, 512) if which == "split" else (1024, 8192, 512)
    x, w = _rows(rng, (m, k), "bf16").to(DEV), _rows(rng, (k, n), "bf16", 1 / math.sqrt(k)).to(DEV)
    status = _i32([0])
    args = dict(act=block.SILU, status=status, out_dtype=ot)
    if which != "split":
        w, args["group_sizes"] = w.unsqueeze(0), _i32([m])
    v = rd_lib.VARIANT_PAIR if which == "pair" else rd_lib.VARIANT_SINGLE
    with rd_lib.tuning(variant=v, wait_timeout_ns=1):
        bounded = rd_lib.linear(x, w, **args)
    torch.cuda.synchronize()
    reported = int(status.item()) & rd_lib.STATUS_TIMEOUT
    assert reported or which == "split" or ot is torch.float32
    status.zero_()
    with rd_lib.tuning(variant=v):
        out = rd_lib.linear(x, w, **args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert reported or torch.equal(out, bounded)
    x64, w64 = _f64(x), _f64(w).reshape(k, n)
    ref, z = block.linear(x64, w64, kind=block.SILU)
    tol = 1.2 * 2.0 ** -22 * (k + 16) * (np.abs(x64) @ np.abs(w64)) + _act_tol(z, block.SILU) + 2.0 ** -8 * np.abs(ref)
    assert_close(_f64(out), ref, tol, "after a timed-out call")
