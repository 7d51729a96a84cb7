"""4-bit microscaled rows and their grouped product on the GPU against the float64 oracle.

Quantisation and its inverse: bit for bit.  Product: the tolerance of the bf16 products
(parity_util: two bf16 ulps and 1e-3 sqrt(k) max|a| max|b|; the operands' products are exact here).
SiLU-GLU: that tolerance carried through the derivatives.  4-bit output: every code must be that of a
value within the GLU's tolerance (less the bf16 rounding, which it does not have) of the float64 one, at
a scale that a largest magnitude within that tolerance has.
"""
import math

import numpy as np
import pytest

import oracle
from oracle import bf16 as obf
from oracle import glu as oglu
from oracle import moe
from parity_util import assert_close, gemm_tol, glu_epilogue_tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
SENT = 0x3C3C


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _width(k):
    return (k // 32 + 15) // 16 * 16


def _rows4(rng, shape):
    """Random 4-bit rows: (q, scales with 0xFF in the bytes nobody may read, float64 values)."""
    codes, byte = moe.mx_quantize(rng.normal(size=shape) * np.exp(rng.normal(size=shape[:-1] + (1,))))
    scales = np.full(shape[:-1] + (_width(shape[-1]),), 0xFF, np.uint8)
    scales[..., :shape[-1] // 32] = byte
    return moe.mx_pack(codes), scales, moe.mx_values(codes, byte)


@pytest.mark.parametrize("rows,k", [(1, 32), (5, 64), (3, 288), (17, 512), (2, 1056), (40, 4096)])
def test_quantize(rd_lib, rows, k):
    rng = np.random.default_rng(rows * k)
    x = rng.normal(size=(rows, k)) * np.exp(4 * rng.normal(size=(rows, 1)))
    x[rng.random(x.shape) < 0.05] = 0.0
    x[0, :32] = 0.0                                          # an empty block
    x[-1, -32:] = np.linspace(-6, 6, 32)                     # the scale's own levels and beyond
    xt = _bf16(x)
    special = xt.clone()
    if rows > 2:
        special[1, 3] = float("inf")
        special[2, k - 1] = float("nan")
        special[2, 0] = 3.3e38                               # the largest exponents
        special[1, 40 % k] = 1e-40 if k > 32 else 0.0        # a subnormal
    for v in (xt, special):
        q, s = rd_lib.mxfp4_quantize(v.to(DEV))
        codes, byte = moe.mx_quantize(v.double().numpy())
        got = s.cpu().numpy()
        np.testing.assert_array_equal(got[:, :k // 32], byte)
        assert np.all(got[:, k // 32:] == 0)
        gc = moe.mx_unpack(q.cpu().numpy())
        # a zero keeps its sign; so does the oracle's
        np.testing.assert_array_equal(gc, np.where((byte == 255).repeat(32, -1).reshape(codes.shape), 0, codes))
        back = rd_lib.mxfp4_dequantize(q, s).double().cpu().numpy()
        np.testing.assert_array_equal(back, moe.mx_values(gc, byte))


def test_every_code_and_scale_dequantizes(rd_lib):
    codes = np.tile(np.arange(16, dtype=np.uint8), 2)[None].repeat(256, 0)
    scales = np.zeros((256, 16), np.uint8)
    scales[:, 0] = np.arange(256)
    got = rd_lib.mxfp4_dequantize(torch.from_numpy(moe.mx_pack(codes)).to(DEV), torch.from_numpy(scales).to(DEV))
    ref = moe.mx_values(codes, scales[:, :1])
    # 6 x 2^127 and 4 x 2^127 are beyond bf16: infinities, as the rounding to bf16 gives
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.sign(ref) * np.inf, ref)
    np.testing.assert_array_equal(got.double().cpu().numpy(), ref)


def test_quantize_to_packed_rows(rd_lib):
    rng = np.random.default_rng(9)
    tokens, topk, k, rows = 37, 5, 1056, 200
    pos = np.full(tokens * topk, -1)
    pos[rng.random(tokens * topk) < 0.9] = 0
    n = int((pos == 0).sum())
    pos[pos == 0] = rng.choice(rows, n, replace=False)
    pos = pos.reshape(tokens, topk)
    pos[3, 2] = rows                                          # outside: skipped
    x = _bf16(rng.normal(size=(tokens, k))).to(DEV)
    out = rd_lib.Mxfp4(torch.full((rows, k // 2), 0xEE, dtype=torch.uint8, device=DEV),
                       torch.full((rows, _width(k)), 0xEE, dtype=torch.uint8, device=DEV))
    rd_lib.mxfp4_quantize(x, pos=_i32(pos), out_rows=rows, out=out, limit=_i32([30]))
    plain = rd_lib.mxfp4_quantize(x)
    want_q = np.full((rows, k // 2), 0xEE, np.uint8)
    want_s = np.full((rows, _width(k)), 0xEE, np.uint8)
    for t in range(30):
        for p in pos[t]:
            if 0 <= p < rows:
                want_q[p] = plain.q[t].cpu().numpy()
                want_s[p] = plain.scales[t].cpu().numpy()
    np.testing.assert_array_equal(out.q.cpu().numpy(), want_q)
    np.testing.assert_array_equal(out.scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("g,k,n", [(1, 32, 8), (3, 96, 264), (2, 544, 40)])
def test_quantize_weights(rd_lib, g, k, n):
    rng = np.random.default_rng(k)
    rhs = _bf16(rng.normal(size=(g, k, n)))
    if k > 64:
        rhs[1, 40, 3] = float("nan")
    q, s = rd_lib.mxfp4_quantize_weights(rhs.to(DEV))
    codes, byte = moe.mx_quantize(rhs.double().numpy().transpose(0, 2, 1))
    codes = np.where((byte == 255).repeat(32, -1).reshape(codes.shape), 0, codes)
    np.testing.assert_array_equal(moe.mx_unpack(q.cpu().numpy()), codes)
    np.testing.assert_array_equal(s.cpu().numpy()[..., :k // 32], byte)
    assert np.all(s.cpu().numpy()[..., k // 32:] == 0)


# ---------------------------------------------------------------------------- product
@pytest.fixture(params=["pair", "single"])
def variant(request, rd_lib):
    v = rd_lib.VARIANT_PAIR if request.param == "pair" else rd_lib.VARIANT_SINGLE
    with rd_lib.tuning(variant=v, band_rows=512):      # bands of two or four m-tiles
        yield request.param


EDGE = [0, 1, 127, 128, 129, 0, 255, 3]        # rows around a tile, empty groups; 643 in all


def _problem(rng, m, k, n, gl):
    aq, a_s, a = _rows4(rng, (m, k))
    bq, b_s, b = _rows4(rng, (gl, n, k))
    b = b / math.sqrt(k)                        # kept near unit size: an exact power of two below
    e = int(round(math.log2(math.sqrt(k))))
    b = b * math.sqrt(k) * 2.0 ** -e
    b_s[..., :k // 32] -= e
    return aq, a_s, a, bq, b_s, b


def _run(rd, epi, m, k, n, sizes, off=0, gl=None, limit=None, seed=0):
    rng = np.random.default_rng(seed)
    gl = len(sizes) - off if gl is None else gl
    aq, a_s, a, bq, b_s, b = _problem(rng, m, k, n, gl)
    bounds, L = oracle.group_bounds(sizes, m, limit)
    a_s[L:] = 0xFF                              # rows past the limit are all NaN
    dev = [torch.from_numpy(v).to(DEV) for v in (aq, a_s, bq, b_s)]
    n_out = n if epi == rd.EPI_NONE else n // 2
    status = _i32([0])
    kw = dict(group_offset=off, limit=None if limit is None else _i32([limit]), epilogue=epi, status=status)
    local = np.zeros(m, bool)
    local[bounds[off]:bounds[off + gl]] = True
    zero = ~local
    zero[L:] = False
    plain = oracle.ragged_dot(np.nan_to_num(a), b.transpose(0, 2, 1), sizes, off, limit)
    amax = np.abs(a[:L]).max() if L else 0.0
    bmax = np.abs(b).max()
    E = 1e-3 * math.sqrt(k) * amax * bmax
    if epi == rd.EPI_SILU_GLU_MXFP4:
        width = _width(n_out)
        out = torch.full((m + 4, n_out // 2), 0xEE, dtype=torch.uint8, device=DEV)
        scales = torch.full((m + 4, width), 0xEE, dtype=torch.uint8, device=DEV)
        rd.ragged_dot_mxfp4(*dev, _i32(sizes), out=out[:m], out_scales=scales[:m], **kw)
        q, s = out.cpu().numpy(), scales.cpu().numpy()
        assert np.all(q[L:] == 0xEE) and np.all(s[L:] == 0xEE)
        assert np.all(q[:m][zero] == 0) and np.all(s[:m][zero] == 0)
        blocks = n_out // 32
        assert np.all(s[:m][local][:, blocks:] == 0xEE)        # the bytes past the blocks stay
        ref, tol = glu_epilogue_tol(plain[:, :n_out], plain[:, n_out:], E)
        tol = tol - obf.ulp(ref) + 2.0 ** -20 * np.abs(ref)
        r = ref[local].reshape(-1, blocks, 32)
        d = np.broadcast_to(tol, ref.shape)[local].reshape(-1, blocks, 32)
        byte = s[:m][local][:, :blocks].astype(np.int64)
        bytes_of = np.vectorize(moe.mx_scale_byte, otypes=[np.int64])
        lo = bytes_of(np.maximum(np.abs(r) - d, 0).max(-1))
        hi = bytes_of((np.abs(r) + d).max(-1))
        assert np.all((byte >= lo) & (byte <= hi))
        codes = moe.mx_unpack(q[:m][local]).reshape(r.shape)
        got = moe.LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
        f = np.exp2(byte - 127.0)[..., None]

        def level(v):
            c = moe.mx_round(v)
            return moe.LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)

        assert np.all(level((r - d) / f) <= got) and np.all(got <= level((r + d) / f))
        assert int(status.item()) == 0
        return q, s
    buf = torch.empty((m + 4, n_out), dtype=torch.bfloat16, device=DEV)
    buf.view(torch.int16).fill_(SENT)
    rd.ragged_dot_mxfp4(*dev, _i32(sizes), out=buf[:m], **kw)
    bits = obf.torch_bf16_bits(buf)
    assert np.all(bits[L:] == SENT) and np.all(bits[:m][zero] == 0)
    got = obf.torch_bf16_to_f64(buf[:m])
    if epi == rd.EPI_SILU_GLU:
        ref, tol = glu_epilogue_tol(plain[:, :n_out], plain[:, n_out:], E)
        np.testing.assert_allclose(ref[local], oglu.glu_fwd_f64(plain[local][:, :n_out], plain[local][:, n_out:]))
    else:
        ref, tol = plain, gemm_tol(plain, k, amax, bmax)
    assert_close(got[local], ref[local], tol[local], "4-bit product")
    assert int(status.item()) == 0
    return bits


@pytest.mark.parametrize("epi", [0, 1, 2])
@pytest.mark.parametrize("k,n", [(32, 64), (224, 192), (256, 448), (544, 384), (800, 832), (1184, 128)])
def test_product(rd_lib, variant, epi, k, n):
    _run(rd_lib, epi, 643, k, n, EDGE, seed=k + n)


@pytest.mark.parametrize("epi,n", [(0, 8), (0, 200), (1, 16), (1, 208)])
def test_product_narrow(rd_lib, variant, epi, n):
    _run(rd_lib, epi, 643, 96, n, EDGE, seed=n)


@pytest.mark.parametrize("epi", [0, 1, 2])
@pytest.mark.parametrize("limit", [0, 1, 127, 300, 642, 700])
def test_product_limit_and_offset(rd_lib, variant, epi, limit):
    _run(rd_lib, epi, 660, 320, 256, EDGE, off=2, gl=3, limit=limit, seed=limit)


@pytest.mark.parametrize("m,sizes", [(1, [1]), (1, [0, 0, 1, 0]), (8, [1] * 8), (5, [0, 0, 0, 2]), (900, [900]),
                                     (2100, [700, 1, 0, 1399]), (17, [9, 9, 9])])
def test_product_group_shapes(rd_lib, variant, m, sizes):
    """Single rows, rows past the groups, many m-tiles (and bands) of one group, sizes past m."""
    rng = np.random.default_rng(m)
    if sum(sizes) > m:
        aq, a_s, a, bq, b_s, b = _problem(rng, m, 96, 64, len(sizes))
        status = _i32([0])
        out = rd_lib.ragged_dot_mxfp4(*[torch.from_numpy(v).to(DEV) for v in (aq, a_s, bq, b_s)], _i32(sizes),
                                      status=status)
        assert int(status.item()) == rd_lib.STATUS_OVERFLOW
        ref = oracle.ragged_dot(a, b.transpose(0, 2, 1), sizes)
        assert_close(obf.torch_bf16_to_f64(out), ref, gemm_tol(ref, 96, np.abs(a).max(), np.abs(b).max()), "clamped")
        return
    for epi in (0, 2):
        _run(rd_lib, epi, m, 288, 384, sizes, seed=m)


@pytest.mark.parametrize("epi", [0, 1, 2])
@pytest.mark.parametrize("k,n,band_rows,limit", [(32, 64, 0, None), (1184, 192, 128, None), (2080, 448, 0, 801),
                                                 (288, 832, 256, 500)])
def test_product_few_rows_a_group(rd_lib, epi, k, n, band_rows, limit):
    """At most 16 rows a group on average: tiles of 32 rows, with groups of several tiles (and bands of
    four or eight tiles) among them."""
    sizes = [0, 1, 31, 32, 33, 64, 65, 200, 2, 250, 0] + [5, 0, 17, 1] * 13
    m = sum(sizes) + 11
    assert m <= 16 * len(sizes)
    with rd_lib.tuning(band_rows=band_rows):
        _run(rd_lib, epi, m, k, n, sizes, off=1, gl=len(sizes) - 3, limit=limit, seed=k + n + epi)


def test_product_of_nothing(rd_lib, variant):
    u8 = dict(dtype=torch.uint8, device=DEV)
    none = rd_lib.ragged_dot_mxfp4(torch.empty((0, 16), **u8), torch.empty((0, 16), **u8), torch.zeros((2, 8, 16), **u8),
                                   torch.zeros((2, 8, 16), **u8), _i32([0, 0]))
    assert none.shape == (0, 8)
    # a contraction of length zero is zero rows
    out = rd_lib.ragged_dot_mxfp4(torch.empty((5, 0), **u8), torch.empty((5, 0), **u8), torch.empty((2, 8, 0), **u8),
                                  torch.empty((2, 8, 0), **u8), _i32([2, 3]))
    assert out.shape == (5, 8) and bool((out == 0).all())


def test_nan_scale_stays_in_its_row_and_column(rd_lib, variant):
    rng = np.random.default_rng(1)
    aq, a_s, a, bq, b_s, b = _problem(rng, 300, 256, 192, 2)
    a_s[7, 3] = 255
    b_s[1, 100, 5] = 255
    out = rd_lib.ragged_dot_mxfp4(*[torch.from_numpy(v).to(DEV) for v in (aq, a_s, bq, b_s)], _i32([150, 150]))
    nan = out.isnan().cpu().numpy()
    want = np.zeros((300, 192), bool)
    want[7] = True
    want[150:, 100] = True
    np.testing.assert_array_equal(nan, want)


def test_product_offsets_past_32_bits(rd_lib):
    """Rows of a and of the output beyond 2^31 bytes: 1.2 million rows of k = 4096 (2.4 GB), one group at
    the far end, the others not local."""
    m, k, n = 1_200_000, 4096, 64
    sizes = [m - 200, 150, 50]
    rng = np.random.default_rng(8)
    q, s, a = _rows4(rng, (200, k))
    bq, b_s, b = _rows4(rng, (2, n, k))
    aq = torch.zeros((m, k // 2), dtype=torch.uint8, device=DEV)
    a_s = torch.zeros((m, 128), dtype=torch.uint8, device=DEV)
    aq[m - 200:] = torch.from_numpy(q).to(DEV)
    a_s[m - 200:] = torch.from_numpy(s).to(DEV)
    out = rd_lib.ragged_dot_mxfp4(aq, a_s, torch.from_numpy(bq).to(DEV), torch.from_numpy(b_s).to(DEV), _i32(sizes),
                                  group_offset=1)
    assert bool((out[:m - 200] == 0).all())
    ref = oracle.ragged_dot(a, b.transpose(0, 2, 1), [150, 50])
    assert_close(obf.torch_bf16_to_f64(out[m - 200:]), ref, gemm_tol(ref, k, np.abs(a).max(), np.abs(b).max()), "far rows")


def test_repeats_graph_and_side_stream(rd_lib, variant):
    """An up product with 4-bit output feeding a down product, eagerly, on a side stream and in a graph
    that follows device-side group sizes: the same bits."""
    rng = np.random.default_rng(6)
    m, d, f, g = 500, 512, 160, 6
    aq, a_s, _, uq, us, _ = _problem(rng, m, d, 2 * f, g)
    _, _, _, dq, ds, _ = _problem(rng, 1, f, d, g)
    a, a_s, uq, us, dq, ds = [torch.from_numpy(v).to(DEV) for v in (aq, a_s, uq, us, dq, ds)]
    gs = _i32([100, 0, 50, 200, 149, 1])

    def chain():
        h = rd_lib.ragged_dot_mxfp4(a, a_s, uq, us, gs, epilogue=rd_lib.EPI_SILU_GLU_MXFP4)
        return rd_lib.ragged_dot_mxfp4(h.q, h.scales, dq, ds, gs)

    want = chain()
    assert torch.equal(chain(), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = chain()
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for sizes in ([100, 0, 50, 200, 149, 1], [0, 0, 0, 0, 0, 500], [1, 2, 3, 4, 5, 6]):
        gs.copy_(torch.tensor(sizes, dtype=torch.int32))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, chain())


def test_timeout_unwinds_and_reports(rd_lib, variant):
    """A 1 ns bound makes every wait give up: the call returns, reports it, and the next one is right."""
    rng = np.random.default_rng(3)
    aq, a_s, a, bq, b_s, b = _problem(rng, 1024, 4096, 512, 4)
    dev = [torch.from_numpy(v).to(DEV) for v in (aq, a_s, bq, b_s)]
    gs = _i32([256, 300, 200, 268])
    want = rd_lib.ragged_dot_mxfp4(*dev, gs)
    status = _i32([0])
    with rd_lib.tuning(wait_timeout_ns=1):
        rd_lib.ragged_dot_mxfp4(*dev, gs, status=status)
    torch.cuda.synchronize()
    with pytest.raises(rd_lib.RdError, match="STATUS_TIMEOUT"):
        rd_lib.check_status(status)
    status.zero_()
    again = rd_lib.ragged_dot_mxfp4(*dev, gs, status=status)
    assert torch.equal(again, want) and int(status.item()) == 0


def test_against_the_bf16_product(rd_lib):
    """The bf16 product of the dequantised operands: the same sums, each rounded to bf16."""
    rng = np.random.default_rng(12)
    sizes = [200, 0, 313, 87]
    x, w = _bf16(rng.normal(size=(600, 1024))).to(DEV), _bf16(rng.normal(size=(4, 1024, 320)) / 32).to(DEV)
    a, b = rd_lib.mxfp4_quantize(x), rd_lib.mxfp4_quantize_weights(w)
    got = rd_lib.ragged_dot_mxfp4(*a, *b, _i32(sizes))
    a16 = rd_lib.mxfp4_dequantize(*a)
    b16 = rd_lib.mxfp4_dequantize(b.q.view(-1, 512), b.scales.view(-1, b.scales.shape[-1])).view(4, 320, 1024)
    ref = rd_lib.ragged_dot(a16, b16.transpose(1, 2).contiguous(), _i32(sizes))
    a64, b64 = obf.torch_bf16_to_f64(a16), obf.torch_bf16_to_f64(b16)
    exact = oracle.ragged_dot(a64, b64.transpose(0, 2, 1), sizes)
    tol = gemm_tol(exact, 1024, np.abs(a64).max(), np.abs(b64).max())
    assert_close(obf.torch_bf16_to_f64(got), exact, tol, "4-bit")
    assert_close(obf.torch_bf16_to_f64(ref), exact, tol, "bf16")


def test_binding_refusals(rd_lib):
    u8 = dict(dtype=torch.uint8, device=DEV)
    a, s = torch.zeros((8, 32), **u8), torch.zeros((8, 16), **u8)
    b, bs = torch.zeros((2, 64, 32), **u8), torch.zeros((2, 64, 16), **u8)
    gs = _i32([4, 4])
    rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs)
    for call in (lambda: rd_lib.ragged_dot_mxfp4(a, s[:, :8].contiguous(), b, bs, gs),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b[:, :, :16].contiguous(), bs, gs),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs[:1], gs),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs.long()),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs, out_scales=s),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs, out=torch.zeros((8, 32), **u8)),
                 lambda: rd_lib.mxfp4_quantize(torch.zeros(4, 64, device=DEV)),
                 lambda: rd_lib.mxfp4_dequantize(a, s[:4])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs, group_offset=1),
                 lambda: rd_lib.ragged_dot_mxfp4(a, s, b, bs, gs, epilogue=5),
                 lambda: rd_lib.mxfp4_quantize(torch.zeros(4, 40, dtype=torch.bfloat16, device=DEV)),
                 lambda: rd_lib.mxfp4_quantize_weights(torch.zeros(1, 40, 8, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(rd_lib.RdError):
            call()
