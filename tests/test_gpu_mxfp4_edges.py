"""4-bit rows at the ends of the exponent range and of the extents, bit for bit; a product of many tiles."""
import numpy as np
import pytest

from oracle import moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


def _check(rd_lib, x):
    """Codes, scale bytes and values of bf16 rows x."""
    q, s = rd_lib.mxfp4_quantize(x.to(DEV))
    codes, byte = moe.mx_quantize(x.double().numpy())
    np.testing.assert_array_equal(s.cpu().numpy()[:, :byte.shape[1]], byte)
    np.testing.assert_array_equal(moe.mx_unpack(q.cpu().numpy()), codes)
    back = rd_lib.mxfp4_dequantize(q, s).double().cpu().numpy()
    np.testing.assert_array_equal(back, moe.mx_values(codes, byte))


def test_blocks_of_subnormal_values(rd_lib):
    """Blocks whose largest magnitude is a bf16 subnormal or among the lowest normal numbers: scale byte 0, 1, 2."""
    rng = np.random.default_rng(3)
    bits = [rng.integers(0, top, (4, 32)) for top in (2, 5, 0x20, 0x40, 0x80, 0x100, 0x180, 0x200, 0x280)]
    bits.append(np.arange(4 * 32).reshape(4, 32))               # every subnormal, block by block
    bits.append(np.arange(0x80, 0x80 + 4 * 32).reshape(4, 32))  # the numbers above them
    bits = np.concatenate(bits) | (rng.integers(0, 2, (44, 32)) << 15)
    x = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    _check(rd_lib, x)
    _check(rd_lib, x.reshape(1, -1))
    w = x.t().contiguous()[None].to(DEV)                         # the same blocks as columns of a weight
    w = torch.cat((w, torch.zeros(1, 32, 4, dtype=torch.bfloat16, device=DEV)), 2)
    q, s = rd_lib.mxfp4_quantize_weights(w)
    codes, byte = moe.mx_quantize(x.double().numpy())
    np.testing.assert_array_equal(moe.mx_unpack(q[0, :44].cpu().numpy()), codes)
    np.testing.assert_array_equal(s[0, :44, :1].cpu().numpy(), byte)


def test_blocks_of_the_largest_values(rd_lib):
    """Blocks up to the largest finite bf16 number, and those that reach beyond four of the scale's sixes."""
    rng = np.random.default_rng(4)
    bits = np.concatenate([rng.integers(0x7F80 - span, 0x7F80, (4, 32)) for span in (1, 0x20, 0x80, 0x100, 0x400, 0x7F80)])
    bits |= rng.integers(0, 2, bits.shape) << 15
    _check(rd_lib, torch.from_numpy(bits.astype(np.uint16).view(np.int16)).view(torch.bfloat16))


def _free(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def test_longest_row(rd_lib):
    """One row of 2^31 - 32 elements, the longest that a call takes, there and back."""
    _free(24)
    k, n = 2 ** 31 - 32, 4096
    x = torch.zeros((1, k), dtype=torch.bfloat16, device=DEV)
    part = torch.randn(1, n, device=DEV).to(torch.bfloat16)
    at = (0, 2 ** 30 + 512, k - n)
    for c in at:
        x[:, c:c + n] = part
    q, s = rd_lib.mxfp4_quantize(x)
    back = rd_lib.mxfp4_dequantize(q, s)
    want = rd_lib.mxfp4_quantize(part)
    values = rd_lib.mxfp4_dequantize(*want)
    for c in at:
        assert torch.equal(q[:, c // 2:(c + n) // 2], want.q)
        assert torch.equal(s[:, c // 32:(c + n) // 32], want.scales)
        assert torch.equal(back[:, c:c + n], values)
    assert not s[:, k // 32:].any()
    assert int(back.count_nonzero()) == len(at) * int(values.count_nonzero())


def test_most_columns_of_a_weight(rd_lib):
    """[1, 32, 2^31 - 8] to 4 bits: the last block of columns is half outside, and is not written."""
    _free(215)
    n, pad = 2 ** 31 - 8, 256
    rhs = torch.empty((1, 32, n), dtype=torch.bfloat16, device=DEV)
    part = torch.randn(1, 32, 512, device=DEV).to(torch.bfloat16)
    at = (0, 2 ** 30 + 8, n - 512)
    for c in at:
        rhs[:, :, c:c + 512] = part
    bufs = [torch.empty((n + pad) * 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for b in bufs:
        b[-16 * pad:] = 0xA5
    out = rd_lib.Mxfp4(*[b[:16 * n].view(1, n, 16) for b in bufs])
    rd_lib.mxfp4_quantize_weights(rhs, out=out)
    want = rd_lib.mxfp4_quantize_weights(part)
    for c in at:
        assert torch.equal(out.q[:, c:c + 512], want.q) and torch.equal(out.scales[:, c:c + 512], want.scales)
    assert all(bool((b[-16 * pad:] == 0xA5).all()) for b in bufs)
    del rhs, bufs, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("k", [4096, 1184])
def test_pair_product_of_many_tiles(rd_lib, k):
    """Hundreds of tiles of many stages on CTA pairs, every element against the float64 product of the same 4-bit
    values within the products' tolerance (two bf16 ulps and 1e-3 sqrt(k) max|a| max|b|), the same bits every time."""
    gen = torch.Generator(device=DEV).manual_seed(k)
    sizes, n = [2600, 0, 1, 3000, 2047, 544], 1536
    m = sum(sizes)
    a = rd_lib.mxfp4_quantize(torch.randn(m, k, generator=gen, device=DEV).to(torch.bfloat16))
    b = rd_lib.mxfp4_quantize_weights(
        (torch.randn(len(sizes), k, n, generator=gen, device=DEV) * k ** -0.5).to(torch.bfloat16))
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR):
        first = rd_lib.ragged_dot_mxfp4(*a, *b, gs, status=status)
        for i in range(30):
            if i % 3 == 0:                       # another kernel's tiles in tensor memory in between
                rd_lib.ragged_dot_mxfp4(*a, *b, gs, epilogue=rd_lib.EPI_SILU_GLU_MXFP4)
            again = rd_lib.ragged_dot_mxfp4(*a, *b, gs, status=status)
            assert torch.equal(again.view(torch.int16), first.view(torch.int16)), i
    assert int(status) == 0
    a64, row = rd_lib.mxfp4_dequantize(*a).double(), 0
    for j, cnt in enumerate(sizes):
        b64 = rd_lib.mxfp4_dequantize(b.q[j], b.scales[j]).double()
        ref = a64[row:row + cnt] @ b64.t()
        ulp = torch.exp2(torch.floor(torch.log2(ref.abs().clamp(min=2.0 ** -126))) - 7)
        tol = 2 * ulp + 1e-3 * k ** 0.5 * a64.abs().max() * b64.abs().max()
        assert bool(((first[row:row + cnt].double() - ref).abs() <= tol).all()), j
        row += cnt
