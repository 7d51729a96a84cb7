"""4-bit rows at the ends of the exponent range, bit for bit against the float64 oracle."""
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
