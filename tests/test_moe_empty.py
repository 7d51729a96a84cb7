"""Calls without rows to write are accepted, with null pointers for what is empty."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3


def _at(i):
    return (i + 1) << 44          # addresses far apart, never dereferenced: nothing is launched


@pytest.fixture(scope="module")
def lib():
    from expert_ffn_ragged_gb300 import build, moe

    lib = ctypes.CDLL(build.build())
    moe.declare(lib)
    return lib


def test_no_packed_rows(lib):
    """A rank whose packed buffer has no row: dispatch, and the quantisation that dispatches."""
    codes = [lib.rd_dispatch_rows(_at(0), _at(1), None, 4, 2, 64, 0, None, None),
             lib.rd_mxfp4_quantize(_at(0), _at(1), None, None, 4, 2, 64, 0, None, None)]
    assert set(codes) <= {OK, CUDA}      # CUDA: past the checks, on a machine without a GPU
    # with a row to write the buffers are needed
    assert lib.rd_mxfp4_quantize(_at(0), _at(1), None, _at(2), 4, 2, 64, 1, None, None) == INVALID
    assert lib.rd_mxfp4_quantize(_at(0), _at(1), _at(2), None, 4, 2, 64, 1, None, None) == INVALID
    assert lib.rd_mxfp4_quantize(_at(0), None, None, None, 4, 1, 64, 0, None, None) == INVALID


@pytest.mark.gpu
def test_quantize_to_no_packed_rows(rd_lib):
    torch = pytest.importorskip("torch")
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    assert rd_lib.dispatch_rows(x, pos, out_rows=0).shape == (0, 64)
    q, s = rd_lib.mxfp4_quantize(x, pos=pos, out_rows=0)
    assert q.shape == (0, 32) and s.shape == (0, 16)
