"""Grouped products at the largest extents: 2^31 - 1 rows in one group, rows of more than 2^31 elements."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
M = 2 ** 31 - 1
ROWS = [0, 1, 127, 128, 255, 2 ** 30, 2 ** 30 + 1, M - 257, M - 256, M - 129, M - 128, M - 2, M - 1]


def _free(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _check(out, want):
    """The rows given have their values, all others are zero."""
    assert torch.equal(out[ROWS], want)
    assert sum(int(c.count_nonzero()) for c in out.split(2 ** 27)) == int(want.count_nonzero())


@pytest.mark.parametrize("variant", ["pair", "single"])
def test_product4_rows(rd_lib, variant):
    _free(130)
    rng = np.random.default_rng(1)
    part = torch.from_numpy(rng.normal(size=(len(ROWS), 32)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w = rd_lib.mxfp4_quantize_weights(
        torch.from_numpy(rng.normal(size=(1, 32, 8)).astype(np.float32)).to(torch.bfloat16).to(DEV))
    a = rd_lib.mxfp4_quantize(part)
    want = rd_lib.ragged_dot_mxfp4(*a, *w, _i32([len(ROWS)]))
    big = [torch.zeros((M, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    for b, v in zip(big, a):
        b[ROWS] = v
    status = _i32([0])
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE):
        out = rd_lib.ragged_dot_mxfp4(*big, *w, _i32([M]), status=status)
    assert int(status) == 0
    _check(out, want)
    del big, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("variant", ["pair", "single"])
def test_product_rows(rd_lib, variant):
    _free(100)
    rng = np.random.default_rng(2)
    part, w = (torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(torch.bfloat16).to(DEV)
               for s in ((len(ROWS), 8), (1, 8, 8)))
    want = rd_lib.ragged_dot(part, w, _i32([len(ROWS)]))
    lhs = torch.zeros((M, 8), dtype=torch.bfloat16, device=DEV)
    lhs[ROWS] = part
    status = _i32([0])
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE):
        out = rd_lib.ragged_dot(lhs, w, _i32([M]), status=status)
    assert int(status) == 0
    _check(out, want)
    del lhs, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("variant", ["pair", "single"])
def test_glu_gradient_of_a_wide_layer(rd_lib, variant):
    """f above 2^30: a row of the fused buffer is more than 2^31 elements long."""
    _free(60)
    rng = np.random.default_rng(3)
    m, f, n, part = 3, 2 ** 30 + 8, 8, 264

    def some(*shape):
        return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(torch.bfloat16).to(DEV)

    d_out, w, gate, up = some(m, n), some(1, part, n), some(m, part), some(m, part)
    want = rd_lib.ragged_dot_trans_rhs_glu_bwd(d_out, w, torch.cat((gate, up), 1), _i32([m]))
    rhs = torch.zeros((1, f, n), dtype=torch.bfloat16, device=DEV)
    fused = torch.zeros((m, 2 * f), dtype=torch.bfloat16, device=DEV)
    for at in (0, 2 ** 29 + 8, f - part):
        rhs[:, at:at + part] = w
        fused[:, at:at + part] = gate
        fused[:, f + at:f + at + part] = up
    status = _i32([0])
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE):
        out = rd_lib.ragged_dot_trans_rhs_glu_bwd(d_out, rhs, fused, _i32([m]), status=status)
    assert int(status) == 0
    for at in (0, 2 ** 29 + 8, f - part):
        assert torch.equal(out[:, at:at + part], want[:, :part])
        assert torch.equal(out[:, f + at:f + at + part], want[:, part:])
    del rhs, fused, out
    torch.cuda.empty_cache()
