"""rd_trans_ragged_dot_no_alloc against the float64 oracle."""

import numpy as np
import pytest

import oracle
from oracle import bf16 as obf
from parity_util import assert_close, gemm_tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("variant", ["pair", "single"])
def test_no_alloc_dw_is_the_oracles(rd_lib, variant):
    """Two calls in a row with other group sizes: empty groups, sizes off every step of 16 and 64 rows, rows past
    the groups; the output's memory holds NaN before."""
    rng = np.random.default_rng(77)
    k, n = 264, 384
    cases = [[300, 0, 129, 17, 64, 1, 431], [5, 700, 0, 250, 63, 65, 9]]
    m = max(sum(c) for c in cases) + 11
    v = rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE
    with rd_lib.tuning(variant=v):
        for call, sizes in enumerate(cases):
            x, y = (torch.from_numpy(rng.standard_normal((m, w)).astype(np.float32)).to(torch.bfloat16).to(DEV)
                    for w in (k, n))
            gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
            got = torch.full((len(sizes), k, n), float("nan"), dtype=torch.bfloat16, device=DEV)
            assert rd_lib.trans_ragged_dot_no_alloc(x, y, gs, out=got) is got
            x64, y64 = obf.torch_bf16_to_f64(x), obf.torch_bf16_to_f64(y)
            ref = oracle.trans_ragged_dot(x64, y64, sizes)
            g64 = obf.torch_bf16_to_f64(got)
            for j, cnt in enumerate(sizes):
                tol = gemm_tol(ref[j], cnt, np.abs(x64).max(), np.abs(y64).max()) if cnt else 0.0
                assert_close(g64[j], ref[j], tol, f"call {call} group {j} ({cnt} rows)")
