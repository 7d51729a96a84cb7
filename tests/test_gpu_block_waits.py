"""Waits inside the kernels of include/rd_block.h that run out: the call returns, what it reports and leaves behind, and the
calls after it."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# kernel for few tiles: rows, k, n, group sizes (None: one weight)
FEW_TILES = {
    "eight share k": (40, 16384, 512, None),
    "four share k": (64, 14336, 4096, None),
    "two share k": (256, 4096, 4096, None),
    "alone": (3, 4096, 14336, None),
    "alone, no wait for a free stage": (3, 256, 14336, None),
    "by group": (30, 4096, 512, [7, 0, 20]),
    "by group, alone": (40, 4096, 4096, [3, 30, 5, 2]),
}


def _linear(rd, which, ot, seed=0):
    """A call of rd_linear on the kernel for few tiles: function of a status word that gives the output."""
    m, k, n, sizes = FEW_TILES[which]
    g = torch.Generator().manual_seed(seed + m)
    lead = () if sizes is None else (len(sizes),)
    x = torch.randn(m, k, generator=g).bfloat16().to(DEV)
    w = (torch.randn(*lead, k, n, generator=g) / math.sqrt(k)).bfloat16().to(DEV)
    b = torch.randn(*lead, n, generator=g).to(DEV)
    gs = None if sizes is None else _i32(sizes)
    return lambda status: rd.linear(x, w, b, act=rd.ACT_SILU, group_sizes=gs, out_dtype=ot, status=status)


@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", list(FEW_TILES))
def test_few_tiles_right_or_reported(rd_lib, which, ot):
    """Bounds from one that no wait keeps to one that nearly all do, so that each role is the one that gives up:
    what is not reported is right, and so is the call after it, on the same memory."""
    call = _linear(rd_lib, which, ot)
    status = _i32([0])
    want = call(status).clone()
    for limit in (1, 1500, 3000, 6000, 12000, 25000) * 3:
        with rd_lib.tuning(wait_timeout_ns=limit):
            bounded = call(status)
        again = call(None)
        torch.cuda.synchronize()
        bits = int(status.item())
        assert bits in (0, rd_lib.STATUS_TIMEOUT)
        assert bits or torch.equal(bounded, want), limit
        assert torch.equal(again, want), limit
        status.zero_()


@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", list(FEW_TILES))
def test_few_tiles_shortest_bound_runs_out(rd_lib, which, ot):
    """No copy lands within a nanosecond, so a bound of one has to run out and be reported, however short the call."""
    call = _linear(rd_lib, which, ot, seed=5)
    status = _i32([0])
    want = call(None).clone()
    for _ in range(3):
        with rd_lib.tuning(wait_timeout_ns=1):
            call(status)
        torch.cuda.synchronize()
        assert int(status.item()) == rd_lib.STATUS_TIMEOUT
        status.zero_()
        assert torch.equal(call(status), want) and int(status.item()) == 0


@pytest.mark.parametrize("ot", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("variant", ["single", "pair"])
@pytest.mark.parametrize("m,k,n,sizes", [(1024, 8192, 512, [1024]), (900, 72, 520, [100, 0, 793, 7]), (3000, 1608, 264, [3000, 0])])
def test_many_tiles_shortest_bound_runs_out(rd_lib, variant, ot, m, k, n, sizes):
    """The persistent kernel, with stretches of k that wait for one another (f32) and with one short one."""
    g = torch.Generator().manual_seed(k)
    x = torch.randn(m, k, generator=g).bfloat16().to(DEV)
    w = (torch.randn(len(sizes), k, n, generator=g) / math.sqrt(k)).bfloat16().to(DEV)
    status, gs = _i32([0]), _i32(sizes)
    with rd_lib.tuning(variant=rd_lib.VARIANT_PAIR if variant == "pair" else rd_lib.VARIANT_SINGLE):
        want = rd_lib.linear(x, w, group_sizes=gs, out_dtype=ot).clone()
        for _ in range(3):
            with rd_lib.tuning(wait_timeout_ns=1):
                rd_lib.linear(x, w, group_sizes=gs, out_dtype=ot, status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == rd_lib.STATUS_TIMEOUT
            status.zero_()
            got = rd_lib.linear(x, w, group_sizes=gs, out_dtype=ot, status=status)
            assert torch.equal(got, want) and int(status.item()) == 0


# rows shared by two, four and eight blocks, several turns each
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,hidden", [(400, 9000), (250, 20000), (120, 40000), (100, 65536)])
def test_norm_gradients_of_long_rows(rd_lib, rows, hidden, dt):
    """Bounds as above: every element of d_x is its own or NaN, all of them NaN with bounds that a block never keeps, the
    column sums need no other block's, and the call after it is right."""
    g = torch.Generator().manual_seed(rows)
    x, d = (torch.randn(rows, hidden, generator=g).to(dt).to(DEV) for _ in range(2))
    w = torch.randn(hidden, generator=g).to(DEV)
    f = rd_lib.layer_norm_fwd(x, w)
    want = [t.clone() for t in rd_lib.layer_norm_bwd(d, x, w, f.mean, f.rstd)]
    assert bool(torch.isfinite(want[0]).all())
    for limit in (1, 500, 1500, 3000, 6000, 12000) * 3:
        with rd_lib.tuning(wait_timeout_ns=limit):
            got = rd_lib.layer_norm_bwd(d, x, w, f.mean, f.rstd)
        again = rd_lib.layer_norm_bwd(d, x, w, f.mean, f.rstd)
        torch.cuda.synchronize()
        late = torch.isnan(got[0])
        assert bool(late.all()) or limit >= 1000, limit
        assert bool(((got[0] == want[0]) | late).all()), limit
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:])), limit
        assert all(torch.equal(a, b) for a, b in zip(again, want)), limit


@pytest.mark.parametrize("limit", [2 ** 63 - 500_000_000, 2 ** 63, 2 ** 64 - 1])
def test_longest_bounds(rd_lib, limit):
    """A wait that takes twice the bound and a second more does not run out early where that leaves 64 bits."""
    status = _i32([0])
    for which in FEW_TILES:
        call = _linear(rd_lib, which, torch.float32, seed=9)
        want = call(None).clone()
        with rd_lib.tuning(wait_timeout_ns=limit):
            assert rd_lib.get_tuning()["wait_timeout_ns"] == limit
            assert torch.equal(call(status), want)
    x = torch.randn(100, 20000, device=DEV)
    f = rd_lib.layer_norm_fwd(x)
    with rd_lib.tuning(wait_timeout_ns=limit):
        assert bool(torch.isfinite(rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)[0]).all())
    assert int(status.item()) == 0
