"""Layer norm, linear products and dropout past 2^31 elements, at the widest rows, and from several threads."""
import threading

import numpy as np
import pytest

from oracle import block

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def _pick(rows):
    return [0, 1, rows // 3, rows // 2, rows - 2, rows - 1]


@pytest.mark.parametrize("rows,hidden", [((1 << 31) // 4096 + 3000, 4096), ((1 << 28) + 1001, 8)])
def test_norm_past_2_31_elements(rd_lib, rows, hidden):
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(rows, hidden, generator=g, device=DEV, dtype=torch.bfloat16)
    f = rd_lib.layer_norm_fwd(x, out_dtype=torch.bfloat16)
    at = _pick(rows)
    ref, mean, rstd = block.layer_norm(x[at].double().cpu().numpy())
    assert np.abs(f.out[at].double().cpu().numpy() - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4
    assert np.abs(f.mean[at].double().cpu().numpy() - mean).max() <= 1e-5
    d_x, d_w, d_b = rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)
    want, _, _ = block.layer_norm_bwd(x[at].double().cpu().numpy(), x[at].double().cpu().numpy(), None,
                                      f.mean[at].double().cpu().numpy(), f.rstd[at].double().cpu().numpy())
    assert np.abs(d_x[at].double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-4
    total = sum(x[i:i + (1 << 24)].sum(0, dtype=torch.float64) for i in range(0, rows, 1 << 24))
    mass = sum(x[i:i + (1 << 24)].abs().sum(0, dtype=torch.float64) for i in range(0, rows, 1 << 24))
    # a block adds rows / blocks of them in order (at most 2^20 here), the rest in a tree: rounding errors of
    # half an ulp each, independent: 2^10 u of the sum of magnitudes, four times over
    assert bool(((d_b.double() - total).abs() <= 4 * 2.0 ** 10 * U * mass).all())


def test_dropout_past_2_31_elements(rd_lib):
    rows, hidden = (1 << 31) // 8192 + 777, 8192
    x = torch.ones(rows, hidden, device=DEV, dtype=torch.bfloat16)
    out = rd_lib.dropout_rows(x, torch.tensor([7, 8], device=DEV), 0.3)
    least = block.dropout_threshold(0.3)
    for r in _pick(rows):
        kept = block.dropout_draws(7, 8, r * (hidden // 8), hidden // 8).reshape(-1) >= least
        assert np.array_equal(out[r].float().cpu().numpy() != 0, kept), r


def test_linear_past_2_31_elements(rd_lib):
    """Output rows past 2^31 elements in one weight and by expert, and their activation gradient."""
    m, k, n = 140000, 64, 16384
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(m, k, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(2, k, n, generator=g, device=DEV, dtype=torch.bfloat16) / 8
    b = torch.randn(2, n, generator=g, device=DEV)
    sizes = torch.tensor([100000, 40000], dtype=torch.int32, device=DEV)
    out, pre = rd_lib.linear(x, w, b, act=block.SILU, group_sizes=sizes, save_pre=True)
    one = rd_lib.linear(x, w[1].contiguous(), b[1].contiguous(), act=block.SILU)
    at = _pick(m) + [99999, 100000]
    for r in at:
        j = int(r >= 100000)
        z = x[r].double() @ w[j].double() + b[j].double()
        ref = z * torch.sigmoid(z)
        assert float((out[r].double() - ref).abs().max()) <= 2.0 ** -8 * float(ref.abs().max()) + 1e-4, r
        assert float((pre[r].double() - z).abs().max()) <= 2.0 ** -8 * float(z.abs().max()) + 1e-4, r
        if j:
            assert torch.equal(one[r], out[r])
    d_pre, d_bias = rd_lib.linear_act_bwd(out, pre, block.SILU, group_sizes=sizes)
    for r in at:
        z = pre[r].double()
        s = torch.sigmoid(z)
        ref = out[r].double() * s * (1 + z * (1 - s))
        assert float((d_pre[r].double() - ref).abs().max()) <= 2.0 ** -8 * float(ref.abs().max()) + 1e-4, r
    parts = d_pre[100000:].double()[:, ::512].sum(0)
    mass = d_pre[100000:].double()[:, ::512].abs().sum(0)
    # of the unrounded products, so the roundings of d_pre to bf16 (independent) stand between them
    assert bool(((d_bias[1, ::512].double() - parts).abs() <= 2.0 ** -8 * mass / 40000 ** 0.5 * 8).all())


def test_widest_rows(rd_lib):
    """Rows of 2^24 elements and weights of 2^22 columns."""
    x = torch.randn(3, 1 << 24, device=DEV, dtype=torch.bfloat16)
    f = rd_lib.layer_norm_fwd(x, out_dtype=torch.float32)
    ref = torch.nn.functional.layer_norm(x.double(), (x.shape[1],), eps=1e-5)
    assert float((f.out.double() - ref).abs().max()) <= 1e-5
    d_x, d_w, d_b = rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)
    assert float((d_b.double() - x.double().sum(0)).abs().max()) <= 1e-5
    assert torch.equal(rd_lib.dropout_rows(x, torch.tensor([1, 2], device=DEV), 0.0), x)
    w = torch.randn(64, 1 << 22, device=DEV, dtype=torch.bfloat16)
    a = torch.randn(5, 64, device=DEV, dtype=torch.bfloat16)
    out = rd_lib.linear(a, w, out_dtype=torch.float32)
    cols = torch.arange(0, 1 << 22, 4099, device=DEV)
    ref = a.double() @ w[:, cols].double()
    assert float((out[:, cols].double() - ref).abs().max()) <= 1e-4
    d_pre, d_bias = rd_lib.linear_act_bwd(out, None, block.NONE)
    assert float((d_bias[cols].double() - out[:, cols].double().sum(0)).abs().max()) <= 1e-4


def test_threads(rd_lib):
    """Calls from four threads, each on its own stream, give what one thread gives."""
    g = torch.Generator().manual_seed(5)
    sets = []
    for i in range(4):
        x = torch.randn(300 + 40 * i, 520, generator=g).to(torch.bfloat16).to(DEV)
        w = torch.randn(520, 264, generator=g).to(torch.bfloat16).to(DEV)
        words = torch.tensor([i, i + 1], device=DEV)
        sets.append((x, w, words))

    def work(x, w, words):
        f = rd_lib.layer_norm_fwd(x)
        u, pre = rd_lib.linear(f.out, w, act=block.GELU, save_pre=True)
        d, b = rd_lib.linear_act_bwd(u, pre, block.GELU)
        grads = rd_lib.layer_norm_bwd(x, x, None, f.mean, f.rstd)
        return [f.out, u, pre, d, b, *grads, rd_lib.dropout_rows(x, words, 0.3)]

    want = [[t.clone() for t in work(*s)] for s in sets]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = work(*sets[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
