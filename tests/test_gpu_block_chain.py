"""The block of examples/feed_forward_block.py (norm, router, experts beside a dense feed-forward, dropout onto
an f32 residual stream): a training step against automatic differentiation in 64 bits, its forward from a
CUDA graph, one decoding token."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import block as oblock

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOKENS, HIDDEN, EXPERTS, TOPK, INNER, DENSE = 40, 64, 8, 2, 32, 96
P = 0.25
WORDS = (41, 1 << 40)


@pytest.fixture(scope="module")
def example(rd_lib):
    path = os.path.join(ROOT, "examples", "feed_forward_block.py")
    spec = importlib.util.spec_from_file_location("feed_forward_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _block(example, seed, device=DEV):
    return example.make_block(TOKENS, EXPERTS, HIDDEN, INNER, DENSE, seed=seed, device=device)


def _forward64(p, ids, kept):
    """The block in 64 bits with the choice of experts and the kept elements held fixed."""
    x = p["x"]
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    n = (x - mean) / torch.sqrt(var + 1e-5) * p["gain"] + p["shift"]
    logits = n @ p["wr"] + p["br"]
    weights = torch.softmax(torch.gather(logits, 1, ids), 1)
    mixed = torch.zeros_like(x)
    for t in range(TOKENS):
        for k in range(TOPK):
            e = int(ids[t, k])
            fused = n[t] @ p["up"][e]
            gate, up = fused[:INNER], fused[INNER:]
            mixed[t] = mixed[t] + weights[t, k] * ((gate * torch.sigmoid(gate) * up) @ p["down"][e])
    z = n @ p["w1"] + p["b1"]
    both = (z * torch.special.ndtr(z)) @ p["w2"] + p["b2"] + mixed
    least = oblock.dropout_threshold(P)
    return torch.where(kept, both * (65536 / (65536 - least)), torch.zeros_like(both)) + x


def test_training_step(example):
    params = _block(example, 1, "cpu")
    p = {k: v.to(DEV) for k, v in params.items()}
    words = torch.tensor(WORDS, device=DEV)
    out, saved = example.forward(p, TOPK, words, P)
    d_out = torch.randn(TOKENS, HIDDEN, generator=torch.Generator().manual_seed(2))
    grads = example.backward(d_out.to(DEV), saved, p, words, P)

    ids = saved[2].ids.long().cpu()
    kept = torch.from_numpy(oblock.dropout(np.ones((TOKENS, HIDDEN)), *WORDS, P)[1])
    p64 = {k: v.double().requires_grad_(True) for k, v in params.items()}
    ref = _forward64(p64, ids, kept)
    ref.backward(d_out.double())
    # a chain of bf16 roundings, 2^-8 each of terms of unit size: norm, two products a branch, activation, sum
    err = (out.double().cpu() - ref.detach()).abs().max()
    assert float(err) <= 2.0 ** -4 * max(1.0, float(ref.detach().abs().max()))
    rng = np.random.default_rng(0)
    for name, want in ((k, v.grad) for k, v in p64.items()):
        got = grads[name].double().cpu()
        assert got.shape == want.shape, name
        # each element carries some five independent roundings of 2^-8: 2^-6 of the norm, and no direction
        # is off by more than that noise
        rel = float((got - want).norm() / want.norm())
        assert rel <= 2.0 ** -5, (name, rel)
        way = torch.from_numpy(rng.normal(size=tuple(want.shape)))
        noise = 2.0 ** -5 * float(((want * way) ** 2).sum().sqrt())
        assert abs(float(((got - want) * way).sum())) <= 5 * noise + 2.0 ** -6 * abs(float((want * way).sum())), name


def test_gradients_against_differences(example):
    """The gradients of the 64-bit block are those of its differences, so that the test above means what it says."""
    p = {k: v.double() for k, v in _block(example, 3, "cpu").items()}
    ids = torch.randint(0, EXPERTS, (TOKENS, TOPK), generator=torch.Generator().manual_seed(4))
    kept = torch.from_numpy(oblock.dropout(np.ones((TOKENS, HIDDEN)), *WORDS, P)[1])
    d = torch.randn(TOKENS, HIDDEN, generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    leaf = {k: v.clone().requires_grad_(True) for k, v in p.items()}
    _forward64(leaf, ids, kept).backward(d)
    for name in ("x", "gain", "w1", "b1", "up", "wr"):
        way = torch.randn(p[name].shape, generator=torch.Generator().manual_seed(6), dtype=torch.float64)
        h = 1e-6
        up, dn = dict(p), dict(p)
        up[name], dn[name] = p[name] + h * way, p[name] - h * way
        want = float((d * (_forward64(up, ids, kept) - _forward64(dn, ids, kept))).sum() / (2 * h))
        got = float((leaf[name].grad * way).sum())
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), name


def test_forward_from_a_graph(example):
    """One capture, replayed with other tokens and other words of the generator: the eager call's bits."""
    p = _block(example, 7)
    words = torch.tensor(WORDS, device=DEV)
    example.forward(p, TOPK, words, P)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = example.forward(p, TOPK, words, P)
    seen = []
    for i in range(3):
        p["x"].copy_(_block(example, 20 + i)["x"])
        words.add_(1)
        graph.replay()
        got = captured.clone()
        assert torch.equal(got, example.forward(p, TOPK, words, P)[0])
        seen.append(got)
    assert not torch.equal(seen[0], seen[1])


def test_one_decoding_token(example, rd_lib):
    """A single token through the dense part, as a decoding step calls it."""
    dev = _block(example, 9)
    p = {k: v.cpu() for k, v in dev.items()}
    x = dev["x"][:1].contiguous()
    n = rd_lib.layer_norm_fwd(x, dev["gain"], dev["shift"], out_dtype=torch.bfloat16, stats=False)
    assert n.mean is None and n.rstd is None
    u = rd_lib.linear(n.out, dev["w1"], dev["b1"], act=rd_lib.ACT_GELU)
    out = rd_lib.linear(u, dev["w2"], dev["b2"], residual=x, out_dtype=torch.float32)
    p64 = {k: v.double() for k, v in p.items()}
    ref, _, _ = oblock.layer_norm(p64["x"][:1].numpy(), p64["gain"].numpy(), p64["shift"].numpy())
    z = ref @ p64["w1"].numpy() + p64["b1"].numpy()
    want = oblock.act(z, oblock.GELU) @ p64["w2"].numpy() + p64["b2"].numpy() + p64["x"][:1].numpy()
    # two bf16 roundings on the way (norm, activation), each 2^-8 of values that add up in quadrature
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -5 * max(1.0, np.abs(want).max())


def test_example_runs(example):
    assert torch.isfinite(example.main([])).all()


def test_first_calls_inside_a_capture(rd_lib):
    """Widths and types that no call has had yet: kernel attributes are set while the stream is captured."""
    x = torch.randn(5, 136, device=DEV)
    y = torch.randn(5, 6008, device=DEV, dtype=torch.bfloat16)
    for v in (x, y):                                   # the entry points themselves have been called before
        f = rd_lib.layer_norm_fwd(torch.ones(2, 64, device=DEV))
        rd_lib.layer_norm_bwd(torch.ones(2, 64, device=DEV), torch.ones(2, 64, device=DEV), None, f.mean, f.rstd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for v in (x, y):
            f = rd_lib.layer_norm_fwd(v)
            got += [f.out, *rd_lib.layer_norm_bwd(v, v, None, f.mean, f.rstd)]
    graph.replay()
    torch.cuda.synchronize()
    want = []
    for v in (x, y):
        f = rd_lib.layer_norm_fwd(v)
        want += [f.out, *rd_lib.layer_norm_bwd(v, v, None, f.mean, f.rstd)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
