"""A whole feed-forward block made of the library's calls: norm, router, experts beside a dense feed-forward,
dropout onto an f32 residual stream; a training step against automatic differentiation in 64 bits, and
its forward from a CUDA graph."""
import numpy as np
import pytest

from oracle import block as oblock

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
TOKENS, HIDDEN, EXPERTS, TOPK, INNER, DENSE = 40, 64, 8, 2, 32, 96
P = 0.25
WORDS = (41, 1 << 40)


def _params(seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, dtype=torch.float64) * std + shift

    p = dict(x=n(TOKENS, HIDDEN, shift=0.2), gain=n(HIDDEN, std=0.1, shift=1.0), shift=n(HIDDEN, std=0.1),
             wr=n(HIDDEN, EXPERTS, std=HIDDEN ** -0.5), br=n(EXPERTS, std=0.1),
             up=n(EXPERTS, HIDDEN, 2 * INNER, std=HIDDEN ** -0.5), down=n(EXPERTS, INNER, HIDDEN, std=INNER ** -0.5),
             w1=n(HIDDEN, DENSE, std=HIDDEN ** -0.5), b1=n(DENSE, std=0.1),
             w2=n(DENSE, HIDDEN, std=DENSE ** -0.5), b2=n(HIDDEN, std=0.1))
    f32 = ("x", "gain", "shift", "br", "b1", "b2")
    return {k: (v.float() if k in f32 else v.to(torch.bfloat16)) for k, v in p.items()}


def _forward(rd, p, words):
    norm = rd.layer_norm_fwd(p["x"], p["gain"], p["shift"], out_dtype=torch.bfloat16)
    logits = rd.linear(norm.out, p["wr"], p["br"], out_dtype=torch.float32)
    r = rd.route(logits, TOPK)
    packed = rd.dispatch_rows(norm.out, r.pos)
    fused = rd.ragged_dot(packed, p["up"], r.group_sizes)
    h = rd.glu_fwd(fused)
    y = rd.ragged_dot(h, p["down"], r.group_sizes)
    mixed = rd.combine_rows(y, r.pos, r.weights)
    u, pre = rd.linear(norm.out, p["w1"], p["b1"], act=rd.ACT_GELU, save_pre=True)
    both = rd.linear(u, p["w2"], p["b2"], residual=mixed)
    out = rd.dropout_rows(both, words, P, residual=p["x"])
    return out, (norm, logits, r, packed, fused, h, y, u, pre)


def _backward(rd, p, words, saved, d_out):
    norm, logits, r, packed, fused, h, y, u, pre = saved
    sizes = torch.tensor([TOKENS], dtype=torch.int32, device=DEV)     # one weight as one group

    def through(d, x, w):
        """(dx, dw) of a product with one weight."""
        return rd.ragged_dot_trans_rhs(d, w.unsqueeze(0), sizes), rd.trans_ragged_dot(x, d, sizes)[0]

    d_both = rd.dropout_rows(d_out, words, P, out_dtype=torch.bfloat16)
    _, d_b2 = rd.linear_act_bwd(d_both, None, rd.ACT_NONE, need_pre=False)
    d_u, d_w2 = through(d_both, u, p["w2"])
    d_pre, d_b1 = rd.linear_act_bwd(d_u, pre, rd.ACT_GELU)
    d_n1, d_w1 = through(d_pre, norm.out, p["w1"])
    d_y, d_weights = rd.combine_rows_bwd(d_both, y, r.pos, r.weights)
    d_fused = rd.ragged_dot_trans_rhs_glu_bwd(d_y, p["down"], fused, r.group_sizes)
    d_down = rd.trans_ragged_dot(h, d_y, r.group_sizes)
    d_up = rd.trans_ragged_dot(packed, d_fused, r.group_sizes)
    d_n2 = rd.combine_rows(rd.ragged_dot_trans_rhs(d_fused, p["up"], r.group_sizes), r.pos)
    d_logits = rd.route_bwd(logits, r.ids, d_weights)
    d_l, d_br = rd.linear_act_bwd(d_logits, None, rd.ACT_NONE)
    d_n3, d_wr = through(d_l, norm.out, p["wr"])
    d_norm = (d_n1.float() + d_n2.float() + d_n3.float())
    d_x, d_gain, d_shift = rd.layer_norm_bwd(d_norm, p["x"], p["gain"], norm.mean, norm.rstd)
    return dict(x=d_x + d_out, gain=d_gain, shift=d_shift, wr=d_wr, br=d_br, up=d_up, down=d_down, w1=d_w1, b1=d_b1,
                w2=d_w2, b2=d_b2)


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


def test_training_step(rd_lib):
    params = _params(1)
    p = {k: v.to(DEV) for k, v in params.items()}
    words = torch.tensor(WORDS, device=DEV)
    out, saved = _forward(rd_lib, p, words)
    d_out = torch.randn(TOKENS, HIDDEN, generator=torch.Generator().manual_seed(2))
    grads = _backward(rd_lib, p, words, saved, d_out.to(DEV))

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


def test_gradients_against_differences(rd_lib):
    """The gradients of the 64-bit block are those of its differences, so that the test above means what it says."""
    p = {k: v.double() for k, v in _params(3).items()}
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


def test_forward_from_a_graph(rd_lib):
    """One capture, replayed with other tokens and other words of the generator: the eager call's bits."""
    p = {k: v.to(DEV) for k, v in _params(7).items()}
    words = torch.tensor(WORDS, device=DEV)
    _forward(rd_lib, p, words)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = _forward(rd_lib, p, words)
    seen = []
    for i in range(3):
        p["x"].copy_(_params(20 + i)["x"])
        words.add_(1)
        graph.replay()
        got = captured.clone()
        assert torch.equal(got, _forward(rd_lib, p, words)[0])
        seen.append(got)
    assert not torch.equal(seen[0], seen[1])


def test_one_decoding_token(rd_lib):
    """A single token through the dense part, as a decoding step calls it."""
    p = _params(9)
    dev = {k: v.to(DEV) for k, v in p.items()}
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
