"""The layer of examples/moe_layer.py: its gradients against differences of a float64 layer, its 4-bit
form against the float64 layer on 4-bit values."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOKENS, EXPERTS, TOPK, HIDDEN, INNER = 24, 8, 2, 64, 32


@pytest.fixture(scope="module")
def example(rd_lib):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _layer64(x, logits, up, down, ids, quant=lambda v: v):
    """The layer in float64 with the choice of experts held fixed."""
    out = np.zeros_like(x)
    for t in range(len(x)):
        w = moe.route_weights(logits[t], ids[t], moe.SOFTMAX, True)
        for k, e in enumerate(ids[t]):
            fused = quant(x[t:t + 1]) @ up[e]
            g, u = fused[:, :INNER], fused[:, INNER:]
            out[t] += w[k] * (quant(g * moe.sigmoid(g) * u) @ down[e])[0]
    return out


def _mx(v):
    return moe.mx_values(*moe.mx_quantize(v))


def test_gradients_against_differences(example):
    x, logits, up, down = example.make_layer(TOKENS, EXPERTS, HIDDEN, INNER, seed=1)
    out, saved = example.forward(x, logits, up, down, TOPK)
    d_out = torch.randn(TOKENS, HIDDEN, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    grads = [g.double().cpu().numpy() for g in example.backward(d_out, saved, logits, up, down)]
    ids = saved[0].ids.cpu().numpy()
    args = [t.double().cpu().numpy() for t in (x, logits, up, down)]
    d64 = d_out.double().cpu().numpy()
    ref = _layer64(*args, ids)
    # bf16 chain: four roundings of 2^-9 each on terms of unit size, sqrt-summed over 2 experts
    assert np.abs(out.double().cpu().numpy() - ref).max() <= 2.0 ** -5 * max(1.0, np.abs(ref).max())
    rng = np.random.default_rng(0)
    for i, g in enumerate(grads):
        direction = rng.normal(size=g.shape)
        h = 1e-4
        up_, dn_ = [a.copy() for a in args], [a.copy() for a in args]
        up_[i] = up_[i] + h * direction
        dn_[i] = dn_[i] - h * direction
        want = float((d64 * (_layer64(*up_, ids) - _layer64(*dn_, ids))).sum() / (2 * h))
        got = float((g * direction).sum())
        # each gradient element carries a few bf16 roundings (2^-8 relative), independent over elements
        noise = 2.0 ** -6 * float(np.sqrt((g ** 2 * direction ** 2).sum()))
        assert abs(got - want) <= noise + 2.0 ** -7 * abs(want), (i, got, want, noise)


def test_four_bit_layer(example, rd_lib):
    x, logits, up, down = example.make_layer(TOKENS, EXPERTS, HIDDEN, INNER, seed=3)
    up4, down4 = rd_lib.mxfp4_quantize_weights(up), rd_lib.mxfp4_quantize_weights(down)
    out = example.forward4(x, logits, up4, down4, TOPK).double().cpu().numpy()
    ids = rd_lib.route(logits, TOPK).ids.cpu().numpy()
    a = [t.double().cpu().numpy() for t in (x, logits, up, down)]
    q_up = _mx(a[2].transpose(0, 2, 1)).transpose(0, 2, 1)
    q_down = _mx(a[3].transpose(0, 2, 1)).transpose(0, 2, 1)
    ref = _layer64(a[0], a[1], q_up, q_down, ids, quant=_mx)
    # a GLU value within f32 error of a rounding boundary may take the neighbouring 4-bit value: at
    # most a step of a third of it, times a weight of 1 / sqrt(32); plus the bf16 roundings
    err = np.abs(out - ref)
    assert err.max() <= 0.25 * np.abs(ref).max()
    assert np.sqrt((err ** 2).mean()) <= 2.0 ** -7 * np.sqrt((ref ** 2).mean())


def test_example_runs(example):
    assert example.main([]) < 0.5
