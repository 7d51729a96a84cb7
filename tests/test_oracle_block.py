"""Pins of the oracle's layer norm, activations, linear products and dropout: differences, published
answers, closed forms."""
import math

import numpy as np
import pytest

from oracle import block


def test_layer_norm_rows():
    x = np.array([[1.0, 3.0], [5.0, 5.0], [-1e6, 1e6]])
    out, mean, rstd = block.layer_norm(x, np.array([2.0, 3.0]), np.array([0.5, -0.5]), eps=0.0 + 1e-12)
    assert mean.tolist() == [2.0, 5.0, 0.0]
    np.testing.assert_allclose(out, [[-1.5, 2.5], [0.5, -0.5], [-1.5, 2.5]], atol=1e-9)
    assert abs(rstd[1] - 1e6) < 1e-3


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w, b, d = rng.normal(size=(5, 16)), rng.normal(size=16), rng.normal(size=16), rng.normal(size=(5, 16))
    out, mean, rstd = block.layer_norm(x, w, b)
    grads = block.layer_norm_bwd(d, x, w, mean, rstd)
    args = [x, w, b]
    for i, g in enumerate(grads):
        way = rng.normal(size=args[i].shape)
        h = 1e-6
        up, dn = [list(args) for _ in range(2)]
        up[i], dn[i] = args[i] + h * way, args[i] - h * way
        want = (d * (block.layer_norm(*up)[0] - block.layer_norm(*dn)[0])).sum() / (2 * h)
        assert abs((g * way).sum() - want) < 1e-6 * (1 + abs(want))


@pytest.mark.parametrize("kind", block.ACTS)
def test_activations(kind):
    z = np.linspace(-9, 9, 721) + 1e-3
    h = 1e-6
    slope = (block.act(z + h, kind) - block.act(z - h, kind)) / (2 * h)
    np.testing.assert_allclose(block.act_slope(z, kind), slope, atol=1e-8, rtol=1e-8)
    if kind == block.GELU_TANH:
        np.testing.assert_allclose(block.act(z, kind), z / 2 * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
                                   rtol=1e-9, atol=1e-13)
    if kind == block.GELU:
        np.testing.assert_allclose(block.act(1.0, kind), 0.8413447460685429, rtol=1e-14)
    assert block.act(np.zeros(1), kind)[0] == 0.0


def test_linear_groups_offset_and_limit():
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(10, 3)), rng.normal(size=(2, 3, 4)), rng.normal(size=(2, 4))
    res = rng.normal(size=(10, 4))
    out, z = block.linear(x, w, b, res, block.SILU, sizes=[2, 3, 4, 1], offset=1, limit=8)
    assert np.all(out[:2] == 0) and np.all(out[8:] == 0)
    want = x[4] @ w[0] + b[0]
    np.testing.assert_allclose(z[4], want)
    np.testing.assert_allclose(out[4], want / (1 + np.exp(-want)) + res[4])
    np.testing.assert_allclose(z[7], x[7] @ w[1] + b[1])
    d = rng.normal(size=(10, 4))
    d_pre, d_bias = block.linear_act_bwd(d, z, block.SILU, [2, 3, 4, 1], 1, 2, limit=8)
    np.testing.assert_allclose(d_bias[1], d_pre[5:8].sum(0))
    assert np.all(d_pre[8:] == 0) and np.all(d_pre[:2] == 0)


def test_generator_known_answers():
    """The answers published with the generator for 4 x 32 bits in ten rounds."""
    assert block.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    f = 0xFFFFFFFF
    assert block.philox([f] * 4, [f] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert block.philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == \
        [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_dropout_draws_are_the_words():
    seed, offset, first = -3, (7 << 32) + 5, (1 << 32) - 2
    draws = block.dropout_draws(seed, offset, first, 5)
    s = seed % 2 ** 64
    for i in range(5):
        v = first + i
        words = block.philox([v & 0xFFFFFFFF, v >> 32, offset & 0xFFFFFFFF, offset >> 32], [s & 0xFFFFFFFF, s >> 32])
        assert draws[i].tolist() == [part for w in words for part in (w & 0xFFFF, w >> 16)]


def test_dropout_rate_and_scale():
    x = np.ones((64, 1024))
    out, kept = block.dropout(x, 1, 2, 0.1)
    least = block.dropout_threshold(0.1)
    assert least == 6554
    n, q = x.size, 1 - least / 65536
    assert abs(kept.mean() - q) < 5 * math.sqrt(q * (1 - q) / n)
    assert set(np.unique(out)) == {0.0, 65536 / (65536 - least)}
    assert block.dropout(x, 1, 2, 1.0)[1].sum() == 0 and block.dropout(x, 1, 2, 0.0)[1].all()
