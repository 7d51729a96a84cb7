"""The router's choice held to its definition exactly, and its gradient at the ends of the range."""
import numpy as np
import pytest

from oracle import moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,topk,groups,topk_groups", [
    (2, 2, 1, 1), (8, 3, 1, 1), (8, 8, 1, 1), (31, 31, 1, 1), (32, 32, 1, 1), (64, 5, 1, 1), (64, 32, 1, 1),
    (256, 8, 1, 1), (1024, 32, 1, 1), (64, 6, 8, 3), (96, 8, 8, 4), (256, 8, 8, 4)])
def test_zeros_of_either_sign_tie(rd_lib, experts, topk, groups, topk_groups, dtype):
    """Rows of 0.0 and -0.0, alone and among other values: at most and more than 32 tied candidates."""
    rng = np.random.default_rng(experts + topk)
    tokens = 48
    l = np.where(rng.random((tokens, experts)) < 0.5, -0.0, 0.0)
    l[0], l[1] = 0.0, -0.0
    l[2, :2] = -0.0, 0.0
    mixed = rng.random((tokens // 2, experts))
    l[tokens // 2:] = np.where(mixed < 0.1, 1.0, np.where(mixed < 0.3, -1.0, l[tokens // 2:]))
    l = torch.from_numpy(l.astype(np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    zeros = torch.from_numpy(np.where(rng.random(experts) < 0.5, -0.0, 0.0).astype(np.float32))
    for bias in (None, zeros):
        r = rd_lib.route(l.to(DEV), topk, groups=groups, topk_groups=topk_groups,
                         bias=None if bias is None else bias.to(DEV))
        want = [moe.route_choose(row, None if bias is None else bias.double().numpy(), topk, moe.SOFTMAX, groups,
                                 topk_groups) for row in l.double().numpy()]
        assert r.ids.tolist() == want
        for t in range(tokens):
            ref = moe.route_weights(l[t].double().numpy(), want[t], moe.SOFTMAX, True)
            assert np.all(np.abs(r.weights[t].double().cpu().numpy() - ref) <= 2.0 ** -23 * 64 * ref)
