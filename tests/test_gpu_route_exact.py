"""The router's choice held to its definition exactly: the keys are f32, so the ids, their order and every
tie follow from the bits of elementwise f32 arithmetic, which torch computes here on the same device.
And its gradient at the ends of the range.

Tolerance of the sigmoid gradient at very negative logits: the relative error of a score is a few units of
2^-23 (two ulps of exp, one each of the sum and the reciprocal; the scores stay above 2^18 units of the
smallest subnormal, so their spacing adds less), of a share twice that and one division, of the sums of
at most 32 slots 5 units: 2^-23 * 64 of scale * share * (|d| + sum |q d|) holds them all; bf16 output
adds half an ulp, 2^-8 relative.
"""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "expert_ffn_ragged_gb300", "csrc")
LOW = float("-inf")


def _choose_f32(logits, bias, topk, score, groups, topk_groups):
    """Expert ids from keys in elementwise f32, best first, ties to the lower index, -1 where none is left."""
    l = logits.float()
    t, e = l.shape
    masked = torch.isnan(l) | (l == LOW)
    key = l if score == moe.SOFTMAX else 1.0 / (1.0 + torch.exp(-l))
    if bias is not None:
        key = key + bias
    key = torch.where(masked, torch.full_like(key, LOW), key).cpu()
    if groups > 1:
        best = torch.topk(key.view(t, groups, e // groups), min(2, e // groups), dim=2).values
        first = best[:, :, 0]
        if score == moe.SIGMOID and best.shape[2] == 2:
            first = torch.where(best[:, :, 1] == LOW, first, first + best[:, :, 1])
        order = torch.sort(first, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        kept = torch.zeros(t, groups, dtype=torch.bool).scatter(1, order, True)
        key = torch.where(kept.repeat_interleave(e // groups, 1), key, torch.full_like(key, LOW))
    # on the host -0.0 and 0.0 compare equal and a stable sort keeps their order
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(key[:, :topk] == LOW, -1, ids[:, :topk]).to(torch.int32)


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


@pytest.mark.parametrize("kind", ["grid", "free"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("experts,topk,groups,topk_groups", [
    (256, 8, 8, 4), (256, 8, 8, 8), (64, 6, 8, 3), (128, 4, 4, 2), (512, 2, 2, 1), (1024, 16, 4, 1), (1024, 32, 32, 7),
    (32, 4, 32, 5), (24, 3, 3, 2), (8, 2, 4, 1), (96, 8, 8, 2), (160, 8, 32, 5), (1000, 32, 10, 3), (256, 8, 1, 1),
    (31, 7, 1, 1)])
def test_choice_equals_elementwise_f32(rd_lib, experts, topk, groups, topk_groups, score, dtype, kind):
    """Ids and their order, bit for bit: groups of a power of two of whole lanes, of other sizes, and none; on a
    coarse grid, where most keys and group scores tie, and on free values; with masked experts and tokens."""
    rng = np.random.default_rng(experts + 7 * groups + score)
    tokens = 300
    l = rng.normal(size=(tokens, experts)) * 1.5
    bias = rng.normal(size=experts) * 0.05
    if kind == "grid":
        l, bias = np.round(2 * l) / 2, np.round(bias * 20) / 8
    l[rng.random(l.shape) < 0.03] = -np.inf
    l[rng.random(l.shape) < 0.01] = np.nan
    l[rng.random(l.shape) < 0.002] = np.inf
    l[rng.random(tokens) < 0.03] = -np.inf
    few = rng.random(tokens) < 0.1                      # tokens with hardly an expert
    l[few] = np.where(rng.random((few.sum(), experts)) < 0.03, l[few], -np.inf)
    l[:4] -= 60.0
    l[4:8] -= 95.0                                      # sigmoids of zero and of subnormal numbers
    l = torch.from_numpy(l.astype(np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16).to(DEV)
    for b in (None, torch.from_numpy(bias.astype(np.float32)).to(DEV)):
        r = rd_lib.route(l, topk, score=score, bias=b, groups=groups, topk_groups=topk_groups)
        want = _choose_f32(l, b, topk, score, groups, topk_groups)
        assert torch.equal(r.ids.cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_tiny_scores(rd_lib, renorm, dtype):
    """All logits far below zero: the scores and their sum are near the smallest normal number, the gradient
    of the renormalised weights is of the order of d all the same."""
    rng = np.random.default_rng(5)
    tokens, experts, topk, scale = 200, 24, 4, 1.5
    l = torch.from_numpy(rng.uniform(-88.0, -80.0, size=(tokens, experts)).astype(np.float32))
    l = l.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    ids = np.array([rng.permutation(experts)[:topk] for _ in range(tokens)])
    d = (rng.normal(size=(tokens, topk)) * 10.0 ** rng.uniform(0, 5, size=(tokens, 1))).astype(np.float32)
    out = rd_lib.route_bwd(l.to(DEV), torch.tensor(ids, dtype=torch.int32, device=DEV), torch.from_numpy(d).to(DEV),
                           score=rd_lib.SCORE_SIGMOID, renormalize=renorm, scale=scale)
    got, l64 = out.double().cpu().numpy(), l.double().numpy()
    for t in range(tokens):
        ref = moe.route_loss_grad(l64[t], ids[t], d[t], moe.SIGMOID, renorm, scale)
        s = moe.sigmoid(l64[t][ids[t]])
        q = s / s.sum()
        spread = np.abs(d[t]).max() + np.abs(q * d[t]).sum()
        tol = np.zeros(experts)
        tol[ids[t]] = 2.0 ** -23 * 64 * scale * (q if renorm else s) * spread
        if dtype == "bf16":
            tol += 2.0 ** -8 * np.abs(ref)
        # a subnormal result is within half a unit of the format's smallest number
        tol += 2.0 ** -149 if dtype == "f32" else 2.0 ** -133
        assert np.all(np.abs(got[t] - ref) <= tol), t


def test_largest_token_count(rd_lib):
    """2^31 - 1 tokens of one expert, the most that a call takes: every token is visited once, the last ones
    too, and nothing outside the outputs is written."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    tokens, pad = 2 ** 31 - 1, 64
    masked = [0, 1, 9727, 2 ** 30, tokens - 14593, tokens - 9729, tokens - 8, tokens - 1]
    logits = torch.zeros((tokens, 1), dtype=torch.bfloat16, device=DEV)
    logits[masked] = float("-inf")

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 77, dtype=dtype, device=DEV)
        return buf, buf[pad:pad + n].view(shape)

    def intact(buf):
        return bool((buf[:pad] == 77).all()) and bool((buf[-pad:] == 77).all())

    bufs = [guarded(s, d) for s, d in (((tokens, 1), torch.int32), ((tokens, 1), torch.float32), ((1,), torch.int32),
                                       ((tokens, 1), torch.int32), ((1,), torch.int32))]
    r = rd_lib.route(logits, 1, out=rd_lib.Routing(*[v for _, v in bufs]))
    live = tokens - len(masked)
    assert int(r.rows) == live and r.group_sizes.tolist() == [live]
    assert all(intact(b) for b, _ in bufs)
    assert r.ids[masked].flatten().tolist() == [-1] * len(masked) and int((r.ids == 0).sum()) == live
    assert not r.weights[masked].any() and int((r.weights == 1).sum()) == live
    assert r.pos[masked].flatten().tolist() == [-1] * len(masked)
    assert r.pos[[2, 9728, tokens - 2]].flatten().tolist() == [0, 9725, live - 1]
    ids = r.ids
    del bufs, r
    d = torch.full((tokens, 1), 2.0, device=DEV)
    buf, out = guarded((tokens, 1), torch.bfloat16)
    rd_lib.route_bwd(logits, ids, d, score=rd_lib.SCORE_SIGMOID, renormalize=False, out=out)
    assert intact(buf)
    assert not out[masked].any() and int((out == 0.5).sum()) == live
    del logits, ids, d, buf, out
    torch.cuda.empty_cache()


def test_reciprocal_of_every_float(rd_lib, tmp_path):
    """The keys' reciprocal (approximation and one Newton step) is the correctly rounded one for every float of
    the range it is used in, 1.03e9 of them."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    lib = str(tmp_path / "libsweep.so")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-shared",
                    "-Xcompiler", "-fPIC", "-I" + CSRC, os.path.join(HERE, "reciprocal_sweep.cu"), "-o", lib], check=True)
    torch.cuda.synchronize()
    count, wrong, lowest = ctypes.c_uint(), ctypes.c_ulonglong(), ctypes.c_uint()
    code = ctypes.CDLL(lib).reciprocal_sweep(ctypes.byref(count), ctypes.byref(wrong), ctypes.byref(lowest))
    assert code == 0
    assert count.value > 1_000_000_000
    assert wrong.value == 0, hex(lowest.value)
