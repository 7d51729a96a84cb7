"""One feed-forward block around the experts: norm, router, experts beside a dense feed-forward, dropout.

    python examples/feed_forward_block.py            # a small block
    python examples/feed_forward_block.py --tokens 64 --experts 16 --topk 4 --hidden 4096 --inner 768 --dense 4096

Training: the residual stream x is f32; layer norm -> router logits (f32) -> the routed experts, and the dense
branch norm -> product + bias + gelu -> product + bias + the experts' output as its residual; dropout adds the sum to x.
Back through all of it to the gradients of x and of every parameter.  Serving: the forward without
dropout, captured once in a CUDA graph and replayed.  Prints the gradients' shapes and the time of a replay.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import expert_ffn_ragged_gb300 as rd  # noqa: E402


def forward(p, topk, words=None, drop=0.0):
    """The block's output (f32) and what the backward pass needs; ``words``: the generator's (int64 [2])."""
    norm = rd.layer_norm_fwd(p["x"], p["gain"], p["shift"], out_dtype=torch.bfloat16)
    logits = rd.linear(norm.out, p["wr"], p["br"], out_dtype=torch.float32)
    r = rd.route(logits, topk)
    packed = rd.dispatch_rows(norm.out, r.pos)
    fused = rd.ragged_dot(packed, p["up"], r.group_sizes)
    h = rd.glu_fwd(fused)
    y = rd.ragged_dot(h, p["down"], r.group_sizes)
    mixed = rd.combine_rows(y, r.pos, r.weights)
    u, pre = rd.linear(norm.out, p["w1"], p["b1"], act=rd.ACT_GELU, save_pre=True)
    branch = rd.linear(u, p["w2"], p["b2"], residual=mixed)
    if words is None:
        out = branch.float() + p["x"]
    else:
        out = rd.dropout_rows(branch, words, drop, residual=p["x"])
    return out, (norm, logits, r, packed, fused, h, y, u, pre)


def backward(d_out, saved, p, words, drop):
    """Gradients of x and of every parameter, by name, from that of the output (f32)."""
    norm, logits, r, packed, fused, h, y, u, pre = saved
    sizes = torch.full((1,), d_out.shape[0], dtype=torch.int32, device=d_out.device)  # one weight as one group

    def through(d, x, w):
        """(dx, dw) of a product with one weight."""
        return rd.ragged_dot_trans_rhs(d, w.unsqueeze(0), sizes), rd.trans_ragged_dot(x, d, sizes)[0]

    d_branch = rd.dropout_rows(d_out, words, drop, out_dtype=torch.bfloat16)     # the same draws
    _, d_b2 = rd.linear_act_bwd(d_branch, None, rd.ACT_NONE, need_pre=False)
    d_u, d_w2 = through(d_branch, u, p["w2"])
    d_pre, d_b1 = rd.linear_act_bwd(d_u, pre, rd.ACT_GELU)
    d_dense, d_w1 = through(d_pre, norm.out, p["w1"])
    d_y, d_weights = rd.combine_rows_bwd(d_branch, y, r.pos, r.weights)
    d_fused = rd.ragged_dot_trans_rhs_glu_bwd(d_y, p["down"], fused, r.group_sizes)
    d_down = rd.trans_ragged_dot(h, d_y, r.group_sizes)
    d_up = rd.trans_ragged_dot(packed, d_fused, r.group_sizes)
    d_routed = rd.combine_rows(rd.ragged_dot_trans_rhs(d_fused, p["up"], r.group_sizes), r.pos)
    d_logits, d_br = rd.linear_act_bwd(rd.route_bwd(logits, r.ids, d_weights), None, rd.ACT_NONE)
    d_router, d_wr = through(d_logits, norm.out, p["wr"])
    d_norm = d_dense.float() + d_routed.float() + d_router.float()
    d_x, d_gain, d_shift = rd.layer_norm_bwd(d_norm, p["x"], p["gain"], norm.mean, norm.rstd)
    return dict(x=d_x + d_out, gain=d_gain, shift=d_shift, wr=d_wr, br=d_br, up=d_up, down=d_down, w1=d_w1, b1=d_b1,
                w2=d_w2, b2=d_b2)


def make_block(tokens, experts, hidden, inner, dense, seed=0, device="cuda"):
    """Tokens (f32) and parameters by name: f32 vectors, bf16 matrices of variance 1 / fan-in."""
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0, shift=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g) * std + shift).to(dtype).to(device)

    def w(*shape):
        return n(*shape, std=shape[-2] ** -0.5, dtype=torch.bfloat16)

    return dict(x=n(tokens, hidden, shift=0.2), gain=n(hidden, std=0.1, shift=1.0), shift=n(hidden, std=0.1),
                wr=w(hidden, experts), br=n(experts, std=0.1), up=w(experts, hidden, 2 * inner),
                down=w(experts, inner, hidden), w1=w(hidden, dense), b1=n(dense, std=0.1), w2=w(dense, hidden),
                b2=n(hidden, std=0.1))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 96), ("experts", 16), ("topk", 4), ("hidden", 512), ("inner", 256), ("dense", 1024)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    p = make_block(a.tokens, a.experts, a.hidden, a.inner, a.dense)
    words = torch.tensor([1, 0], device="cuda")       # a seed; the offset counts the steps
    out, saved = forward(p, a.topk, words, 0.1)
    grads = backward(torch.ones_like(out), saved, p, words, 0.1)
    print("training step: out", tuple(out.shape), {k: tuple(t.shape) for k, t in grads.items()})

    forward(p, a.topk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served, _ = forward(p, a.topk)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"serving: {start.elapsed_time(end) * 50:.1f} us a replay")
    return served


if __name__ == "__main__":
    main()
