"""One MoE layer, from router logits to token outputs: a training step in bf16 and serving in 4 bits.

    python examples/moe_layer.py            # a small layer
    python examples/moe_layer.py --tokens 256 --experts 128 --topk 8 --hidden 4096 --inner 768

Training: route -> dispatch -> up -> SiLU-GLU -> down -> combine, and back through all of it to the
gradients of the tokens, the router logits and both weights.  Serving: the same layer with its weights
held in 4 bits, captured once in a CUDA graph and replayed.  Prints how far the two forwards are apart
(the 4-bit error) and the time of a replay.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import expert_ffn_ragged_gb300 as rd  # noqa: E402


def forward(x, logits, up, down, topk):
    """The layer in bf16; returns its output and what the backward pass needs."""
    r = rd.route(logits, topk)
    packed = rd.dispatch_rows(x, r.pos)
    fused = rd.ragged_dot(packed, up, r.group_sizes)
    h = rd.glu_fwd(fused)
    y = rd.ragged_dot(h, down, r.group_sizes)
    return rd.combine_rows(y, r.pos, r.weights), (r, packed, fused, h, y)


def backward(d_out, saved, logits, up, down):
    """Gradients of the tokens, the router logits and both weights from that of the output."""
    r, packed, fused, h, y = saved
    d_y, d_w = rd.combine_rows_bwd(d_out, y, r.pos, r.weights)
    d_fused = rd.ragged_dot_trans_rhs_glu_bwd(d_y, down, fused, r.group_sizes)
    d_down = rd.trans_ragged_dot(h, d_y, r.group_sizes)
    d_up = rd.trans_ragged_dot(packed, d_fused, r.group_sizes)
    d_packed = rd.ragged_dot_trans_rhs(d_fused, up, r.group_sizes)
    d_x = rd.combine_rows(d_packed, r.pos)          # dispatch copies: its gradient sums
    d_logits = rd.route_bwd(logits, r.ids, d_w)
    return d_x, d_logits, d_up, d_down


def forward4(x, logits, up4, down4, topk):
    """The layer with 4-bit weights and activations."""
    r = rd.route(logits, topk)
    q = rd.mxfp4_quantize(x, pos=r.pos)
    h = rd.ragged_dot_mxfp4(*q, *up4, r.group_sizes, epilogue=rd.EPI_SILU_GLU_MXFP4)
    y = rd.ragged_dot_mxfp4(*h, *down4, r.group_sizes)
    return rd.combine_rows(y, r.pos, r.weights)


def make_layer(tokens, experts, hidden, inner, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    return (normal(tokens, hidden), torch.randn(tokens, experts, generator=g, device="cuda"),
            normal(experts, hidden, 2 * inner, std=hidden ** -0.5),
            normal(experts, inner, hidden, std=inner ** -0.5))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 96), ("experts", 16), ("topk", 4), ("hidden", 512), ("inner", 256)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    x, logits, up, down = make_layer(a.tokens, a.experts, a.hidden, a.inner)
    out, saved = forward(x, logits, up, down, a.topk)
    grads = backward(torch.ones_like(out), saved, logits, up, down)
    print("training step: out", tuple(out.shape), "gradients", [tuple(t.shape) for t in grads])

    up4, down4 = rd.mxfp4_quantize_weights(up), rd.mxfp4_quantize_weights(down)
    out4 = forward4(x, logits, up4, down4, a.topk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out4 = forward4(x, logits, up4, down4, a.topk)
    for _ in range(3):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    rel = float((out4.float() - out.float()).norm() / out.float().norm())
    print(f"4-bit layer: {start.elapsed_time(end) * 50:.1f} us a replay, relative difference {rel:.3f}")
    return rel


if __name__ == "__main__":
    main()
