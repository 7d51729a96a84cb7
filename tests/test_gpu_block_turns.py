"""The norm's kernels with several rows a block, one after another: rings and slots that are written again, and a limit that
ends within a later turn.  Resident blocks and rows of a turn are those of csrc/layer_norm.cu on 152 SMs; on more of them
the turns are fewer and the results the same.  Checks and tolerances are those of test_gpu_block.py."""
import os
import subprocess
import sys
import threading

import pytest

from test_gpu_block import _check_norm, _check_norm_bwd

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# hidden -> rows for three turns at least
FORWARD = {256: 15000, 512: 11000, 1024: 7500, 2048: 3700, 4096: 1900, 8192: 950, 12288: 480, 16392: 480, 32768: 480,
           33000: 950}


@pytest.mark.parametrize("hidden", list(FORWARD))
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_norm_of_many_rows(rd_lib, hidden, dt, ot):
    rows = FORWARD[hidden] + (hidden + len(dt)) % 7
    limit = None if dt == ot else rows - rows // 5      # within the last turn, or before it
    _check_norm(rd_lib, rows, hidden, dt, ot, limit=limit)


# rows that four or eight blocks share (38 and 19 clusters), and those whose columns are summed by a kernel of their own
@pytest.mark.parametrize("rows,hidden", [(190, 20000), (190, 32768), (100, 32776), (100, 65536), (400, 12288), (400, 65544)])
@pytest.mark.parametrize("dt,ot", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("short", [False, True])
def test_norm_gradients_of_many_long_rows(rd_lib, rows, hidden, dt, ot, short):
    _check_norm_bwd(rd_lib, rows, hidden, dt, ot, limit=rows * 4 // 5 + 1 if short else None)


@pytest.mark.parametrize("hidden", [256, 1024, 2048, 4096, 8192])
def test_norm_gradients_of_many_rows(rd_lib, hidden):
    """... of rows that a block holds: 456 x 8 x 8 of them, 608 x 2, 304 x 2, 304 and 152 are a turn."""
    rows = {256: 60000, 1024: 3700, 2048: 1900, 4096: 1500, 8192: 1100}[hidden]
    _check_norm_bwd(rd_lib, rows, hidden, "f32", "bf16", limit=rows - 70)


def _calls(rd, seed):
    """Calls of each kernel with a workspace, or with blocks that wait for one another: functions that give tensors."""
    g = torch.Generator().manual_seed(seed)

    def n(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    rows = 1100 + 137 * seed
    x, wide, long = n(rows, 1000), n(90 + seed, 20000, dtype=torch.bfloat16), n(70, 70000)
    fx, fw, fl = (rd.layer_norm_fwd(t) for t in (x, wide, long))
    d, pre = n(3000 + seed, 264), n(3000 + seed, 264, dtype=torch.bfloat16)
    a, w = n(64, 4096, dtype=torch.bfloat16), n(4096, 520, dtype=torch.bfloat16)
    return [lambda: rd.layer_norm_bwd(x, x, None, fx.mean, fx.rstd),
            lambda: rd.layer_norm_bwd(wide, wide, None, fw.mean, fw.rstd),
            lambda: rd.layer_norm_bwd(long, long, None, fl.mean, fl.rstd),
            lambda: rd.linear_act_bwd(d, pre, rd.ACT_GELU),
            lambda: (rd.linear(a, w, act=rd.ACT_SILU),)]


def test_threads_with_workspaces(rd_lib):
    """Several host threads, each on its own stream: the bits of the same calls made alone."""
    work = [(calls, [[t.clone() for t in c()] for c in calls]) for calls in (_calls(rd_lib, s) for s in range(4))]
    torch.cuda.synchronize()
    wrong = []

    def run(t):
        calls, ref = work[t]
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                got = [calls[i % len(calls)]() for i in range(8 * len(calls))]
            stream.synchronize()
            wrong.extend((t, i) for i, out in enumerate(got)
                         if not all(torch.equal(a, b) for a, b in zip(out, ref[i % len(calls)])))
        except Exception as e:  # reported below, on the main thread
            wrong.append((t, e))

    threads = [threading.Thread(target=run, args=(t,)) for t in range(len(work))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not wrong, wrong


FIRST_CALLS = """
import torch
import expert_ffn_ragged_gb300 as rd

def n(*shape, dtype=torch.float32):
    return torch.randn(*shape, device="cuda").to(dtype)

# the entry points themselves have been called; the kernels below have not
one = torch.ones(8, 64, device="cuda")
f = rd.layer_norm_fwd(one)
rd.layer_norm_bwd(one, one, None, f.mean, f.rstd)
rd.linear_act_bwd(one, None)
rd.linear(one.bfloat16(), torch.ones(64, 64, device="cuda").bfloat16())
torch.cuda.synchronize()
rows = [n(1300, 1000), n(1300, 4096, dtype=torch.bfloat16), n(60, 20000), n(40, 40000, dtype=torch.bfloat16), n(60, 70000)]
d, pre = n(3000, 264), n(3000, 264, dtype=torch.bfloat16)
a, w = n(3000, 520, dtype=torch.bfloat16), n(520, 2056, dtype=torch.bfloat16)

def calls():
    out = []
    for v in rows:
        f = rd.layer_norm_fwd(v)
        out += [f.out, *rd.layer_norm_bwd(v, v, None, f.mean, f.rstd)]
    out += rd.linear_act_bwd(d, pre, rd.ACT_GELU)
    out += [rd.linear(a[:40], w), rd.linear(a[:300], w[:, :136].contiguous(), out_dtype=torch.float32),
            rd.linear(a, w), rd.linear(a, w, out_dtype=torch.float32)]
    return out

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, calls()))
print("captured", len(got))
"""


def test_first_calls_of_kernels_inside_a_capture(rd_lib):
    """Their attributes are set, and the clusters that fit counted, while the stream is captured: in a process of its own, so
    that no other test has called them."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("captured"), r.stdout + r.stderr
