"""First calls of the layer's parts from several host threads at once, each with its own stream and workspace (what overlapping calls
need); in a process of its own, whose kernels no call has configured yet."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
import sparse_moe_ffn_router_gb300 as moe

moe.load_library()
torch.cuda.init()
g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
T, N, K = 600, 512, 256
lin, norm = moe.LinearDims(T, N, K, act=moe.ACT_GELU), moe.NormDims(T, N)
few = moe.LinearDims(40, N, K)
x, w, b, gamma = rand(T, K), rand(N, K), rand(N), rand(N)
ids = torch.randint(0, 32, (4096, 4), generator=g, device="cuda", dtype=torch.int32)


def buffers():
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    i = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    return dict(out=e(T, N), z=e(T, N), few=e(40, N), dx=e(T, K), dw=e(N, K), db=e(N), dy=e(T, N), dg=e(N), sort=[i(32), i(33), i(16384), i(16384)],
                ws=moe.new_linear_workspace(lin, True), fws=moe.new_linear_workspace(few), nws=moe.new_norm_workspace(norm), stream=torch.cuda.Stream())


def calls(v):
    s = v["stream"].cuda_stream
    moe.moe_linear(lin, x, w, b, None, None, v["out"], v["z"], v["ws"], stream=s)
    moe.moe_linear(few, x[:40], w, b, None, None, v["few"], None, v["fws"], stream=s)
    moe.moe_linear_backward(lin, x, w, None, v["z"], v["out"], v["dx"], v["dw"], v["db"], v["ws"], stream=s)
    moe.moe_norm_residual_backward(norm, None, v["out"], v["z"], v["z"], None, gamma, gamma, None, v["dy"], None, v["dg"], None, v["nws"], stream=s)
    moe.moe_sort_pairs(32, ids, *v["sort"], stream=s)


sets = [buffers() for _ in range(9)]
torch.cuda.synchronize()
start, errors = threading.Barrier(8), []


def run(v):
    try:
        start.wait()
        calls(v)
    except Exception as e:  # (shown below)
        errors.append(e)


threads = [threading.Thread(target=run, args=(v,)) for v in sets[:8]]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
calls(sets[8])
torch.cuda.synchronize()
for v in sets:
    assert moe.moe_last_device_error(v["ws"]) == 0 and moe.moe_last_device_error(v["fws"]) == 0
    for name in ("out", "z", "few", "dx", "dw", "db", "dy", "dg"):
        assert torch.equal(v[name], sets[8][name]), name
    assert all(torch.equal(p, q) for p, q in zip(v["sort"], sets[8]["sort"]))
print("threads ok")
"""


def test_first_calls_from_eight_threads():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr
