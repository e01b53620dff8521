"""The parts together, as a training step of a block uses them: norm, routing, dispatch, the experts' two products, combine into
the stream, norm; and the way back. Each stage against 64 bits from the stage before."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import parts_reference as ref

pytestmark = pytest.mark.gpu
B = torch.bfloat16


class Block:
    """A block's weights, buffers and workspaces; forward() and backward() only call the library."""

    def __init__(self, T, H=256, E=16, K=4, I=128, seed=0):  # noqa: E741
        self.T, self.H, self.E, self.K, self.I = T, H, E, K, I
        P = T * K
        r = lambda i, *s, scale=1.0: ref.randn(seed + i, B, *s, scale=scale)  # noqa: E731
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        new = lambda *s: torch.zeros(*s, dtype=B, device="cuda")  # noqa: E731
        self.dims = (T, H, E, K, I, 64)
        self.weights = moe.Weights(r(1, E, H, scale=H ** -0.5), None, r(2, E, 2 * I, H, scale=H ** -0.5), r(3, E, H, I, scale=I ** -0.5),
                                   r(4, 128, H, scale=H ** -0.5), torch.zeros(H, 64, dtype=B, device="cuda"), r(6, 1, H))
        self.gamma1, self.gamma2 = (1 + r(7, H, scale=0.1).float()).to(B), (1 + r(8, H, scale=0.1).float()).to(B)
        self.gate = r(9, H)
        self.x, self.y0 = r(10, T, H), r(11, T, H)
        self.n0 = moe.NormDims(T, H, post=False)
        self.n1 = moe.NormDims(T, H, gate=moe.GATE_CHANNEL, gate_act=moe.ACT_SIGMOID, branch_scale=0.5)
        self.up, self.down = moe.LinearDims(P, 2 * I, H, E=E, act=moe.ACT_SWIGLU), moe.LinearDims(P, H, I, E=E)
        self.ws = moe.new_workspace(self.dims)
        self.ws_up, self.ws_down = moe.new_linear_workspace(self.up, backward=True), moe.new_linear_workspace(self.down, backward=True)
        self.ws_n = moe.new_norm_workspace(self.n1)
        self.s0, self.xn, self.moe_out, self.s1, self.xn1 = (new(T, H) for _ in range(5))
        self.ids, self.topw, self.counts, self.offsets, self.perm, self.inv = i32(T, K), torch.zeros(T, K, device="cuda"), i32(E), i32(E + 1), i32(P), i32(P)
        self.rows, self.h, self.z, self.yrows = new(P, H), new(P, I), new(P, 2 * I), new(P, H)
        self.ds, self.dxn1 = r(12, T, H), r(13, T, H)
        self.dres, self.dmoe, self.dgate, self.dg2, self.dg1 = new(T, H), new(T, H), new(H), new(H), new(H)
        self.dyrows, self.dtopw, self.dh, self.dwd, self.drows, self.dwu, self.dxn = (new(P, H), torch.zeros(T, K, device="cuda"), new(P, I),
                                                                                     new(E, H, I), new(P, H), new(E, 2 * I, H), new(T, H))

    def forward(self):
        w = self.weights
        moe.moe_norm_residual(self.n0, self.y0, self.x, None, None, self.gamma1, self.s0, self.xn)
        moe.moe_route(self.dims, self.xn, w, self.ids, self.topw, self.counts, self.offsets, self.perm, self.ws)
        moe.moe_sort_pairs(self.E, self.ids, self.counts, self.offsets, self.perm, self.inv)
        moe.moe_dispatch(self.xn, self.inv, None, self.rows)
        moe.moe_linear(self.up, self.rows, w.gate_up, None, self.offsets, None, self.h, self.z, self.ws_up)
        moe.moe_linear(self.down, self.h, w.down, None, self.offsets, None, self.yrows, None, self.ws_down)
        moe.moe_combine(self.yrows, self.inv, self.topw, None, self.moe_out)
        moe.moe_norm_residual(self.n1, self.moe_out, self.s0, self.gate, self.gamma2, self.gamma1, self.s1, self.xn1)

    def backward(self):
        w = self.weights
        moe.moe_norm_residual_backward(self.n1, self.ds, self.dxn1, self.s1, self.moe_out, self.gate, self.gamma2, self.gamma1,
                                       self.dres, self.dmoe, self.dgate, self.dg2, self.dg1, self.ws_n)
        moe.moe_combine_backward(self.dmoe, self.inv, self.topw, self.yrows, self.dyrows, self.dtopw)
        moe.moe_linear_backward(self.down, self.h, w.down, self.offsets, None, self.dyrows, self.dh, self.dwd, None, self.ws_down)
        moe.moe_linear_backward(self.up, self.rows, w.gate_up, self.offsets, self.z, self.dh, self.drows, self.dwu, None, self.ws_up)
        moe.moe_dispatch_backward(self.drows, self.inv, None, None, self.dxn)

    def results(self):
        return [self.s0, self.xn, self.ids, self.topw, self.rows, self.h, self.z, self.yrows, self.moe_out, self.s1, self.xn1, self.dres, self.dmoe,
                self.dgate, self.dg2, self.dg1, self.dyrows, self.dtopw, self.dh, self.dwd, self.drows, self.dwu, self.dxn]


@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_block(T):
    b = Block(T)
    b.forward()
    b.backward()
    for ws in (b.ws, b.ws_up, b.ws_down):
        assert moe.moe_last_device_error(ws) == 0
    w, T, K = b.weights, b.T, b.K
    s64, xn64 = ref.norm_forward(b.n0, b.y0.double(), b.x.double(), None, None, b.gamma1.double())
    assert float((b.s0.double() - s64).abs().max() / s64.abs().max()) <= 2 ** -7 and float((b.xn.double() - xn64).abs().max() / xn64.abs().max()) <= 2 ** -7
    assert torch.equal(b.rows.double(), ref.spread(b.xn, b.inv, None, torch.zeros_like(b.rows)))
    o, z, mo, mz = ref.linear(b.up, b.rows, w.gate_up, None, b.offsets, None)
    ref.check(b.h, o, mo, b.H, "h")
    ref.check(b.z, z, mz, b.H, "z")
    o, _, mo, _ = ref.linear(b.down, b.h, w.down, None, b.offsets, None)
    ref.check(b.yrows, o, mo, b.I, "y")
    s, m = ref.gather(b.yrows, b.inv, b.topw, T)
    ref.check(b.moe_out, s, m, K, "combine")
    # the fused layer (its shared expert's down matrix is zero) on the same input
    fused = torch.empty_like(b.x)
    moe.moe_forward(b.dims, b.xn, w, None, fused, b.ws)
    assert float((fused.double() - b.moe_out.double()).abs().max()) <= 1e-2 * float(fused.double().abs().max()) + 1e-3
    # the way back
    live = (b.inv >= 0).view(T, K)
    want = ref.spread(b.dmoe, b.inv, b.topw, torch.zeros_like(b.dyrows))
    ref.check(b.dyrows, want, want.abs(), 1, "dyrows")
    d, dm = ref.dots(b.dmoe, b.yrows, b.inv, T)
    ref.check(b.dtopw, d, dm, b.H, "dtopw")
    assert bool(live.all())
    for name, got, (res, bound) in (("down", (b.dh, b.dwd), ref.linear_backward(b.down, b.h, w.down, b.offsets, None, b.dyrows)),
                                    ("up", (b.drows, b.dwu), ref.linear_backward(b.up, b.rows, w.gate_up, b.offsets, b.z, b.dh))):
        for g, r, e in zip(got, res, bound):
            assert not bool((~((g.double() - r).abs() <= e)).any()), name
    s, m = ref.gather(b.drows, b.inv, None, T)
    ref.check(b.dxn, s, m, K, "dxn")


def test_same_bits_again_in_a_graph_and_on_two_streams():
    """Eager passes twice, a captured one replayed on other inputs, and two blocks at once on two streams."""
    a, b = Block(130, seed=1), Block(77, seed=50)
    for blk in (a, b):
        blk.forward()
        blk.backward()
    torch.cuda.synchronize()
    want = [[t.clone() for t in blk.results()] for blk in (a, b)]
    for blk in (a, b):
        for t in blk.results():
            t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            b.forward()
            b.backward()
        a.forward()
        a.backward()
    torch.cuda.synchronize()
    for blk, w in zip((a, b), want):
        assert all(torch.equal(p, q) for p, q in zip(blk.results(), w))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.forward()
        a.backward()
    x, ds = a.x.clone(), a.ds.clone()
    a.x.copy_(ref.randn(99, B, *a.x.shape))
    a.ds.copy_(ref.randn(98, B, *a.ds.shape))
    g.replay()
    torch.cuda.synchronize()
    other = [t.clone() for t in a.results()]
    assert not torch.equal(other[0], want[0][0])
    a.forward()
    a.backward()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a.results(), other))
    a.x.copy_(x)
    a.ds.copy_(ds)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a.results(), want[0]))


def test_stream_argument():
    d = moe.LinearDims(40, 64, 64)
    x, w = ref.randn(1, B, 40, 64), ref.randn(2, B, 1, 64, 64)
    out, ws, s = torch.zeros(40, 64, dtype=B, device="cuda"), moe.new_linear_workspace(d), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_linear(d, x, w, None, None, None, out, None, ws, stream=s)
    s.synchronize()
    want, _, m, _ = ref.linear(d, x, w, None, None, None)
    ref.check(out, want, m, 64, "out")


def test_tensors_of_another_kind_are_refused():
    d = moe.LinearDims(8, 64, 64)
    x, w = ref.randn(1, B, 8, 64), ref.randn(2, B, 1, 64, 64)
    ws, out = moe.new_linear_workspace(d), torch.zeros(8, 64, dtype=B, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_linear(d, ref.randn(1, B, 64, 8).T, w, None, None, None, out, None, ws)  # not contiguous
    with pytest.raises(ValueError):
        moe.moe_linear(d, x, w.cpu(), None, None, None, out, None, ws)
    with pytest.raises(moe.MoEError):
        moe.moe_linear(d, x, w, None, None, None, x, None, ws)


FIRST = """
import torch, sparse_moe_ffn_router_gb300 as moe
from tests.test_gpu_parts_block import Block
moe.load_library()
b = Block(130)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    b.forward()
    b.backward()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in b.results()]
b.forward()
b.backward()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, b.results()))
print("same")
"""


def test_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
