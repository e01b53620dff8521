"""Norms before and after a block with its gate and residual scale, and their gradients, against plain forms."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import parts_reference as ref

pytestmark = pytest.mark.gpu
DT = {moe.BF16: torch.bfloat16, moe.FP16: torch.float16, moe.FP32: torch.float32}
SIZES = [(1, 2048), (1, 1), (3, 2), (5, 33), (2, 4104), (9, 8192), (2, 8191), (700, 256), (40, 1544), (307, 7)]
GATES = [(moe.GATE_NONE, moe.ACT_NONE), (moe.GATE_TOKEN, moe.ACT_SIGMOID), (moe.GATE_CHANNEL, moe.ACT_NONE), (moe.GATE_CHANNEL, moe.ACT_SILU),
         (moe.GATE_FULL, moe.ACT_SIGMOID), (moe.GATE_FULL, moe.ACT_SILU), (moe.GATE_TOKEN, moe.ACT_NONE)]


def inputs(d, seed=0):
    dt = DT[d.dtype]
    shape = {moe.GATE_TOKEN: (d.T,), moe.GATE_CHANNEL: (d.H,), moe.GATE_FULL: (d.T, d.H)}.get(d.gate)
    gate = None if shape is None else ref.randn(seed + 3, dt, *shape)
    gp = (1 + ref.randn(seed + 4, torch.float32, d.H, scale=0.2)).to(dt) if d.flags & moe.NORM_POST else None
    gq = (1 + ref.randn(seed + 5, torch.float32, d.H, scale=0.2)).to(dt)
    return ref.randn(seed + 1, dt, d.T, d.H, scale=2.0), ref.randn(seed + 2, dt, d.T, d.H), gate, gp, gq


def wide(*ts):
    return [None if t is None else t.double() for t in ts]


def dims(T, H, dtype, gate, post=True, **k):
    return moe.NormDims(T, H, dtype=dtype, post=post, gate=gate[0], gate_act=gate[1], **k)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("gate", GATES)
def test_forward_and_backward(dtype, T, H, gate):
    """The magnitudes: s is a sum of two products of a few factors, each rounded in fp32 (its norm's mean of H squares is off by H
    roundings of itself, so by H / 2 after the root); xn scales s by the same kind of factor."""
    post = (T + H + gate[0]) % 3 != 0
    d = dims(T, H, dtype, gate, post, branch_scale=0.5, residual_scale=0.75)
    y, r, g, gp, gq = inputs(d, T)
    s, xn = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, g, gp, gq, s, xn)
    s64, xn64 = ref.norm_forward(d, *wide(y, r, g, gp, gq))
    branch = (s64 - d.residual_scale * r.double()).abs()
    mag = branch + (d.residual_scale * r.double()).abs()
    ref.check(s, s64, mag, H, "s")
    rs = 1 / (s64.square().mean(1, keepdim=True) + d.eps).sqrt()
    # an error of s moves xn directly and through the mean square of its row (at most by the row's own relative error, summed)
    direct = mag * rs * gq.double().abs()
    through = xn64.abs() * rs * rs * (mag * s64.abs()).mean(1, keepdim=True)
    ref.check(xn, xn64, direct + through + xn64.abs(), H, "xn")
    # gradients of both results, at the s that the forward pass kept
    ds, dxn = ref.randn(T + 7, DT[dtype], T, H), ref.randn(T + 8, DT[dtype], T, H)
    new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    dres, dy, dg, dgp, dgq = new(y), new(y), new(g), new(gp), new(gq)
    ws = moe.new_norm_workspace(d)
    ws.fill_(255)
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, dres, dy, dg, dgp, dgq, ws)
    leaves = [t.double().requires_grad_() for t in (y, g, gp) if t is not None]
    names = [k for k, t in (("y", y), ("g", g), ("gp", gp)) if t is not None]
    leaf = dict(zip(names, leaves))
    n = ref.norm(leaf["y"], leaf.get("gp"), d.eps) if post else leaf["y"]
    branch = d.branch_scale * ref.gate_of(d, leaf.get("g")) * n
    s64, q64 = s.double().requires_grad_(), gq.double().requires_grad_()
    through, dgq64 = torch.autograd.grad(ref.norm(s64, q64, d.eps), (s64, q64), dxn.double())
    gs = ds.double() + through
    got = dict(zip(names, torch.autograd.grad(branch, leaves, gs)))
    # magnitudes: the norm's backward pass is the difference of two terms
    with torch.no_grad():
        rs = 1 / (s64.square().mean(1, keepdim=True) + d.eps).sqrt()
        a = (dxn.double() * gq.double()).abs()
        mgs = ds.double().abs() + rs * a + s64.abs() * rs ** 3 * (a * s64.abs()).mean(1, keepdim=True)
        ref.check(dres, d.residual_scale * gs, d.residual_scale * mgs, H, "dresidual")
        ref.check(dgq, dgq64, (dxn.double() * s64 * rs).abs().sum(0), H + T, "dgamma_pre")
        ry = 1 / (y.double().square().mean(1, keepdim=True) + d.eps).sqrt() if post else 1.0
        av = ref.gate_of(d, None if g is None else g.double())
        av = av.abs() if g is not None else 1.0
        one = gp.double().abs() if post else 1.0
        mdn = d.branch_scale * av * mgs
        mdy = mdn
        if post:
            b = mdn * one
            mdy = ry * b + y.double().abs() * ry ** 3 * (b * y.double().abs()).mean(1, keepdim=True)
            ref.check(dgp, got["gp"], (mdn * y.double().abs() * ry).sum(0), H + T, "dgamma_post")
        ref.check(dy, got["y"], mdy, H, "dy")
        if g is not None:
            m = d.branch_scale * mgs * (y.double().abs() * ry * one) * (1 + g.double().abs()[:, None] if d.gate == moe.GATE_TOKEN else 1 + g.double().abs())
            m = m if d.gate == moe.GATE_FULL else m.sum(1 if d.gate == moe.GATE_TOKEN else 0)
            ref.check(dg, got["g"], m, 2 * H + T, "dgate")


@pytest.mark.parametrize("T,H,dtype,gate", [(5003, 1003, moe.BF16, 3), (2500, 65, moe.FP16, 4), (3100, 2048, moe.BF16, 5), (4001, 96, moe.FP32, 3), (700, 8190, moe.FP32, 4),
                                            (640, 8187, moe.BF16, 1), (5200, 256, moe.FP16, 0), (1300, 6152, moe.BF16, 2)])
def test_many_rows(T, H, dtype, gate):
    """More rows than the CTAs hold at once, several rows on their way, rows that begin anywhere."""
    test_forward_and_backward(dtype, T, H, GATES[gate])


@pytest.mark.parametrize("dtype", list(DT))
def test_optional_parts(dtype):
    """What is left out is as if it were zeros (results: not written), and the rest keeps its bits."""
    d = dims(50, 264, dtype, (moe.GATE_FULL, moe.ACT_SIGMOID))
    y, r, g, gp, gq = inputs(d)
    s, xn = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, g, gp, gq, s, xn)
    a, b = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, g, gp, None, a, None)
    moe.moe_norm_residual(d, y, r, g, gp, gq, None, b)
    assert torch.equal(a, s) and torch.equal(b, xn)
    moe.moe_norm_residual(d, y, None, g, gp, torch.ones_like(gq), a, b)
    c, e = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, torch.zeros_like(r), g, gp, None, c, e)
    assert torch.equal(a, c) and torch.equal(b, e)
    ds, dxn, ws = ref.randn(7, y.dtype, 50, 264), ref.randn(8, y.dtype, 50, 264), moe.new_norm_workspace(d)
    full = [torch.empty_like(t) for t in (y, y, g, gp, gq)]
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, *full, ws)
    for i in range(5):
        some = [torch.empty_like(t) if j == i else None for j, t in enumerate(full)]
        moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, *some, ws)
        assert torch.equal(some[i], full[i]), i
    some = [torch.empty_like(t) for t in full]
    zero = torch.zeros_like(ds)
    moe.moe_norm_residual_backward(d, zero, dxn, s, y, g, gp, gq, *full, ws)
    moe.moe_norm_residual_backward(d, None, dxn, s, y, g, gp, gq, *some, ws)
    assert all(torch.equal(p, q) for p, q in zip(full, some))
    moe.moe_norm_residual_backward(d, ds, zero, s, y, g, gp, gq, *full, ws)
    moe.moe_norm_residual_backward(d, ds, None, None, y, g, gp, None, *some[:4], None, ws)
    assert all(torch.equal(p, q) for p, q in zip(full[:4], some[:4]))


def test_results_over_their_inputs():
    d = dims(300, 2048, moe.BF16, (moe.GATE_CHANNEL, moe.ACT_NONE))
    y, r, g, gp, gq = inputs(d)
    s, xn = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, g, gp, gq, s, xn)
    a, b = r.clone(), y.clone()
    moe.moe_norm_residual(d, b, a, g, gp, gq, a, b)
    assert torch.equal(a, s) and torch.equal(b, xn)
    ds, dxn, ws = ref.randn(7, y.dtype, 300, 2048), ref.randn(8, y.dtype, 300, 2048), moe.new_norm_workspace(d)
    dres, dy = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, dres, dy, None, None, None, ws)
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, ds, dxn, None, None, None, ws)
    assert torch.equal(ds, dres) and torch.equal(dxn, dy)


@pytest.mark.parametrize("H", [64, 65, 1003])
@pytest.mark.parametrize("dtype", list(DT))
def test_rows_do_not_reach_one_another(dtype, H):
    """A row of NaN beside rows that share its 16-byte pieces of memory."""
    d = dims(40, H, dtype, (moe.GATE_FULL, moe.ACT_SIGMOID))
    y, r, g, gp, gq = inputs(d)
    ds, dxn = ref.randn(6, y.dtype, 40, H), ref.randn(7, y.dtype, 40, H)

    def run():
        out = [torch.empty_like(y) for _ in range(5)]
        moe.moe_norm_residual(d, y, r, g, gp, gq, out[0], out[1])
        moe.moe_norm_residual_backward(d, ds, dxn, r, y, g, gp, gq, *out[2:], None, None, moe.new_norm_workspace(d))
        return out

    clean = run()
    for t in (y, r, g, ds, dxn):
        t[17] = float("nan")
    for a, b in zip(run(), clean):
        assert bool(a[17].isnan().all())
        assert torch.equal(torch.cat((a[:17], a[18:])), torch.cat((b[:17], b[18:])))


def test_agrees_with_rmsnorm():
    """The last norm alone: s = y, xn as moe_rmsnorm gives it, up to the order of fp32 sums (two roundings to bf16 a step apart at most)."""
    x, gamma = ref.randn(1, torch.bfloat16, 37, 2048), ref.randn(2, torch.bfloat16, 2048)
    d = moe.NormDims(37, 2048, post=False)
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_norm_residual(d, x, None, None, None, gamma, None, a)
    moe.moe_rmsnorm((37, 2048, 8, 1, 64, 64), x, gamma, 1e-6, b)
    assert float(((a.double() - b.double()).abs() / b.double().abs().clamp(min=1e-30)).max()) <= 2 ** -7


@pytest.mark.parametrize("eps,scale", [(0.0, 1.0), (1e-6, 0.0), (1e-6, 1e-12), (1.0, 1e4)])
def test_eps_zero_rows_and_far_values(eps, scale):
    d = moe.NormDims(4, 512, dtype=moe.FP32, eps=eps)
    y, r = ref.randn(1, torch.float32, 4, 512, scale=scale), ref.randn(2, torch.float32, 4, 512, scale=scale)
    s, xn = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, None, None, None, s, xn)
    s64, xn64 = ref.norm_forward(d, y.double(), r.double(), None, None, None)
    mag = s64.abs() + 2 * r.double().abs()
    ref.check(s, s64, mag, 512, "s")
    rs = 1 / (s64.square().mean(1, keepdim=True) + d.eps).sqrt()
    ref.check(xn, xn64, mag * rs + xn64.abs() * (1 + rs * rs * (mag * s64.abs()).mean(1, keepdim=True)), 512, "xn")


@pytest.mark.parametrize("eps,scale", [(1e-30, 0.0), (0.0, 1e-15), (0.0, 1e15), (1e-6, 1e-12)])
def test_gradients_of_zero_rows_and_far_values(eps, scale):
    """Where the cube of a norm's factor leaves fp32's range and the gradients do not."""
    d = moe.NormDims(4, 512, dtype=moe.FP32, eps=eps)
    y, s = ref.randn(1, torch.float32, 4, 512, scale=scale), ref.randn(2, torch.float32, 4, 512, scale=scale)
    dxn = ref.randn(3, torch.float32, 4, 512)
    dres, dy = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual_backward(d, None, dxn, s, y, None, None, None, dres, None, None, None, None, moe.new_norm_workspace(d))
    moe.moe_norm_residual_backward(d, dxn, None, s, y, None, None, None, None, dy, None, None, None, moe.new_norm_workspace(d))
    for got, v, what in ((dres, s, "dresidual"), (dy, y, "dy")):
        v64 = v.double().requires_grad_()
        want, = torch.autograd.grad(ref.norm(v64, None, d.eps), v64, dxn.double())
        with torch.no_grad():
            r = 1 / (v64.square().mean(1, keepdim=True) + d.eps).sqrt()
            a = dxn.double().abs()
            ref.check(got, want, r * a + v64.abs() * r ** 3 * (a * v64.abs()).mean(1, keepdim=True), 512, what)


def test_no_rows():
    d = dims(0, 64, moe.BF16, (moe.GATE_CHANNEL, moe.ACT_NONE))
    z, h = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.full((64,), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_norm_residual(d, z, z, h, h, h, z, z)
    grads = [h.clone() for _ in range(3)]
    moe.moe_norm_residual_backward(d, z, z, z, z, h, h, h, z, z, *grads, moe.new_norm_workspace(d))
    assert all(bool((t == 0).all()) for t in grads)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 150, 153, 290, 297, 305, 700])
@pytest.mark.parametrize("H", [64, 65, 1003, 2048, 8191])
def test_nothing_is_written_behind_the_workspace(T, H):
    """Row counts around the CTAs' and rows of any length, with the workspace at the end of what may be written."""
    d = dims(T, H, moe.BF16, (moe.GATE_CHANNEL, moe.ACT_NONE))
    y, r, g, gp, gq = inputs(d)
    s, ds, dxn = ref.randn(5, y.dtype, T, H), ref.randn(6, y.dtype, T, H), ref.randn(7, y.dtype, T, H)
    size = moe.new_norm_workspace(d).numel()
    room = torch.full((size + (4 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    new = lambda t: torch.empty_like(t)  # noqa: E731
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, new(y), new(y), new(g), new(gp), new(gq), room[:size])
    assert bool((room[size:] == 0x5A).all())


@pytest.mark.parametrize("T,H,dtype,gate", [(2500, 1003, moe.BF16, 0), (2500, 1003, moe.FP16, 3), (1201, 77, moe.FP32, 4), (2051, 1544, moe.BF16, 4), (700, 8191, moe.FP32, 3),
                                            (640, 8187, moe.FP32, 5), (641, 8192, moe.FP32, 1), (643, 8191, moe.BF16, 2), (5003, 33, moe.BF16, 5), (9, 8190, moe.FP32, 4), (3, 5, moe.FP16, 0)])
def test_results_over_their_inputs_of_any_row(T, H, dtype, gate):
    """Each pair of buffers that may be shared, with rows that begin anywhere (whose pieces of 16 bytes reach into rows that others
    are writing), rows that are read from memory twice, and every kind of gate: the bits are those of results with buffers of
    their own."""
    d = dims(T, H, dtype, GATES[gate], branch_scale=0.5, residual_scale=0.75)
    y, r, g, gp, gq = inputs(d)
    s, xn = torch.empty_like(y), torch.empty_like(y)
    moe.moe_norm_residual(d, y, r, g, gp, gq, s, xn)
    for over in ("ry", "yr", "y-", "-y", "r-", "-r"):
        b = {"y": y.clone(), "r": r.clone(), "-": torch.empty_like(y)}
        moe.moe_norm_residual(d, b["y"], b["r"], g, gp, gq, b[over[0]], b[over[1]])
        assert torch.equal(b[over[0]], s) and torch.equal(b[over[1]], xn), over
    ds, dxn, ws = ref.randn(7, y.dtype, T, H), ref.randn(8, y.dtype, T, H), moe.new_norm_workspace(d)
    new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    want = [new(t) for t in (y, y, g, gp, gq)]
    moe.moe_norm_residual_backward(d, ds, dxn, s, y, g, gp, gq, *want, ws)
    for over in ("dx", "xd", "sy", "ys", "d-", "-d", "x-", "-y"):
        b = {"d": ds.clone(), "x": dxn.clone(), "s": s.clone(), "y": y.clone(), "-": torch.empty_like(y)}
        got = [b[over[0]], b[over[1]], *[new(t) for t in (g, gp, gq)]]
        moe.moe_norm_residual_backward(d, b["d"], b["x"], b["s"], b["y"], g, gp, gq, *got, ws)
        assert all(p is None or torch.equal(p, q) for p, q in zip(got, want)), over
