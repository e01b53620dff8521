"""Host-side checks of the layer's parts: sizes, and refusals before any launch (the fake device addresses are
never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from sparse_moe_ffn_router_gb300 import binding
from sparse_moe_ffn_router_gb300.binding import LinearDims, NormDims

A = 0x100000000
M = 0x10000000  # apart: more than any buffer here


def at(i):
    return A + i * M


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def R(d):
    return ctypes.byref(d)


def test_sort_refuses(lib):
    def call(T=4, K=2, E=8, ids=at(0), counts=at(1), offsets=at(2), perm=at(3), inv=at(4)):
        return lib.moe_sort_pairs(T, K, E, ids, counts, offsets, perm, inv, None)

    assert call(T=-1) == 1
    for k in (0, 9, -1):
        assert call(K=k) == 2
    for e in (0, 257, -3):
        assert call(E=e) == 2
    assert call(T=2 ** 30, K=2) == 2 and call(T=2 ** 28, K=8) == 2 and call(T=2 ** 31 - 2 ** 16 + 1, K=1) == 2
    for name in ("ids", "counts", "offsets", "perm", "inv"):
        assert call(**{name: None}) == 1
        assert call(**{name: at(9) + 4}) == 3
    assert call(perm=at(0)) == 1 and call(inv=at(0) + 16) == 1 and call(inv=at(3)) == 1 and call(offsets=at(1) + 16) == 1


def test_exchange_refuses(lib):
    def dispatch(dt=0, T=4, K=2, H=64, x=at(0), inv=at(1), w=at(2), rows=at(3)):
        return lib.moe_dispatch(dt, T, K, H, x, inv, w, rows, None)

    def combine(dt=0, T=4, K=2, H=64, rows=at(3), inv=at(1), w=at(2), res=at(0), out=at(4)):
        return lib.moe_combine(dt, T, K, H, rows, inv, w, res, out, None)

    def dispatch_backward(dt=0, T=4, K=2, H=64, rows=at(3), inv=at(1), w=at(2), x=at(0), out=at(4), dw=at(5)):
        return lib.moe_dispatch_backward(dt, T, K, H, rows, inv, w, x, out, dw, None)

    def combine_backward(dt=0, T=4, K=2, H=64, x=at(0), inv=at(1), w=at(2), rows=at(3), out=at(4), dw=at(5)):
        return lib.moe_combine_backward(dt, T, K, H, x, inv, w, rows, out, dw, None)

    for call in (dispatch, combine, dispatch_backward, combine_backward):
        for dt in (-1, 3):
            assert call(dt=dt) == 1
        assert call(T=-1) == 1
        for over in (dict(K=0), dict(K=9), dict(H=0), dict(H=65537), dict(T=2 ** 30, K=2)):
            assert call(**over) == 2
        assert call(T=0) == 0
        assert call(inv=None) == 1 and call(inv=at(1) + 4) == 3 and call(w=at(2) + 8) == 3 and call(rows=None) == 1 and call(rows=at(3) + 2) == 3
    assert dispatch(x=None) == 1 and dispatch(rows=at(0)) == 1 and dispatch(rows=at(2) - 64) == 1
    assert combine(out=None) == 1 and combine(out=at(3)) == 1 and combine(out=at(0) + 16) == 1  # a residual's buffer as a whole or not at all
    assert dispatch_backward(x=None) == 1 and dispatch_backward(out=at(0)) == 1 and dispatch_backward(dw=at(2)) == 1 and dispatch_backward(dw=at(4)) == 1
    assert combine_backward(x=None) == 1 and combine_backward(out=at(3)) == 1 and combine_backward(out=at(0)) == 1 and combine_backward(dw=at(5) + 4) == 3


def test_linear_sizes(lib):
    size = lambda d, b: lib.moe_linear_workspace_size(R(d), b)  # noqa: E731
    assert size(LinearDims(4, 64, 64), 0) > 0 and size(LinearDims(4, 64, 64), 0) % 256 == 0
    d = LinearDims(1000, 1003, 64, act=moe.ACT_SILU)
    assert size(d, 1) >= size(d, 0) + 1000 * 1008 * 2 + 17 * 1003 * 4
    assert size(LinearDims(0, 64, 64), 1) > 0
    for d in (LinearDims(-1, 64, 64), LinearDims(4, 64, 64, act=6), LinearDims(4, 64, 64, act=-1), LinearDims(4, 64, 64, dtype=moe.FP32),
              LinearDims(4, 0, 64), LinearDims(4, 64, 0), LinearDims(4, 64, 4), LinearDims(4, 64, 12), LinearDims(4, 2 ** 20 + 1, 64),
              LinearDims(4, 64, 2 ** 20 + 8), LinearDims(4, 64, 64, E=0), LinearDims(4, 64, 64, E=257), LinearDims(4, 48, 64, act=moe.ACT_SWIGLU),
              LinearDims(2 ** 31 - 1, 64, 64), LinearDims(2 ** 30, 1024, 64), LinearDims(2 ** 30, 64, 1024), LinearDims(4, 2 ** 20, 2 ** 20)):
        assert size(d, 0) == 0 and size(d, 1) == 0
    assert lib.moe_linear_workspace_size(None, 0) == 0
    most = 2 ** 31 - 2 ** 16
    assert size(LinearDims(most, 256, 256), 0) > 0 and size(LinearDims(most + 1, 256, 256), 0) == 0


def test_linear_refuses(lib):
    def call(d=None, x=at(0), w=at(1), bias=at(2), off=None, res=at(4), out=at(5), z=at(6), ws=at(7), wb=None):
        d = d or LinearDims(8, 64, 64, act=moe.ACT_SILU)
        return lib.moe_linear(R(d), x, w, bias, off, res, out, z, ws, lib.moe_linear_workspace_size(R(d), 0) if wb is None else wb, None)

    assert lib.moe_linear(None, *[None] * 8, 0, None) == 1
    assert call(d=LinearDims(8, 64, 64, act=9)) == 1 and call(d=LinearDims(8, 64, 64, dtype=2)) == 1 and call(d=LinearDims(8, 64, 60)) == 2
    assert call(d=LinearDims(8, 64, 64, E=4)) == 1  # several matrices need offsets
    for name in ("x", "w", "out", "ws"):
        assert call(**{name: None}) == 1
    for name in ("x", "w", "res", "out", "z", "ws"):
        assert call(**{name: at(9) + 8}) == 3
    assert call(bias=at(2) + 1) == 3 and call(off=at(3) + 2) == 3
    assert call(wb=100) == 4
    for over in (dict(out=at(0)), dict(out=at(1)), dict(out=at(2)), dict(z=at(5)), dict(z=at(4)), dict(out=at(4) + 16), dict(ws=at(0)), dict(z=at(1) + 64)):
        assert call(**over) == 1
    assert call(d=LinearDims(0, 64, 64), x=None, out=None) == 0


def test_linear_backward_refuses(lib):
    def call(d=None, x=at(0), w=at(1), off=None, z=at(2), dout=at(3), dx=at(4), dw=at(5), db=at(6), ws=at(7), wb=None):
        d = d or LinearDims(8, 64, 64, act=moe.ACT_SILU)
        return lib.moe_linear_backward(R(d), x, w, off, z, dout, dx, dw, db, ws, lib.moe_linear_workspace_size(R(d), 1) if wb is None else wb, None)

    assert call(d=LinearDims(8, 64, 64, act=9)) == 1 and call(d=LinearDims(8, 64, 60)) == 2 and call(d=LinearDims(8, 64, 64, E=4)) == 1
    for name in ("x", "w", "z", "dout", "ws"):
        assert call(**{name: None}) == 1
    for name in ("x", "w", "z", "dout", "dx", "dw", "ws"):
        assert call(**{name: at(9) + 8}) == 3
    assert call(db=at(6) + 1) == 3
    assert call(wb=lib.moe_linear_workspace_size(R(LinearDims(8, 64, 64)), 0)) == 4
    for over in (dict(dx=at(0)), dict(dx=at(3)), dict(dw=at(1)), dict(db=at(5)), dict(ws=at(3) - 512), dict(dx=at(2))):
        assert call(**over) == 1


def test_norm_refuses(lib):
    def forward(d=None, y=at(0), res=at(1), gate=None, gp=at(3), gq=at(4), s=at(5), xn=at(6)):
        return lib.moe_norm_residual(R(d or NormDims(8, 64)), y, res, gate, gp, gq, s, xn, None)

    def backward(d=None, ds=at(0), dxn=at(1), s=at(2), y=at(3), gate=None, gp=at(5), gq=at(6), dres=at(7), dy=at(8), dg=None, dgp=at(10), dgq=at(11), ws=at(12), wb=None):
        d = d or NormDims(8, 64)
        return lib.moe_norm_residual_backward(R(d), ds, dxn, s, y, gate, gp, gq, dres, dy, dg, dgp, dgq, ws, lib.moe_norm_workspace_size(R(d)) if wb is None else wb, None)

    bad = [NormDims(-1, 64), NormDims(8, 64, dtype=3), NormDims(8, 64, gate=4), NormDims(8, 64, gate=-1), NormDims(8, 64, gate_act=moe.ACT_SILU),
           NormDims(8, 64, gate=1, gate_act=moe.ACT_GELU), NormDims(8, 64, eps=-1.0), NormDims(8, 64, eps=float("nan"))]
    flags = NormDims(8, 64)
    flags.flags = 2
    for d in bad + [flags]:
        assert forward(d=d, gate=at(2)) == 1 and backward(d=d, gate=at(2)) == 1 and lib.moe_norm_workspace_size(R(d)) == 0
    for h in (0, 8193, -8):
        assert forward(d=NormDims(8, h)) == 2 and backward(d=NormDims(8, h)) == 2
    assert forward(y=None) == 1 and forward(s=None, xn=None) == 1
    assert forward(gate=at(2)) == 1 and forward(d=NormDims(8, 64, gate=3)) == 1           # a gate where the dims have none, and the other way round
    assert forward(d=NormDims(8, 64, post=False)) == 1                                     # gamma_post without its norm
    for name in ("y", "res", "gp", "gq", "s", "xn"):
        assert forward(**{name: at(13) + 4}) == 3
    assert forward(s=at(6)) == 1 and forward(s=at(0) + 16) == 1 and forward(xn=at(4)) == 1 and forward(d=NormDims(8, 64, gate=3), gate=at(2), s=at(2)) == 1
    assert forward(d=NormDims(0, 64), y=None) == 0
    assert backward(y=None) == 1 and backward(ws=None) == 1 and backward(ds=None, dxn=None) == 1 and backward(s=None) == 1
    assert backward(dxn=None, s=None) == 1                                                 # dgamma_pre without the gradient it is of
    assert backward(dg=at(9)) == 1 and backward(d=NormDims(8, 64, post=False)) == 1 and backward(wb=16) == 4
    for name in ("ds", "dxn", "s", "y", "gp", "gq", "dres", "dy", "dgp", "dgq", "ws"):
        assert backward(**{name: at(13) + 4}) == 3
    assert backward(dres=at(8)) == 1 and backward(dy=at(3) + 64) == 1 and backward(dgp=at(5)) == 1 and backward(ws=at(1)) == 1
    assert forward(d=NormDims(2 ** 31 - 2 ** 16 + 1, 1)) == 2 and lib.moe_norm_workspace_size(R(NormDims(2 ** 31 - 1, 1))) == 0
    assert lib.moe_norm_workspace_size(R(NormDims(10 ** 6, 2048))) == lib.moe_norm_workspace_size(R(NormDims(304, 2048))) > 0
    assert lib.moe_norm_workspace_size(R(NormDims(2, 8191))) >= 8 * 3 * 8191 * 4  # eight CTAs, whatever the rows


def test_binding_refuses():
    b, f, i = torch.bfloat16, torch.float32, torch.int32
    x, rows, inv, w = torch.zeros(4, 64, dtype=b), torch.zeros(8, 64, dtype=b), torch.zeros(8, dtype=i), torch.zeros(4, 2)
    with pytest.raises(ValueError):  # CPU tensors
        moe.moe_dispatch(x, inv, w, rows)
    for bad in (dict(rows=rows.float()), dict(rows=torch.zeros(7, 64, dtype=b)), dict(inv=inv.long()), dict(inv=inv[:7]), dict(w=w.double()), dict(w=w[:, :1])):
        a = dict(x=x, inv=inv, w=w, rows=rows) | bad
        with pytest.raises((TypeError, ValueError)):
            moe.moe_dispatch(a["x"], a["inv"], a["w"], a["rows"])
    with pytest.raises(TypeError):
        moe.moe_sort_pairs(8, torch.zeros(4, 2), *[torch.zeros(n, dtype=i) for n in (8, 9, 8, 8)])
    with pytest.raises(ValueError):
        moe.moe_sort_pairs(8, torch.zeros(4, 2, dtype=i), *[torch.zeros(n, dtype=i) for n in (8, 8, 8, 8)])
    d = moe.LinearDims(4, 32, 64, act=moe.ACT_SWIGLU)
    good = dict(x=x, w=torch.zeros(1, 32, 64, dtype=b), bias=None, offsets=None, residual=None, out=torch.zeros(4, 16, dtype=b), z=None)
    for bad in (dict(), dict(x=x.float()), dict(x=x[:3]), dict(w=torch.zeros(64, 32, dtype=b)), dict(out=torch.zeros(4, 32, dtype=b)),
                dict(bias=torch.zeros(16, dtype=b)), dict(z=torch.zeros(4, 16, dtype=b)), dict(residual=torch.zeros(4, 16)), dict(offsets=torch.zeros(3, dtype=i))):
        a = good | bad
        with pytest.raises((TypeError, ValueError)):
            moe.moe_linear(d, *a.values(), torch.zeros(512, dtype=torch.uint8))
    n = moe.NormDims(4, 64, gate=moe.GATE_TOKEN)
    good = dict(y=x, residual=x, gate=torch.zeros(4, dtype=b), gp=None, gq=None, s=x, xn=x)
    for bad in (dict(), dict(y=x.float()), dict(residual=x[:3]), dict(gate=torch.zeros(64, dtype=b)), dict(gp=torch.zeros(4, dtype=b)), dict(gq=torch.zeros(64, dtype=f))):
        a = good | bad
        with pytest.raises((TypeError, ValueError)):
            moe.moe_norm_residual(n, *a.values())
    for size in (moe.new_linear_workspace, ):
        with pytest.raises(moe.MoEError):
            size(moe.LinearDims(4, 33, 64, act=moe.ACT_SWIGLU), device="cpu")
    with pytest.raises(moe.MoEError):
        moe.new_norm_workspace(moe.NormDims(4, 9000), device="cpu")


def test_dims_may_be_changed():
    """What the checks work out of the dims once is worked out again when a field is set."""
    d = moe.LinearDims(4, 32, 64)
    assert d.checked[1] == (4, 64) and d.checked[2] == (4, 32)
    d.T, d.act = 6, moe.ACT_SWIGLU
    assert d.checked[1] == (6, 64) and d.checked[2] == (6, 16)
    n = moe.NormDims(4, 64, gate=moe.GATE_TOKEN)
    assert n.checked[3] == (4,)
    n.gate = moe.GATE_FULL
    assert n.checked[3] == (4, 64)
    with pytest.raises(AttributeError):
        d.nothing
    d.dtype = 9
    with pytest.raises(moe.MoEError):
        d.checked


def test_binding_names_an_argument_of_another_kind():
    """A tensor that is missing or something else, and dims of another call: a TypeError that says which."""
    b, i = torch.bfloat16, torch.int32
    x, ids, inv = torch.zeros(4, 64, dtype=b), torch.zeros(4, 2, dtype=i), torch.zeros(4, dtype=i)
    d, n = moe.LinearDims(4, 64, 64), moe.NormDims(4, 64)
    for what, call in (("ids", lambda: moe.moe_sort_pairs(8, None, ids, ids, ids, ids)), ("token rows", lambda: moe.moe_dispatch(None, inv, None, x)),
                       ("experts' rows", lambda: moe.moe_combine([x], inv, None, None, x)), ("token rows", lambda: moe.moe_dispatch_backward(x, inv, None, None, 3)),
                       ("experts' rows", lambda: moe.moe_combine_backward(x, inv, None, None, None)), ("x", lambda: moe.moe_linear(d, None, x, None, None, None, x, None, x)),
                       ("dout", lambda: moe.moe_linear_backward(d, x, x, None, None, None, x, x, None, x)), ("y", lambda: moe.moe_norm_residual(n, None, x, None, None, None, x, x)),
                       ("y", lambda: moe.moe_norm_residual_backward(n, x, x, x, None, None, None, None, x, x, None, None, None, x)),
                       ("dims", lambda: moe.moe_linear(n, x, x, None, None, None, x, None, x)), ("dims", lambda: moe.moe_norm_residual((4, 64), x, x, None, None, None, x, x))):
        with pytest.raises(TypeError, match=f"^{what}: expected"):
            call()
