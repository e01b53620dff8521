"""Linear layers with bias, activation and residual, dense and by expert, and their gradients, against plain forms."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import parts_reference as ref

pytestmark = pytest.mark.gpu
DT = {moe.BF16: torch.bfloat16, moe.FP16: torch.float16}
NAN = float("nan")


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def inputs(d, bias=True, residual=True, seed=0):
    dt, wide = DT[d.dtype], d.N // 2 if d.act == moe.ACT_SWIGLU else d.N
    x, w = ref.randn(seed + 1, dt, d.T, d.K), ref.randn(seed + 2, dt, d.E, d.N, d.K, scale=d.K ** -0.5)
    return x, w, ref.randn(seed + 3, dt, d.E, d.N) if bias else None, ref.randn(seed + 4, dt, d.T, wide) if residual else None


def forward(d, x, w, bias, offsets, residual, fill=7.0, keep=True):
    wide = d.N // 2 if d.act == moe.ACT_SWIGLU else d.N
    out = torch.full((d.T, wide), fill, dtype=x.dtype, device="cuda")
    z = torch.full((d.T, d.N), fill, dtype=x.dtype, device="cuda") if keep else None
    ws = moe.new_linear_workspace(d)
    moe.moe_linear(d, x, w, bias, offsets, residual, out, z, ws)
    assert moe.moe_last_device_error(ws) == 0
    return out, z


def check_forward(d, x, w, bias, offsets, residual):
    out, z = forward(d, x, w, bias, offsets, residual)
    o64, z64, mo, mz = ref.linear(d, x, w, bias, offsets, residual)
    n = d.T if offsets is None else int(offsets[-1])
    ref.check(out[:n], o64[:n], mo[:n], d.K + 2, "out")
    ref.check(z[:n], z64[:n], mz[:n], d.K + 2, "z")
    assert bool((out[n:] == 7).all()) and bool((z[n:] == 7).all())
    return z


def check_backward(d, x, w, offsets, z, seed=9):
    wide = d.N // 2 if d.act == moe.ACT_SWIGLU else d.N
    dout = ref.randn(seed, x.dtype, d.T, wide)
    n = d.T if offsets is None else int(offsets[-1])
    dout[n:] = NAN  # rows of no expert are read into nothing
    dx, dw, db = torch.full_like(x, 7.0), torch.full_like(w, 7.0), torch.full((d.E, d.N), 7.0, dtype=x.dtype, device="cuda")
    ws = moe.new_linear_workspace(d, backward=True)
    ws[512:] = 255  # the error word's line apart, it holds nothing yet: NaN in both types
    moe.moe_linear_backward(d, x, w, offsets, z if d.act != moe.ACT_NONE else None, dout, dx, dw, db, ws)
    assert moe.moe_last_device_error(ws) == 0
    clean = torch.nan_to_num(dout)
    want, bound = ref.linear_backward(d, x.nan_to_num(), w, offsets, z.nan_to_num() if d.act != moe.ACT_NONE else None, clean)
    for name, g, r, b in zip(("dx", "dw", "db"), (dx[:n], dw, db), (want[0][:n], *want[1:]), (bound[0][:n], *bound[1:])):
        off = (g.double() - r).abs()
        assert not bool((~(off <= b)).any()), f"{name}: worst {float((off / b).max()):.2f} x the bound"
    assert bool((dx[n:] == 7).all())
    for keep in range(3):  # each gradient alone has the same bits
        some = [torch.empty_like(t) if i == keep else None for i, t in enumerate((dx, dw, db))]
        if keep == 0:
            some[0].fill_(7.0)
        moe.moe_linear_backward(d, x if keep == 1 else None, w if keep == 0 else None, offsets, z if d.act != moe.ACT_NONE else None, dout, *some, ws)
        assert torch.equal(some[keep], (dx, dw, db)[keep])


DENSE = [(1, 2048, 2048), (1, 1, 8), (2, 7, 16), (3, 130, 72), (15, 64, 64), (16, 257, 512), (17, 5003, 144), (31, 128, 1032), (33, 256, 200), (64, 1024, 2048), (65, 96, 88),
         (100, 1000, 264), (129, 40, 1544), (255, 513, 96), (257, 2048, 512), (700, 1003, 1544), (1021, 2056, 72), (2500, 384, 640)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,N,K", DENSE)
def test_dense(dtype, T, N, K):
    act = (moe.ACT_NONE, moe.ACT_RELU, moe.ACT_SILU, moe.ACT_GELU, moe.ACT_SIGMOID)[(T + N + K) % 5]
    d = moe.LinearDims(T, N, K, act=act, dtype=dtype)
    x, w, b, r = inputs(d, bias=T % 3 != 0, residual=T % 2 == 0)
    check_backward(d, x, w, None, check_forward(d, x, w, b, None, r))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", range(6))
@pytest.mark.parametrize("T", [5, 300])
def test_activations(dtype, act, T):
    d = moe.LinearDims(T, 160, 128, act=act, dtype=dtype)
    x, w, b, r = inputs(d)
    check_backward(d, x, w, None, check_forward(d, x, w, b, None, r))


COUNTS = [[0, 1], [3, 0, 0, 5], [0, 0, 0], [1] * 40, [64, 65, 0, 63, 1], [16, 0, 17, 15, 256, 257, 100], [700, 1, 0, 2], [0, 0, 1000], [33] * 256]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K,act", [(128, 64, moe.ACT_NONE), (96, 200, moe.ACT_SWIGLU), (77, 136, moe.ACT_SILU), (352, 72, moe.ACT_SWIGLU)])
@pytest.mark.parametrize("spare", [0, 29])
def test_experts(dtype, counts, N, K, act, spare):
    """Experts without rows, with one, around 16, 64 and 256; rows behind the last expert's that hold NaN."""
    off = offsets_of(counts)
    T = int(off[-1]) + spare
    if T == 0:
        T = 4
    d = moe.LinearDims(T, N, K, E=len(counts), act=act, dtype=dtype)
    x, w, b, r = inputs(d)
    n = int(off[-1])
    x[n:] = NAN
    z = check_forward(d, x, w, b, off, r)
    z[n:] = NAN
    check_backward(d, x, w, off, z)


def test_one_expert_with_offsets_takes_a_part():
    d = moe.LinearDims(90, 64, 64, act=moe.ACT_SILU)
    x, w, b, r = inputs(d)
    off = torch.tensor([7, 50], dtype=torch.int32, device="cuda")
    out, z = forward(d, x, w, b, off, r)
    whole, _ = forward(d, x, w, b, None, r)
    assert torch.equal(out[7:50], whole[7:50]) and bool((out[:7] == 7).all()) and bool((out[50:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_experts_do_not_reach_one_another(bad):
    """Non-finite weights and rows of one expert stay in that expert's results: tiles read past its rows and columns."""
    counts = [5, 70, 0, 33, 1]
    off = offsets_of(counts)
    d = moe.LinearDims(int(off[-1]), 100, 136, E=5)
    x, w, b, _ = inputs(d, residual=False)
    dout = ref.randn(5, x.dtype, d.T, d.N)
    ws = moe.new_linear_workspace(d, backward=True)

    def grads(x, w, dout):
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        moe.moe_linear_backward(d, x, w, off, None, dout, dx, dw, db, ws)
        return dx, dw, db

    out, _ = forward(d, x, w, b, off, None)
    clean = grads(x, w, dout)
    for e in (1, 3):
        xb, wb, db_ = x.clone(), w.clone(), dout.clone()
        a, c = int(off[e]), int(off[e + 1])
        xb[a:c], wb[e], db_[a:c] = bad, bad, bad
        rows = torch.ones(d.T, dtype=torch.bool, device="cuda")
        rows[a:c] = False
        others = [i for i in range(5) if i != e]
        got, _ = forward(d, xb, wb, b, off, None)
        assert torch.equal(got[rows], out[rows])
        g = grads(xb, wb, db_)
        assert torch.equal(g[0][rows], clean[0][rows]) and torch.equal(g[1][others], clean[1][others]) and torch.equal(g[2][others], clean[2][others])


def test_residual_may_be_the_result():
    for T in (3, 300):
        d = moe.LinearDims(T, 200, 64, act=moe.ACT_GELU)
        x, w, b, r = inputs(d)
        out, _ = forward(d, x, w, b, None, r)
        moe.moe_linear(d, x, w, b, None, r, r, None, moe.new_linear_workspace(d))
        assert torch.equal(r, out)


def test_offsets_out_of_order_are_flagged():
    d = moe.LinearDims(64, 64, 64, E=3)
    x, w, b, _ = inputs(d, residual=False)
    ws = moe.new_linear_workspace(d)
    out = torch.zeros(64, 64, dtype=x.dtype, device="cuda")
    for off in ([0, 40, 20, 64], [0, 10, 20, 65], [-1, 10, 20, 64], [2 ** 31 - 1, -2 ** 31, 5, 6]):
        moe.moe_linear(d, x, w, b, torch.tensor(off, dtype=torch.int32, device="cuda"), None, out, None, ws)
        assert moe.moe_last_device_error(ws) == 7 and moe.moe_last_device_error(ws) == 0
    moe.moe_linear(d, x, w, b, torch.tensor([0, 10, 20, 64], dtype=torch.int32, device="cuda"), None, out, None, ws)
    assert moe.moe_last_device_error(ws) == 0


def test_no_rows():
    d = moe.LinearDims(0, 64, 64)
    z, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear(d, z, w, None, None, None, z, None, moe.new_linear_workspace(d))
    dw, db = w.clone(), w[0].clone()
    moe.moe_linear_backward(d, z, w, None, None, z, z, dw, db, moe.new_linear_workspace(d, backward=True))
    assert not bool(dw.any()) and not bool(db.any())


def test_gradients_against_differences():
    """Central differences of the plain forward pass in 64 bits along random directions. Their error is h^2 / 6 of the third
    derivative (below 2 for these functions of arguments of unit size: 1e-6 of the magnitudes with h = 1e-3 is ample); the
    kernel's side carries the bounds of its rounding."""
    d = moe.LinearDims(70, 64, 40, E=3, act=moe.ACT_SWIGLU, dtype=moe.FP16)
    off = offsets_of([20, 0, 50])
    x, w, b, _ = inputs(d, residual=False)
    _, z = forward(d, x, w, b, off, None)
    dout = ref.randn(8, x.dtype, 70, 32)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    moe.moe_linear_backward(d, x, w, off, z, dout, dx, dw, db, moe.new_linear_workspace(d, backward=True))
    _, bounds = ref.linear_backward(d, x, w, off, z, dout)
    loss = lambda x, w, b: float((ref.linear(d, x, w, b, off, None)[0] * dout.double()).sum())  # noqa: E731
    h, wide = 1e-3, [t.double() for t in (x, w, b)]
    for i, (g, bound) in enumerate(zip((dx, dw, db), bounds)):
        v = ref.randn(20 + i, torch.float64, *g.shape)
        up, down = ([t + s * h * v if j == i else t for j, t in enumerate(wide)] for s in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # the z that the pass kept is rounded: its slopes are off by half a step of z times the second derivative (below 1.2)
        kept = 2 * ref.unit(x.dtype) * float((g.double().abs() * v.abs()).sum()) * 4
        assert abs(diff - float((g.double() * v).sum())) <= float((bound * v.abs()).sum()) + kept + 1e-6 * float((g.double() * v).abs().sum())


def test_a_held_back_load_ends_in_an_error():
    """A stage that never fills: the kernel gives up after the limit and says so, and the next call is whole."""
    for T in (1, 300):
        d = moe.LinearDims(T, 2048, 1024)
        x, w, b, r = inputs(d)
        out, _ = forward(d, x, w, b, None, r, keep=False)
        ws = moe.new_linear_workspace(d)
        again = torch.empty_like(out)
        try:
            moe.moe_test_set_wait(2_000_000, moe.TEST_SUPPRESS_STAGE)
            moe.moe_linear(d, x, w, b, None, r, again, None, ws)
            assert moe.moe_last_device_error(ws) == 6
        finally:
            moe.moe_test_set_wait()
        moe.moe_linear(d, x, w, b, None, r, again, None, ws)
        assert moe.moe_last_device_error(ws) == 0 and torch.equal(again, out)


def test_offsets_out_of_order_are_flagged_for_few_rows():
    d = moe.LinearDims(6, 64, 64, E=3)
    x, w, b, _ = inputs(d, residual=False)
    ws, out = moe.new_linear_workspace(d), torch.zeros(6, 64, dtype=x.dtype, device="cuda")
    for off in ([0, 4, 2, 6], [0, 1, 2, 7], [-1, 1, 2, 6], [2 ** 31 - 1, -2 ** 31, 5, 6], [0, 6, 0, 6]):
        moe.moe_linear(d, x, w, b, torch.tensor(off, dtype=torch.int32, device="cuda"), None, out, None, ws)
        assert moe.moe_last_device_error(ws) == 7 and moe.moe_last_device_error(ws) == 0


@pytest.mark.parametrize("T", [64, 700])
@pytest.mark.parametrize("wanted", ["dx", "dw", "dbias"])
def test_offsets_out_of_order_are_flagged_by_every_gradient(T, wanted):
    d = moe.LinearDims(T, 64, 64, E=3, act=moe.ACT_SILU)
    x, w, b, _ = inputs(d, residual=False)
    ws, z, dout = moe.new_linear_workspace(d, backward=True), ref.randn(7, x.dtype, T, 64), ref.randn(8, x.dtype, T, 64)
    out = {"dx": torch.zeros_like(x), "dw": torch.zeros_like(w), "dbias": torch.zeros_like(b)}
    one = [out[k] if k == wanted else None for k in out]
    for off in ([0, 40, 20, T], [0, 10, 20, T + 1], [-1, 10, 20, T], [2 ** 31 - 1, -2 ** 31, 5, 6]):
        moe.moe_linear_backward(d, x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), z, dout, *one, ws)
        assert moe.moe_last_device_error(ws) == 7 and moe.moe_last_device_error(ws) == 0
    moe.moe_linear_backward(d, x, w, torch.tensor([0, 10, 20, T], dtype=torch.int32, device="cuda"), z, dout, *one, ws)
    assert moe.moe_last_device_error(ws) == 0


@pytest.mark.parametrize("T", [1, 2, 8, 9, 40, 64, 65])
def test_residual_may_be_the_result_of_every_kernel(T):
    for act, N in ((moe.ACT_NONE, 2048), (moe.ACT_SWIGLU, 1024)):
        d = moe.LinearDims(T, N, 2048, act=act)
        x, w, b, r = inputs(d)
        out, _ = forward(d, x, w, b, None, r)
        moe.moe_linear(d, x, w, b, None, r, r, None, moe.new_linear_workspace(d))
        assert torch.equal(r, out)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,N,K,E", [(2, 2048, 512, 0), (3, 1003, 1024, 0), (4, 96, 2048, 0), (8, 130, 4104, 0), (5, 64, 64, 40), (64, 224, 520, 32), (64, 32, 1032, 256), (17, 77, 8, 9)])
def test_few_rows(dtype, T, N, K, E):
    """One to four features a warp, rows in batches of four and eight, rows of experts one at a time; with every part of the epilogue."""
    for act in (moe.ACT_GELU, moe.ACT_SWIGLU):
        n = N // 32 * 32 if act == moe.ACT_SWIGLU else N
        d = moe.LinearDims(T, n, K, E=max(E, 1), act=act, dtype=dtype)
        off = None
        if E:
            g = torch.Generator().manual_seed(T)
            off = offsets_of(torch.bincount(torch.randint(0, E, (T,), generator=g), minlength=E).tolist())
        x, w, b, r = inputs(d)
        check_forward(d, x, w, b, off, r)


@pytest.mark.parametrize("T,N,K", [(300, 1001, 64), (513, 259, 72), (700, 1004, 136)])
def test_rows_that_do_not_start_on_16_bytes(T, N, K):
    """The whole epilogue and the way back where a row of the result begins anywhere: nothing beside the rows is touched."""
    for act in (moe.ACT_NONE, moe.ACT_SILU):
        d = moe.LinearDims(T, N, K, act=act)
        x, w, b, r = inputs(d)
        room = torch.full((T * N + 64,), 7.0, dtype=x.dtype, device="cuda")
        out = room[:T * N].view(T, N)
        moe.moe_linear(d, x, w, b, None, r, out, None, moe.new_linear_workspace(d))
        o64, _, mo, _ = ref.linear(d, x, w, b, None, r)
        ref.check(out, o64, mo, K + 2, "out")
        assert bool((room[T * N:] == 7).all())
        check_backward(d, x, w, None, check_forward(d, x, w, b, None, r))


@pytest.mark.parametrize("keep", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
def test_bias_gradient_beside_any_product(keep):
    """The bias' sums are added up by whichever kernel runs, or one of its own."""
    for counts in ([500, 0, 33, 1], [130] * 7):
        off = offsets_of(counts)
        d = moe.LinearDims(int(off[-1]) + 5, 264, 136, E=len(counts), act=moe.ACT_SILU)
        x, w, b, _ = inputs(d)
        _, z = forward(d, x, w, b, off, None)
        dout, ws = ref.randn(5, x.dtype, d.T, d.N), moe.new_linear_workspace(d, backward=True)
        full = [torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(b)]
        moe.moe_linear_backward(d, x, w, off, z, dout, *full, ws)
        some = [torch.zeros_like(t) if k else None for t, k in zip(full, keep)]
        moe.moe_linear_backward(d, x, w, off, z, dout, *some, ws)
        assert all(s is None or torch.equal(s, t) for s, t in zip(some, full))


@pytest.mark.parametrize("T,N,K,counts", [(1, 7, 16, None), (33, 1003, 72, None), (700, 130, 64, None), (45, 77, 40, [0, 33, 0, 7, 5]), (600, 96, 64, [33] * 18 + [6])])
def test_nothing_is_written_behind_the_workspace(T, N, K, counts):
    off = None if counts is None else offsets_of(counts)
    d = moe.LinearDims(T, N, K, E=1 if counts is None else len(counts), act=moe.ACT_SILU)
    x, w, b, _ = inputs(d, residual=False)
    z, dout = ref.randn(5, x.dtype, T, N), ref.randn(6, x.dtype, T, N)
    size = moe.new_linear_workspace(d, backward=True).numel()
    room = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    room[:512] = 0
    moe.moe_linear_backward(d, x, w, off, z, dout, torch.empty_like(x), torch.empty_like(w), torch.empty_like(b), room[:size])
    assert moe.moe_last_device_error(room[:size]) == 0 and bool((room[size:] == 0x5A).all())


@pytest.mark.parametrize("T,N,counts,act", [(8192, 1203, None, moe.ACT_GELU), (0, 1280, [33] * 256, moe.ACT_SILU), (0, 2560, [0, 127, 1, 0, 128, 129, 6000, 700], moe.ACT_SWIGLU)])
def test_many_rows_in_chunks_of_128(T, N, counts, act):
    """Row counts from which the elementwise pass of the way back takes four times the rows at once."""
    off = None if counts is None else offsets_of(counts)
    d = moe.LinearDims(T if counts is None else int(off[-1]) + 3, N, 72, E=1 if counts is None else len(counts), act=act)
    x, w, b, _ = inputs(d, residual=False)
    check_backward(d, x, w, off, ref.randn(5, x.dtype, d.T, N))


@pytest.mark.parametrize("counts", [[0, 1, 3, 0, 2] * 30, [8] * 64, [0] * 255 + [5], [1] * 256, [513] + [0] * 63, [7, 0]])
@pytest.mark.parametrize("N,act", [(317, moe.ACT_SILU), (256, moe.ACT_SWIGLU)])
def test_experts_with_a_handful_of_rows(N, act, counts):
    """Row counts up to which the elementwise pass of the way back takes four rows at once, and the sums' place behind its workspace."""
    off = offsets_of(counts)
    d = moe.LinearDims(int(off[-1]) + 2, N, 72, E=len(counts), act=act)
    x, w, b, _ = inputs(d, residual=False)
    z = ref.randn(5, x.dtype, d.T, N)
    check_backward(d, x, w, off, z)
    size = moe.new_linear_workspace(d, backward=True).numel()
    room = torch.zeros(size + (1 << 20), dtype=torch.uint8, device="cuda")
    room[size:] = 0x5A
    moe.moe_linear_backward(d, x, w, off, z, torch.ones(d.T, N // 2 if act == moe.ACT_SWIGLU else N, dtype=x.dtype, device="cuda"), None, None, torch.empty_like(b), room[:size])
    assert moe.moe_last_device_error(room[:size]) == 0 and bool((room[size:] == 0x5A).all())


def test_results_past_32_bits_of_elements():
    """Rows and matrices that begin behind element 2^31."""
    d = moe.LinearDims(32800, 65560, 64, act=moe.ACT_RELU)
    assert d.T * d.N > 2 ** 31
    x, w, b, _ = inputs(d, residual=False)
    out, z = (torch.empty(d.T, d.N, dtype=x.dtype, device="cuda") for _ in range(2))
    moe.moe_linear(d, x, w, b, None, None, out, z, moe.new_linear_workspace(d))
    for rows in (slice(0, 40), slice(d.T // 2, d.T // 2 + 40), slice(d.T - 40, d.T)):
        part = moe.LinearDims(40, d.N, d.K, act=d.act)
        o64, z64, mo, mz = ref.linear(part, x[rows], w, b, None, None)
        ref.check(out[rows], o64, mo, d.K + 2, "out")
        ref.check(z[rows], z64, mz, d.K + 2, "z")
    dx, db = torch.empty_like(x), torch.empty_like(b)
    moe.moe_linear_backward(d, None, w, None, z, out, dx, None, db, moe.new_linear_workspace(d, backward=True))
    for rows in (slice(0, 40), slice(d.T - 40, d.T)):
        part = moe.LinearDims(40, d.N, d.K, act=d.act)
        want, bound = ref.linear_backward(part, x[rows], w, None, z[rows], out[rows])
        assert not bool((~((dx[rows].double() - want[0]).abs() <= bound[0])).any())


def test_matrices_past_32_bits_of_elements():
    d = moe.LinearDims(700, 4104, 2056, E=256)
    assert d.E * d.N * d.K > 2 ** 31
    off = offsets_of([2] * 250 + [0, 100, 0, 30, 0, 70])
    x, w = ref.randn(1, torch.bfloat16, d.T, d.K), torch.empty(d.E, d.N, d.K, dtype=torch.bfloat16, device="cuda")
    for i in range(0, d.E, 16):
        w[i:i + 16] = ref.randn(i, torch.bfloat16, 16, d.N, d.K, scale=d.K ** -0.5)
    out, dout, dw = torch.empty(d.T, d.N, dtype=x.dtype, device="cuda"), ref.randn(3, torch.bfloat16, d.T, d.N), torch.empty_like(w)
    moe.moe_linear(d, x, w, None, off, None, out, None, moe.new_linear_workspace(d))
    dx = torch.empty_like(x)
    moe.moe_linear_backward(d, x, w, off, None, dout, dx, dw, None, moe.new_linear_workspace(d, backward=True))
    for e, a, c in ((0, 0, 2), (251, 500, 600), (253, 600, 630), (255, 630, 700)):
        part = moe.LinearDims(c - a, d.N, d.K)
        o64, _, mo, _ = ref.linear(part, x[a:c], w[e:e + 1], None, None, None)
        ref.check(out[a:c], o64, mo, d.K, "out")
        want, bound = ref.linear_backward(part, x[a:c], w[e:e + 1], None, None, dout[a:c])
        for name, g, r, v in (("dx", dx[a:c], want[0], bound[0]), ("dw", dw[e], want[1][0], bound[1][0])):
            assert not bool((~((g.double() - r).abs() <= v)).any()), name
    assert not bool(dw[250].any()) and not bool(dw[254].any())


@pytest.mark.parametrize("T,N,K,E,which,limit_us", [(32768, 8192, 4096, 1, "out", 300), (32768, 4096, 8192, 1, "dx", 300), (1 << 19, 1024, 1024, 1, "dw", 200), (1 << 19, 1024, 1024, 2, "dw", 200),
                                                    (1 << 22, 256, 256, 1, "dw", 200)])
def test_a_limit_bounds_a_stall_not_the_call(T, N, K, E, which, limit_us):
    """Products of a millisecond or more under a limit that no wait of theirs comes near: tiles one after another, one tile's long
    contraction, and a ragged last block of rows at the end of one. They are whole and report no time-out."""
    d = moe.LinearDims(T, N, K, E=E)
    x, w, _, _ = inputs(d, bias=False, residual=False)
    off = offsets_of([T // 2, T // 2 - 5]) if E == 2 else None
    ws, dout = moe.new_linear_workspace(d, backward=True), ref.randn(5, x.dtype, T, N)

    def call():
        o = torch.zeros_like(dout) if which == "out" else torch.zeros_like(x) if which == "dx" else torch.zeros_like(w)
        if which == "out":
            moe.moe_linear(d, x, w, None, off, None, o, None, ws)
        else:
            moe.moe_linear_backward(d, x, w, off, None, dout, o if which == "dx" else None, o if which == "dw" else None, None, ws)
        return o

    want = call()
    assert moe.moe_last_device_error(ws) == 0
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    try:
        moe.moe_test_set_wait(limit_us * 1000)
        start.record()
        got = call()
        end.record()
        torch.cuda.synchronize()
    finally:
        moe.moe_test_set_wait()
    assert moe.moe_last_device_error(ws) == 0
    assert torch.equal(got, want)
    assert start.elapsed_time(end) * 1e3 > limit_us  # (else the limit would show nothing)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("N,K,step", [(1024, 512, 1), (520, 2048, 3)])
def test_weight_gradients_of_ragged_experts_see_their_rows_alone(N, K, step, bad):
    """Experts of every count around whole 16s, each second one's rows non-finite: they are in the same 64 rows of both operands of
    both SMs of a pair as the ends of the others, tile after tile."""
    counts = [33 + step * i % 97 for i in range(128)]
    off = offsets_of(counts)
    d = moe.LinearDims(int(off[-1]) + 3, N, K, E=128)
    x, w, _, _ = inputs(d, bias=False, residual=False)
    dout, ws = ref.randn(5, x.dtype, d.T, N), moe.new_linear_workspace(d, backward=True)
    want = torch.empty_like(w)
    moe.moe_linear_backward(d, x, None, off, None, dout, None, want, None, ws)
    r64, bounds = ref.linear_backward(d, x, w, off, None, dout)
    assert not bool((~((want.double() - r64[1]).abs() <= bounds[1])).any())
    for turn in range(8):
        xb, db, got = x.clone(), dout.clone(), torch.empty_like(w)
        for e in range(turn % 2, 128, 2):
            a, c = int(off[e]), int(off[e + 1])
            if turn % 4 < 2:
                xb[a:c] = bad
            else:
                db[a:c] = bad
        moe.moe_linear_backward(d, xb, None, off, None, db, None, got, None, ws)
        assert torch.equal(got[1 - turn % 2::2], want[1 - turn % 2::2])
    assert moe.moe_last_device_error(ws) == 0
