"""Pairs sorted by expert, rows to their experts and back, and the gradients, against plain forms."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import parts_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def make_ids(seed, T, E, K, drop=0.0, same=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    if same:
        ids[:, :] = int(ids[0, 0])
    if drop:
        gone = torch.rand(T, K, generator=g) < drop
        ids[gone] = torch.where(torch.rand(T, K, generator=g) < 0.5, -1, E)[gone].to(torch.int32)
    return ids.cuda()


@pytest.mark.parametrize("T,E,K,drop,same", [
    (1, 256, 8, 0, False), (1, 1, 1, 0, False), (1, 4, 3, 1.0, False), (31, 256, 8, 0.2, False), (128, 33, 8, 0, False), (129, 32, 8, 0.5, False),
    (1000, 7, 1, 0.1, False), (513, 2, 2, 0, True), (1025, 256, 8, 0.05, False), (4096, 256, 8, 0, False), (4099, 255, 7, 0.3, False), (5000, 3, 5, 0.01, True)])
def test_sort(T, E, K, drop, same):
    """Every cluster size, dropped ids below and above the experts', an expert named twice by a token, one expert for all."""
    ids = make_ids(T + E, T, E, K, drop, same)
    got = ref.sort_gpu(ids, E)
    for name, a, b in zip(("counts", "offsets", "perm", "inv"), got, ref.sort(ids, E)):
        assert torch.equal(a.cpu(), b), name


def test_sort_extreme_ids_and_none():
    ids = torch.tensor([[2 ** 31 - 1, -2 ** 31, 5, 256], [-1, 4, 5, 5]], dtype=torch.int32, device="cuda")
    for a, b in zip(ref.sort_gpu(ids, 6), ref.sort(ids, 6)):
        assert torch.equal(a.cpu(), b)
    none = ref.sort_gpu(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert none[0].tolist() == [0] * 9 and none[1].tolist() == [0] * 10


def test_sort_agrees_with_the_routing():
    dims = (300, 512, 32, 4, 128, 128)
    w = moe.Weights(*[ref.randn(i, torch.bfloat16, *s, scale=0.05) for i, s in enumerate(
        [(32, 512), (32,), (32, 256, 512), (32, 512, 128), (256, 512), (512, 128), (1, 512)])])
    x = ref.randn(9, torch.bfloat16, 300, 512)
    ids, counts, offsets, perm = (torch.empty(n, dtype=torch.int32, device="cuda") for n in ((300, 4), (32,), (33,), (1200,)))
    moe.moe_route(dims, x, w, ids, torch.empty(300, 4, device="cuda"), counts, offsets, perm, moe.new_workspace(dims))
    got = ref.sort_gpu(ids, 32)
    assert torch.equal(got[0], counts) and torch.equal(got[1], offsets) and torch.equal(got[2], perm)


SIZES = [(1, 8, 256, 2048), (1, 1, 1, 1), (3, 2, 4, 8), (5, 8, 16, 77), (33, 6, 60, 1541), (64, 8, 8, 4096), (2433, 3, 11, 264), (2432, 8, 256, 100)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,E,H", SIZES)
@pytest.mark.parametrize("weights,drop", [(False, 0), (True, 0.3), (True, 1.0)])
def test_all_directions(dtype, T, K, E, H, weights, drop):
    """Each call against 64 bits; rows that are no pair's place keep what they held, and NaN in them or in the
    token rows' place of a dropped slot reaches nothing."""
    ids = make_ids(T * K, T, E, K, drop)
    inv = ref.sort_gpu(ids, E)[3]
    n_live = int((inv >= 0).sum())
    x, res = ref.randn(1, dtype, T, H), ref.randn(2, dtype, T, H)
    rows = ref.randn(3, dtype, T * K, H)
    rows[n_live:] = float("nan")
    w = torch.softmax(ref.randn(4, torch.float32, T, K), 1) if weights else None
    one = 0 if w is None else 1  # roundings of a scaled row before its last: none, the product's is the last
    # dispatch
    out = torch.full((T * K, H), 7.0, dtype=dtype, device="cuda")
    moe.moe_dispatch(x, inv, w, out)
    want = ref.spread(x, inv, w, torch.full_like(out, 7.0))
    if w is None:
        assert torch.equal(out.double(), want)
    else:
        ref.check(out, want, want.abs(), one, "dispatch")
    assert bool((out[n_live:] == 7).all())
    # combine, with and without the residual, and over it
    s, mag = ref.gather(rows, inv, w, T)
    out = torch.empty_like(x)
    moe.moe_combine(rows, inv, w, None, out)
    ref.check(out, s, mag, K, "combine")
    moe.moe_combine(rows, inv, w, res, out)
    ref.check(out, s + res.double(), mag + res.double().abs(), K + 1, "combine with residual")
    over = res.clone()
    moe.moe_combine(rows, inv, w, over, over)
    assert torch.equal(over, out)
    # gradients
    d, dmag = ref.dots(x, rows, inv, T)
    dx, dw = torch.empty_like(x), torch.full((T, K), 7.0, device="cuda")
    moe.moe_dispatch_backward(rows, inv, w, x, dx, dw)
    ref.check(dx, s, mag, K, "dx")
    ref.check(dw, d, dmag, H, "dw of dispatch")
    alone = torch.empty_like(dx)
    moe.moe_dispatch_backward(rows, inv, w, None, alone)
    assert torch.equal(alone, dx)
    drows, dw2 = torch.full((T * K, H), 7.0, dtype=dtype, device="cuda"), torch.full((T, K), 7.0, device="cuda")
    moe.moe_combine_backward(x, inv, w, rows, drows, dw2)
    want = ref.spread(x, inv, w, torch.full_like(drows, 7.0))
    ref.check(drows, want, want.abs(), one, "drows")
    ref.check(dw2, d, dmag, H, "dw of combine")
    alone = torch.full_like(drows, 7.0)
    moe.moe_combine_backward(x, inv, w, None, alone)
    assert torch.equal(alone, drows)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,E,H", [(700, 8, 64, 2044), (2500, 4, 16, 262), (40, 3, 9, 1030), (1300, 2, 5, 516), (9, 8, 12, 6)])
def test_rows_that_start_on_8_or_4_bytes(dtype, T, K, E, H):
    test_all_directions(dtype, T, K, E, H, True, 0.2)


def test_gradients_against_differences():
    """Central differences of the plain forward pass in 64 bits along a random direction: linear in each input, so exact but for
    64-bit rounding; the kernel's side carries its fp32 bounds."""
    T, K, E, H = 17, 3, 5, 40
    inv = ref.sort_gpu(make_ids(3, T, E, K, 0.2), E)[3]
    rows, x, w, dout = ref.randn(1, torch.float32, T * K, H), ref.randn(2, torch.float32, T, H), ref.randn(3, torch.float32, T, K), ref.randn(4, torch.float32, T, H)
    drows, dw = torch.zeros_like(rows), torch.empty_like(w)
    moe.moe_combine_backward(dout, inv, w, rows, drows, dw)

    def loss(r, v):
        return float((ref.gather(r, inv, v, T)[0] * dout.double()).sum())

    vr, vw, h = ref.randn(5, torch.float64, T * K, H), ref.randn(6, torch.float64, T, K), 1e-3
    diff = (loss(rows.double() + h * vr, w) - loss(rows.double() - h * vr, w)) / (2 * h)
    assert abs(diff - float((drows.double() * vr).sum())) <= 1e-6 * float((drows.double() * vr).abs().sum())
    diff = (loss(rows, w.double() + h * vw) - loss(rows, w.double() - h * vw)) / (2 * h)
    assert abs(diff - float((dw.double() * vw).sum())) <= 1e-5 * float((ref.dots(dout, rows, inv, T)[1] * vw.abs()).sum())
    del x


def test_places_out_of_range_count_as_dropped():
    T, K, H = 4, 2, 64
    inv = torch.tensor([0, 1, 8, 2 ** 31 - 1, -5, 3, 2, -2 ** 31], dtype=torch.int32, device="cuda")
    x, rows = ref.randn(1, torch.bfloat16, T, H), ref.randn(2, torch.bfloat16, T * K, H)
    fixed = torch.where((inv >= 0) & (inv < T * K), inv, -1)
    out, want = torch.empty_like(x), torch.empty_like(x)
    moe.moe_combine(rows, inv, None, None, out)
    moe.moe_combine(rows, fixed, None, None, want)
    assert torch.equal(out, want)
    a, b = torch.zeros_like(rows), torch.zeros_like(rows)
    moe.moe_dispatch(x, inv, None, a)
    moe.moe_dispatch(x, fixed, None, b)
    assert torch.equal(a, b)


def test_long_rows_pass_32_bits():
    """Row offsets beyond 2^31 elements."""
    T, K, H = 40000, 8, 8192
    inv = torch.arange(T * K, dtype=torch.int32, device="cuda").flip(0).contiguous()
    x = ref.randn(1, torch.bfloat16, T, H)
    rows = torch.empty(T * K, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch(x, inv, None, rows)
    assert torch.equal(rows, x.repeat_interleave(K, 0).flip(0))
    out = torch.empty_like(x)
    moe.moe_combine(rows, inv, torch.full((T, K), 0.125, device="cuda"), None, out)
    assert torch.equal(out, x)


def test_empty():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.empty(0, dtype=torch.int32, device="cuda")
    moe.moe_dispatch(z, inv, None, z)
    moe.moe_combine(z, inv, None, None, z)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [520, 77])
def test_a_large_residual_costs_one_rounding(dtype, H):
    """Rows are added up at their own size and the residual last: its size is rounded to once. (K products and sums of the rows: 2 K
    roundings of their magnitudes in fp32; then the sum with the residual, rounded in fp32, and to the type.)"""
    T, K = 300, 8
    inv = ref.sort_gpu(make_ids(1, T, 16, K, 0.1), 16)[3]
    rows, w = ref.randn(2, dtype, T * K, H), torch.softmax(ref.randn(3, torch.float32, T, K), 1)
    res = (4096 + 512 * ref.randn(4, torch.float32, T, H)).to(dtype)
    out = torch.empty_like(res)
    moe.moe_combine(rows, inv, w, res, out)
    s, mag = ref.gather(rows, inv, w, T)
    want = s + res.double()
    last = 0.0 if dtype == torch.float32 else ref.unit(dtype) * (1 + ref.U32)
    off, bound = (out.double() - want).abs(), (ref.U32 * (1 + last) + last) * want.abs() + 2 * (2 * K + 1) * ref.U32 * mag
    assert not bool((~(off <= bound)).any()), float((off / bound).max())


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_without_slots_keep_their_residual(dtype):
    """Bit for bit, a negative zero among them; without a residual they are zeros."""
    T, K, H = 5, 3, 24
    inv = torch.full((T * K,), -1, dtype=torch.int32, device="cuda")
    rows, res = ref.randn(1, dtype, T * K, H), ref.randn(2, dtype, T, H)
    res[:, ::3] = -0.0
    out = torch.empty_like(res)
    for w in (None, torch.rand(T, K, device="cuda")):
        moe.moe_combine(rows, inv, w, res, out)
        assert torch.equal(out.view(torch.uint8), res.view(torch.uint8))
        moe.moe_combine(rows, inv, w, None, out)
        assert not bool(out.view(torch.uint8).any())


@pytest.mark.parametrize("K", [1, 8])
def test_no_tokens_with_pairs_by_token(K):
    """An empty batch of a router's own tensors [0, K]: nothing to do in any direction."""
    z, inv, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, K, dtype=torch.int32, device="cuda"), torch.empty(0, K, device="cuda")
    moe.moe_dispatch(z, inv, w, z)
    moe.moe_combine(z, inv.view(-1), w, z, z)
    moe.moe_dispatch_backward(z, inv, w, z, z, w)
    moe.moe_combine_backward(z, inv.view(-1), None, z, z, w)
