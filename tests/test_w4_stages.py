"""The bounds of w4_stages.py: an honest computation of each stage keeps them, and a wrong one does not."""
from __future__ import annotations

import pytest
import torch

from tests import w4_reference as ref
from tests import w4_stages as st

DIMS = [(40, 512, 6, 3, 128, 192), (30, 2048, 4, 2, 512, 64)]


def bf16(t):
    return t.float().to(torch.bfloat16)


class Honest:
    """Each stage in fp32 with the roundings that the kernels make."""

    def __init__(self, dims, name="int4", group=64, rounded=True):
        T, H, E, K, I, Is = self.dims = dims
        self.rounded = rounded
        g = torch.Generator().manual_seed(sum(dims))
        self.m = {k: ref.matrices(name, group, n, r, c, seed=n + r + c, device="cpu")
                  for k, n, r, c in (("gu", E, 2 * I, H), ("dn", E, H, I), ("sgu", 1, 2 * Is, H), ("sdn", 1, H, Is))}
        self.w = {k: st.weights(name, group, m, rounded) for k, m in self.m.items()}
        self.x = bf16(torch.randn(T, H, generator=g))
        self.residual = bf16(torch.randn(T, H, generator=g))
        router, gate = bf16(torch.randn(E, H, generator=g) * 0.02), bf16(torch.randn(1, H, generator=g) / H ** 0.5)
        ids, w, sg = st.routing(self.x, router, None, gate, K)
        self.ids, self.topw, self.sgate = ids, w.float(), sg.float()
        pair, x = st.dispatch(ids), self.x.float()
        expert = ids.reshape(-1)[pair]
        self.h = torch.zeros(T * K + T, max(I, Is), dtype=torch.bfloat16)
        self.Y = torch.zeros(T, K + 1, H)
        for p in range(T * K):
            s = self.w["gu"][expert[p]].float() @ x[pair[p] // K]
            self.h[p, :I] = bf16(torch.nn.functional.silu(s[:I]) * s[I:])
            self.Y[pair[p] // K, pair[p] % K] = (self.w["dn"][expert[p]].float() @ self.h[p, :I].float()) * self.topw.reshape(-1)[pair[p]]
        s = x @ self.w["sgu"][0].float().T
        self.h[T * K:, :Is] = bf16(torch.nn.functional.silu(s[:, :Is]) * s[:, Is:])
        self.Y[:, K] = (self.h[T * K:, :Is].float() @ self.w["sdn"][0].float().T) * self.sgate[:, None]
        self.half = ref.HALF if rounded else 0.0
        if rounded:
            self.Y = bf16(self.Y)
        self.out = bf16(self.residual.float() + self.Y.float().sum(1))


@pytest.fixture(scope="module", params=[(d, r) for d in DIMS for r in (True, False)], ids=str)
def honest(request):
    return Honest(request.param[0], rounded=request.param[1])


def within(got, want, bound):
    """Share of the values that are compared and lie within the bound."""
    live = ~want.isnan()
    return float(((got.double() - want).abs() <= bound)[live].double().mean())


def test_honest_stages_keep_the_bounds(honest):
    o = honest
    assert within(o.h, *st.activations(o.dims, o.x, o.ids, o.w["gu"], o.w["sgu"][0])) == 1.0
    assert within(o.Y, *st.outputs(o.dims, o.h, o.ids, o.topw, o.sgate, o.w["dn"], o.w["sdn"][0], o.half)) == 1.0
    assert within(o.out, *st.combined(o.Y, o.residual)) == 1.0


@pytest.mark.parametrize("mistake", ["another token", "another expert", "gate and up swapped", "sign", "another group's scale"])
def test_wrong_activations_are_rejected(honest, mistake):
    o = honest
    x, ids, gu, sgu = o.x, o.ids, o.w["gu"], o.w["sgu"][0]
    if mistake == "another token":
        x = x.roll(1, 0)
    elif mistake == "another expert":
        gu, sgu = gu.roll(1, 0), sgu.flip(0)
    elif mistake == "gate and up swapped":
        gu, sgu = gu.roll(gu.shape[1] // 2, 1), sgu.roll(sgu.shape[0] // 2, 0)
    elif mistake == "sign":
        gu, sgu = -gu, -sgu
    else:
        gu, sgu = (st.weights("int4", 64, (c, s.roll(1, 2), z), o.rounded) for c, s, z in (o.m["gu"], o.m["sgu"]))
        sgu = sgu[0]
    assert within(o.h, *st.activations(o.dims, x, ids, gu, sgu)) < 0.1


@pytest.mark.parametrize("mistake", ["another row of h", "another expert", "another token's weights", "the next slot", "sign", "nothing"])
def test_wrong_outputs_are_rejected(honest, mistake):
    o = honest
    T, H, E, K, I, Is = o.dims
    h, ids, w, g, dn, sdn, Y = o.h, o.ids, o.topw, o.sgate, o.w["dn"], o.w["sdn"][0], o.Y
    if mistake == "another row of h":
        h = torch.cat([h[:T * K].roll(1, 0), h[T * K:].roll(1, 0)])
    elif mistake == "another expert":
        dn, sdn = dn.roll(1, 0), sdn.flip(0)
    elif mistake == "another token's weights":
        w, g = w.roll(1, 0), g.roll(1, 0)
    elif mistake == "the next slot":
        Y = Y.roll(1, 1)
    elif mistake == "sign":
        dn, sdn = -dn, -sdn
    else:
        Y = torch.zeros_like(Y)
    assert within(Y, *st.outputs(o.dims, h, ids, w, g, dn, sdn, o.half)) < 0.25  # (weights of two tokens can be near one another)


@pytest.mark.parametrize("mistake", ["residual alone", "a slot dropped", "no shared expert", "another token", "no residual"])
def test_wrong_sums_are_rejected(honest, mistake):
    o = honest
    Y, r = o.Y.clone(), o.residual
    if mistake == "residual alone":
        Y[:] = 0
    elif mistake == "a slot dropped":
        Y[:, 1] = 0
    elif mistake == "no shared expert":
        Y[:, -1] = 0
    elif mistake == "another token":
        Y = Y.roll(1, 0)
    else:
        r = None
    assert within(o.out, *st.combined(Y, r)) < 0.25


def test_weights_round_once():
    """s * v through fp32 is exact, so its rounding to bf16 is the one that the tensor-core path makes."""
    for name in ref.FORMATS:
        m = ref.matrices(name, 32, 1, 16, 128, seed=1, device="cpu")
        exact = ref.values(name, 32, m)
        assert torch.equal(exact, exact.float().double())
        off = (st.weights(name, 32, m, True) - exact).abs()
        assert bool((off <= ref.HALF * exact.abs()).all()) and (name == "e2m1" or bool((off > 0).any()))
