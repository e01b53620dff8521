"""The 4-bit layer stage by stage, in 64 bits: each stage from the values that the stage before left in the
workspace, with the bound of a correct result's error. An error does not pass through several stages, so a bound
is little more than the stage's own last rounding, and a wrong token, slot, expert or scale is far outside it.

The weights are those that the path multiplies by: s * v, or s * v rounded once to bf16 (rounded). s * v has at most
16 bits, so the conversion through fp32 rounds once."""
from __future__ import annotations

import torch

from tests import w4_reference as ref

HALF = ref.HALF
SILU = 2.0 ** -16  # relative: exponential and division, at most ~100 fp32 steps
TINY = 1e-30


def weights(name, group, m, rounded):
    v = ref.values(name, group, m)
    return v.float().to(torch.bfloat16).double() if rounded else v


def dispatch(ids):
    """Pairs (t * K + k) by expert, tokens ascending within one."""
    return ids.long().reshape(-1).argsort(stable=True)


def routing(x, router_w, router_b, shared_gate, K):
    """Experts, their weights and the shared expert's gate of each token."""
    x = x.double()
    score = x @ router_w.double().T + (0.0 if router_b is None else router_b.double())
    top = score.sort(dim=1, descending=True, stable=True)
    return top.indices[:, :K], torch.softmax(top.values[:, :K], 1), torch.sigmoid(x @ shared_gate.double().T)[:, 0]


def gated(x, gu):
    """silu(x . gate) * (x . up), rounded to bf16. gu [2I, H]."""
    x, inner = x.double(), gu.shape[0] // 2
    s, e = x @ gu.T, ref.sum_error(gu.shape[1]) * (x.abs() @ gu.abs().T)
    g, u, eg, eu = s[:, :inner], s[:, inner:], e[:, :inner], e[:, inner:]
    act = g * torch.sigmoid(g)
    h = act * u
    # |d silu| <= 1.1; the last rounding is of the value with its error
    before = 1.1 * eg * (u.abs() + eu) + act.abs() * eu + SILU * h.abs()
    return h, before + HALF * (h.abs() + before) + TINY


def slot(h, d, scale, y_half):
    """scale * (h . d^T), in fp32 (y_half 0) or rounded to bf16 (y_half HALF). d [H, I], scale a row."""
    h, scale = h.double(), scale.double()[:, None]
    y, before = scale * (h @ d.T), ref.sum_error(d.shape[1]) * scale.abs() * (h.abs() @ d.abs().T)
    before = before + 2.0 ** -23 * y.abs()  # the product with the scale
    return y, before + y_half * (y.abs() + before) + TINY


def combined(Y, residual):
    """The residual and the slots of Y [T, K + 1, H], added in fp32 and rounded to bf16."""
    y = Y.double()
    r = torch.zeros_like(y[:, 0]) if residual is None else residual.double()
    out, size = r + y.sum(1), r.abs() + y.abs().sum(1)
    before = y.shape[1] * 2.0 ** -24 * size
    return out, before + HALF * (out.abs() + before) + TINY


def activations(dims, x, ids, gu, sgu):
    """h [P + T, max(I, Is)] and its bound: routed rows in dispatch order, then the shared expert's; columns past a row's
    own are NaN. gu [E, 2I, H], sgu [2Is, H]."""
    T, H, E, K, I, Is = dims[:6]
    want = torch.full((T * K + T, max(I, Is)), float("nan"), dtype=torch.float64, device=x.device)
    bound = want.clone()
    pair = dispatch(ids)
    expert = ids.long().reshape(-1)[pair]
    for e in range(E):
        p = torch.nonzero(expert == e)[:, 0]
        if p.numel():
            want[p, :I], bound[p, :I] = gated(x[pair[p] // K], gu[e])
    want[T * K:, :Is], bound[T * K:, :Is] = gated(x, sgu)
    return want, bound


def outputs(dims, h, ids, topw, sgate, dn, sdn, y_half):
    """Y [T, K + 1, H] and its bound, from the h rows. dn [E, H, I], sdn [H, Is]."""
    T, H, E, K, I, Is = dims[:6]
    want = torch.empty(T, K + 1, H, dtype=torch.float64, device=h.device)
    bound = torch.empty_like(want)
    pair = dispatch(ids)
    expert = ids.long().reshape(-1)[pair]
    for e in range(E):
        p = torch.nonzero(expert == e)[:, 0]
        if p.numel():
            at = pair[p]
            want[at // K, at % K], bound[at // K, at % K] = slot(h[p, :I], dn[e], topw.reshape(-1)[at], y_half)
    want[:, K], bound[:, K] = slot(h[T * K:, :Is], sdn, sgate, y_half)
    return want, bound
