"""Plain 64-bit forms of the layer's parts, and the bounds their tests use.

A result is rounded once from fp32: at most half a step, u = finfo.eps / 2, relative to its value. Before that the
kernels work in fp32. For a sum of n products, whatever its order, the error is at most n * 2^-24 * (the sum of the
products' magnitudes) to first order; `sums` below is that magnitude, formed in 64 bits from absolute values, and
n is doubled to cover the second-order terms and the few fp32 operations around the sum. Functions (exp, erfc, rsqrt) are
good to a few units in the last place of fp32: FN units of 2^-24 are allowed for each, relative to the magnitudes they scale.
"""
from __future__ import annotations

import math

import torch

import sparse_moe_ffn_router_gb300 as moe

TYPES = {moe.BF16: torch.bfloat16, moe.FP16: torch.float16, moe.FP32: torch.float32}
U32 = 2.0 ** -24
FN = 16


def unit(dtype) -> float:
    """Half a step of a type, and its smallest step (what a value below the normal range is rounded to)."""
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def check(got, want, magnitude, n, what=""):
    """|got - want| <= one rounding of want + 2 n fp32 roundings of the magnitude."""
    got64 = got.double()
    bound = (unit(got.dtype) if got.dtype != torch.float32 else 0.0) * want.abs() + (2 * n + FN) * U32 * magnitude * (1 + unit(got.dtype)) + smallest(got.dtype)
    off = (got64 - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound).max()):.2f} x the bound"


def randn(seed, dtype, *shape, scale=1.0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=device) * scale).to(dtype)


# ---------------------------------------------------------------------------------------- exchange

def sort(ids, E):
    """counts, offsets, perm, inv by a plain walk over the pairs."""
    flat = ids.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for p, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(p)
    counts = [len(v) for v in lists]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    perm = [p for v in lists for p in v]
    inv = [-1] * len(flat)
    for i, p in enumerate(perm):
        inv[p] = i
    perm += [-1] * (len(flat) - len(perm))
    return [torch.tensor(v, dtype=torch.int32) for v in (counts, offsets, perm, inv)]


def sort_gpu(ids, E):
    T, K = ids.shape
    out = [torch.full((n,), -7, dtype=torch.int32, device=ids.device) for n in (E, E + 1, T * K, T * K)]
    moe.moe_sort_pairs(E, ids, *out)
    return out


def spread(tok, inv, w, rows):
    """rows with rows[inv[p]] = w[p] * tok[t] in 64 bits."""
    T, H = tok.shape
    K = inv.numel() // max(T, 1)
    out = rows.double().clone()
    live = inv >= 0
    src = tok.double().repeat_interleave(K, 0) * (1.0 if w is None else w.double().reshape(-1, 1))
    out[inv[live].long()] = src[live]
    return out


def gather(rows, inv, w, T):
    """(sum_k w rows[inv], the same of magnitudes) in 64 bits."""
    K, H = inv.numel() // T, rows.shape[1]
    r = torch.where((inv >= 0)[:, None], rows.double()[inv.clamp(min=0).long()], 0.0).view(T, K, H)
    r = r if w is None else r * w.double()[:, :, None]
    return r.sum(1), r.abs().sum(1)


def dots(tok, rows, inv, T):
    K = inv.numel() // T
    r = torch.where((inv >= 0)[:, None], rows.double()[inv.clamp(min=0).long()], 0.0).view(T, K, -1)
    p = r * tok.double()[:, None]
    return p.sum(2), p.abs().sum(2)


# ---------------------------------------------------------------------------------------- linear

def act(name, z):
    if name == moe.ACT_RELU:
        return z.clamp(min=0)
    if name == moe.ACT_SILU:
        return z * torch.sigmoid(z)
    if name == moe.ACT_GELU:
        return z * torch.special.ndtr(z)
    if name == moe.ACT_SIGMOID:
        return torch.sigmoid(z)
    if name == moe.ACT_SWIGLU:
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z


def experts(T, E, offsets):
    """Rows of each expert as (first, last + 1)."""
    if offsets is None:
        return [(0, T)]
    o = offsets.tolist()
    return [(o[e], o[e + 1]) for e in range(E)]


def linear(d, x, w, bias, offsets, residual):
    """(out, z, magnitude of out's error, magnitude of z's) in 64 bits; rows of no expert are zero."""
    wide = d.N // 2 if d.act == moe.ACT_SWIGLU else d.N
    out, z, mz = (torch.zeros(d.T, n, dtype=torch.float64, device=x.device) for n in (wide, d.N, d.N))
    for e, (a, b) in enumerate(experts(d.T, d.E, offsets)):
        z[a:b] = x[a:b].double() @ w[e].double().T
        mz[a:b] = x[a:b].double().abs() @ w[e].double().abs().T
        if bias is not None:
            z[a:b] += bias[e].double()
            mz[a:b] += bias[e].double().abs()
        out[a:b] = act(d.act, z[a:b])
    # an error of z passes through act with its slope (at most 1.13); swiglu's gate and up each scale the other's
    if d.act == moe.ACT_SWIGLU:
        g, u = z.chunk(2, -1)
        mg, mu = mz.chunk(2, -1)
        mo = 1.13 * mg * u.abs() + mu * (g * torch.sigmoid(g)).abs() + out.abs()
    else:
        mo = 1.13 * mz + out.abs()
    if residual is not None:
        out = out + residual.double()
        mo = mo + residual.double().abs()
    return out, z, mo, mz


def linear_backward(d, x, w, offsets, z, dout):
    """(dx, dw, db) in 64 bits and the bound of each. The kernel's dz is off by at most e = half a step of |dz| (it is rounded to the
    type) + FN * 2^-24 * |dout| * m before that, m over the magnitudes of the slope's terms: a slope is a sum of products of
    numbers below 1 with 1, z and the other half's z, each formed in a few fp32 operations. The products carry e on as a sum of
    magnitudes, and add 2 n fp32 roundings of theirs."""
    dz, m = dout.double(), torch.zeros(())
    if d.act != moe.ACT_NONE:
        zz = z.double().requires_grad_()
        dz, = torch.autograd.grad(act(d.act, zz), zz, dz)
        za = z.double().abs()
        if d.act == moe.ACT_SWIGLU:
            g, u = za.chunk(2, -1)
            m = torch.cat([dout.double().abs() * u * (2 + g), dout.double().abs() * (1 + g)], 1)
        else:
            m = dout.double().abs() * (2 + za)
    e32 = FN * U32 * m if d.act != moe.ACT_NONE else torch.zeros_like(dz)
    e = e32 + (unit(x.dtype) * dz.abs() + smallest(x.dtype) if d.act != moe.ACT_NONE else 0.0)
    res = [torch.zeros(d.T, d.K, dtype=torch.float64, device=x.device), torch.zeros(d.E, d.N, d.K, dtype=torch.float64, device=x.device),
           torch.zeros(d.E, d.N, dtype=torch.float64, device=x.device)]
    bounds = [torch.zeros_like(t) for t in res]
    for i, (a, b) in enumerate(experts(d.T, d.E, offsets)):
        xe, we, n = x[a:b].double(), w[i].double(), b - a
        res[0][a:b] = dz[a:b] @ we
        bounds[0][a:b] = (e[a:b] + 2 * d.N * U32 * dz[a:b].abs()) @ we.abs()
        res[1][i] = dz[a:b].T @ xe
        bounds[1][i] = (e[a:b] + 2 * n * U32 * dz[a:b].abs()).T @ xe.abs()
        res[2][i] = dz[a:b].sum(0)
        bounds[2][i] = (e32[a:b] + 2 * n * U32 * dz[a:b].abs()).sum(0)
    u = unit(x.dtype)
    return res, [(1 + u) * v + u * r.abs() + smallest(x.dtype) for r, v in zip(res, bounds)]


# ---------------------------------------------------------------------------------------- norm

def norm(v, gamma, eps):
    return v / (v.square().mean(1, keepdim=True) + eps).sqrt() * (1.0 if gamma is None else gamma)


def gate_of(d, gate):
    if gate is None:
        return 1.0
    g = gate[:, None] if d.gate == moe.GATE_TOKEN else gate
    return g if d.gate_act == moe.ACT_NONE else torch.sigmoid(g) * (g if d.gate_act == moe.ACT_SILU else 1.0)


def norm_forward(d, y, residual, gate, gp, gq):
    """s, xn in 64 bits, differentiable."""
    n = norm(y, gp, d.eps) if d.flags & moe.NORM_POST else y
    s = d.branch_scale * gate_of(d, gate) * n
    if residual is not None:
        s = s + d.residual_scale * residual
    return s, norm(s, gq, d.eps)


assert math.isclose(unit(torch.bfloat16), 2 ** -8) and math.isclose(unit(torch.float16), 2 ** -11) and math.isclose(unit(torch.float32), 2 ** -24)
