"""Plain 64-bit forms of the operators on 4-bit weights, and the error bounds their results must keep.

Matrices are held as a checkpoint holds them: codes [n, rows, cols] (one per byte), scales
[n, rows, cols / G] bf16, zero points [n, rows, cols / G] or None."""
from __future__ import annotations

import torch

import sparse_moe_ffn_router_gb300 as moe

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
FORMATS = {"int4": moe.W4_INT4, "int4_zp": moe.W4_INT4_ZP, "e2m1": moe.W4_E2M1}
HALF = 2.0 ** -8  # half a step of bf16, relative


def fmt(name: str, group: int) -> moe.W4Format:
    return moe.W4Format(FORMATS[name], group)


def matrices(name, group, n, rows, cols, seed, device="cuda", scale=None):
    """Random codes over the whole range, scales within a factor of two, all zero points 0 .. 15."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    codes = torch.randint(0, 16, (n, rows, cols), generator=g, dtype=torch.uint8)
    s = (torch.rand(n, rows, cols // group, generator=g) + 0.5) * (scale if scale else 0.25 / cols ** 0.5)
    z = torch.randint(0, 16, (n, rows, cols // group), generator=g, dtype=torch.uint8) if name == "int4_zp" else None
    return codes.to(device), s.to(torch.bfloat16).to(device), None if z is None else z.to(device)


def values(name, group, m):
    """The weights [n, rows, cols] in 64 bits."""
    codes, scales, zeros = m
    if name == "e2m1":
        v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=codes.device)[codes.long()]
    else:
        v = codes.double() - (8.0 if zeros is None else zeros.double().repeat_interleave(group, 2))
    return v * scales.double().repeat_interleave(group, 2)


def pack(name, group, m, layout=moe.W4_ROWS):
    """The packed form, made by moe_w4_pack from two codes to a byte."""
    codes, scales, zeros = m
    n, rows, cols = codes.shape
    out = moe.new_w4(fmt(name, group), rows, cols, n, device=codes.device)
    moe.moe_w4_pack(fmt(name, group), (codes[..., ::2] | (codes[..., 1::2] << 4)).contiguous(), scales, zeros, out, layout)
    return out


def sum_error(cols: int) -> float:
    """Bound of an fp32 sum of `cols` products relative to the sum of their magnitudes: products of
    bf16 values are exact; one MMA adds 16 of them to the running sum (one rounding or truncation,
    at most 2^-22 of the magnitudes so far), each group of at least 32 columns one scaled addition,
    and up to 8 shares of the columns are added at the end."""
    return (cols / 16 + cols / 32 + 8) * 2.0 ** -22


GEMM_TOKENS = 64  # the linear layer rounds its weights to bf16 at most from here on in matrices of a few thousand rows


def linear_rounds(T, N, sms):
    """Whether the linear layer takes the tensor-core path, which rounds each weight once to bf16."""
    waves = -(-(-(-N // 256) * -(-T // 128)) // sms)
    return -(-N // 16) * -(-T // 8) > 14 * sms * waves


def linear(x, w, bias, rounded=False):
    """x . w^T + bias and the bound of a correct result's error. w in 64 bits. rounded: the tensor-core
    path, which rounds each weight w to bf16 once, at most HALF |w| off: HALF sum |x w| on the sum. The
    error of the sum before the last rounding is itself rounded with it: (1 + HALF)."""
    x = x.double()
    ref = x @ w.T + (0.0 if bias is None else bias.double())
    before = (sum_error(w.shape[1]) + (HALF if rounded else 0.0)) * (x.abs() @ w.abs().T)
    return ref, HALF * ref.abs() + (1 + HALF) * before + 1e-30


def layer(dims, x, router_w, router_b, shared_gate, gu, dn, sgu, sdn, residual, ids=None, weight_half=0.0, y_half=0.0,
          score_error=5e-4):
    """The layer in 64 bits and the bound of a correct result's error. gu [E, 2I, H], dn [E, H, I],
    sgu [2Is, H], sdn [H, Is] in 64 bits. Roundings counted: h to bf16, the result to bf16, the
    routing weights (score_error, absolute), and, on the tensor-core path, each weight (weight_half)
    and each slot's output (y_half) to bf16."""
    T, H, E, K, I, Is = dims[:6]
    x = x.double()
    score = x @ router_w.double().T + (0.0 if router_b is None else router_b.double())
    if ids is None:
        ids = score.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = torch.softmax(score.gather(1, ids.long()), 1)
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)

    def expert(rows, g_u, d, inner):
        ax = rows.abs()
        s = rows @ g_u.T
        e = (sum_error(H) + weight_half) * (ax @ g_u.abs().T)
        g, u, eg, eu = s[:, :inner], s[:, inner:], e[:, :inner], e[:, inner:]
        act = g * torch.sigmoid(g)
        h = act * u
        # |d silu| <= 1.1; expf and the division add at most a few 2^-22 relative
        eh = 1.1 * eg * (u.abs() + eu) + act.abs() * eu + (HALF + 2.0 ** -19) * h.abs()
        ad = d.abs()
        return h @ d.T, eh @ ad.T + (sum_error(inner) + weight_half) * ((h.abs() + eh) @ ad.T)

    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        y, ey = expert(x[t], gu[e], dn[e], I)
        wk = w[t, k][:, None]
        out.index_add_(0, t, wk * y)
        err.index_add_(0, t, wk * ey + (score_error + y_half * wk) * (y.abs() + ey))
    y, ey = expert(x, sgu, sdn, Is)
    gate = torch.sigmoid(x @ shared_gate.double().T)
    out += gate * y
    err += gate * ey + (score_error + y_half * gate) * (y.abs() + ey)
    if residual is not None:
        out += residual.double()
    return out, err + HALF * (out.abs() + err) + 1e-30


def quantize(name, group, w):
    """Codes and scales by the definition in moe.h; w [n, rows, cols] fp32, finite. The scale's
    divisions are the fp32 ones of the definition."""
    n, rows, cols = w.shape
    v = w.float().view(n, rows, cols // group, group)
    zeros = None
    if name == "int4_zp":
        hi, lo = v.amax(3).clamp(min=0), v.amin(3).clamp(max=0)
        s = (hi / 15 - lo / 15).to(torch.bfloat16)
        d = s.float()
        zeros = torch.where(d > 0, (-lo / d).round().clamp(max=15), 0.0)
        q = torch.where(d[..., None] > 0, ((v / d[..., None]).round() + zeros[..., None]).clamp(0, 15), zeros[..., None])
        zeros = zeros.to(torch.uint8)
        codes = q.to(torch.uint8)
    else:
        s = (v.abs().amax(3) / (7 if name == "int4" else 6)).to(torch.bfloat16)
        d = s.float()[..., None]
        q = torch.where(d > 0, v / d, 0.0)
        if name == "int4":
            codes = (q.round().clamp(-8, 7) + 8).to(torch.uint8)
        else:
            table = torch.tensor(E2M1, device=w.device)
            dist = (q.abs()[..., None] - table).abs()
            near = dist == dist.amin(-1, keepdim=True)
            even = torch.arange(8, device=w.device) % 2 == 0
            pick = torch.where((near & even).any(-1), (near & even).int().argmax(-1), near.int().argmax(-1))
            codes = (pick + 8 * (q < 0)).to(torch.uint8)
    return codes.view(n, rows, cols), s, zeros
