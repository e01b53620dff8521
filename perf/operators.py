"""Cases of the 4-bit weight operators: quantising a bank of weights, a linear layer and the whole
sparse Mixture-of-Experts layer on 4-bit weights with group scales.

A 4-bit weight matrix [rows, cols] stands for w[n, k] = s[n, k / G] * v[n, k], G = 32, 64 or 128:
  int4     v = code - 8           (codes 0 .. 15)
  int4_zp  v = code - z[n, k / G] (codes and zero points 0 .. 15)
  e2m1     v = sign * {0, 0.5, 1, 1.5, 2, 3, 4, 6}[code & 7], sign = bit 3 of the code
with s in bf16. A program keeps its weights packed: strips of 16 rows (for a merged gate_up
matrix 8 gate rows and the 8 matching up rows), each a run of records of 128 columns:
  1024 bytes of codes   [row / 8, row % 8, t, c] 32-bit words, t, c = 0 .. 3; the word holds the
                        columns 32 c + 8 t + e, e = 0 .. 7, even e in its low half and odd e in
                        its high half, as the (e / 2)-th code of that half
  16 x (128 / G) scales [row, group], bf16
  16 x (128 / G) zero points (int4_zp only), bytes
A half's codes: int4 and int4_zp have code i in bits 4i .. 4i+3; e2m1 has the sign bits of codes
0 .. 3 in bits 15, 12, 9, 14 and the other three bits, high to low, in bits (8, 7, 6), (5, 4, 3),
(2, 1, 0), (13, 10, 11). Rows and columns past the matrix have scale 0.
"""
import math

import torch

own = False

FORMATS = ("int4", "int4_zp", "e2m1")
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


# ----------------------------------------------------------------------------------------
# the cases

def listed():
    full = dict(kind="layer", H=2048, E=256, K=8, I=512, Is=512, zipf=False)
    return [
        # the expert bank of the smallest layer, quantised and read back
        dict(name="quantize_tiny_bank", kind="quantize", format="int4", group=32, n=32, rows=256, cols=512, gate_up=True),
        # a checkpoint's down projections of odd sizes, with zero points
        dict(name="quantize_odd_zp", kind="quantize", format="int4_zp", group=64, n=5, rows=1003, cols=1344, gate_up=False),
        # the whole gate_up bank of one full-shape layer, as a program quantises it at load
        dict(name="quantize_full_bank", kind="quantize", format="e2m1", group=32, n=256, rows=1024, cols=2048, gate_up=True),
        # one token through a square projection: latency
        dict(name="linear_T1", kind="linear", format="int4", group=128, T=1, N=2048, K=2048, bias=False),
        # one token through a long projection
        dict(name="linear_T1_wide", kind="linear", format="e2m1", group=32, T=1, N=24576, K=4096, bias=True),
        # a ragged decode batch, odd output width, columns that are no whole number of tiles
        dict(name="linear_T17_odd", kind="linear", format="int4_zp", group=32, T=17, N=5003, K=1440, bias=True),
        # a prompt
        dict(name="linear_T4096", kind="linear", format="int4", group=128, T=4096, N=4096, K=2048, bias=False),
        # the smallest layer, eight tokens
        dict(name="layer_tiny_T8", kind="layer", format="int4", group=32, T=8, H=512, E=32, K=4, I=128, Is=128, zipf=False),
        # one decode token, full layer shape
        dict(full, name="layer_T1", format="int4", group=32, T=1),
        # decode batches
        dict(full, name="layer_T8", format="e2m1", group=32, T=8),
        dict(full, name="layer_T64", format="int4_zp", group=128, T=64),
        # a prompt with skewed expert load
        dict(full, name="layer_T4096_zipf", format="int4", group=64, T=4096, zipf=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("quantize", "linear", "linear", "layer", "layer", "layer"))
    c = dict(kind=kind, format=rng.choice(FORMATS), group=rng.choice((32, 64, 128)))
    if kind == "quantize":
        c["gate_up"] = rng.random() < 0.5
        rows = _log_int(rng, 16, 4096)
        c["rows"] = 16 * ((rows + 15) // 16) if c["gate_up"] else rows
        c["cols"] = c["group"] * max(1, _log_int(rng, 128, 4096) // c["group"])
        c["n"] = max(1, min(256, _log_int(rng, 1 << 18, 1 << 28) // (c["rows"] * c["cols"])))
    elif kind == "linear":
        c["T"] = _log_int(rng, 1, 4096)
        c["K"] = c["group"] * max(1, _log_int(rng, 128, 8192) // c["group"])
        c["N"] = max(1, min(_log_int(rng, 64, 16384), (4096 * 4096 * 2048) // (c["T"] * c["K"])))
        c["bias"] = rng.random() < 0.5
    else:
        c["T"] = _log_int(rng, 1, 4096)
        c["H"] = 128 * rng.randint(1, 16)
        step = max(64, c["group"])
        c["I"], c["Is"] = (step * rng.randint(1, 512 // step) for _ in range(2))
        c["E"] = _log_int(rng, 8, 256)
        c["K"] = rng.randint(1, 8)
        c["zipf"] = rng.random() < 0.3
    return c


def _pad(v, m):
    return (v + m - 1) // m * m


def _record(fmt, group):
    return 1024 + 16 * (128 // group) * (3 if fmt == "int4_zp" else 2)


def _packed_bytes(fmt, group, rows, cols):
    return (_pad(rows, 16) // 16) * (_pad(cols, 128) // 128) * _record(fmt, group)


def _stored_bytes(fmt, group, rows, cols):
    """Codes, scales and zero points of one matrix, without any padding."""
    return rows * cols // 2 + rows * (cols // group) * (3 if fmt == "int4_zp" else 2)


def work(case):
    c, f, g = case, case["format"], case["group"]
    if c["kind"] == "quantize":  # the weights in, the packed weights out, the values they stand for out
        n = c["n"] * c["rows"] * c["cols"]
        return {"bytes": 4 * n + c["n"] * _stored_bytes(f, g, c["rows"], c["cols"]), "flops": 0}
    if c["kind"] == "linear":
        b = _stored_bytes(f, g, c["N"], c["K"]) + 2 * c["T"] * (c["K"] + c["N"]) + (2 * c["N"] if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * c["T"] * c["N"] * c["K"]}
    T, H, E, K, I, Is = (c[k] for k in ("T", "H", "E", "K", "I", "Is"))
    touched = E * (1.0 - (1.0 - K / E) ** T)  # experts that T tokens reach under even routing
    expert = _stored_bytes(f, g, 2 * I, H) + _stored_bytes(f, g, H, I)
    shared = _stored_bytes(f, g, 2 * Is, H) + _stored_bytes(f, g, H, Is)
    return {"bytes": int(touched * expert + shared + 2 * (E + 1) * H + 3 * 2 * T * H),
            "flops": 2 * T * (H * (E + 1) + 3 * H * (K * I + Is))}


# ----------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _matrix(gen, fmt, group, n, rows, cols):
    """n matrices of 4-bit weights as a checkpoint holds them: codes [n, rows, cols] (one per byte),
    scales [n, rows, cols / group] bf16 and zero points (or None), for weights ~ N(0, 1 / cols)."""
    codes = torch.empty(n, rows, cols, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (rows * cols))
    groups = cols // group
    zeros = torch.randint(5, 11, (n, rows, groups), generator=gen, device=DEV, dtype=torch.uint8) if fmt == "int4_zp" else None
    mids = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=DEV)
    spread = 2.2
    for i in range(0, n, step):
        v = torch.randn(codes[i:i + step].shape, generator=gen, device=DEV) * spread
        if fmt == "e2m1":
            codes[i:i + step] = torch.bucketize(v.abs(), mids).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        else:
            z = 8.0 if zeros is None else zeros[i:i + step].float().repeat_interleave(group, 2)
            codes[i:i + step] = (v.round() + z).clamp(0, 15).to(torch.uint8)
    scales = torch.rand(n, rows, groups, generator=gen, device=DEV) * 0.5 + 0.75
    return codes, (scales / (spread * math.sqrt(cols))).to(torch.bfloat16), zeros


def _pack(fmt, group, matrix, gate_up):
    """The packed form of a checkpoint's matrices: uint8 [n, bytes of one matrix]."""
    codes, scales, zeros = matrix
    n, rows, cols = codes.shape
    R, C, per = _pad(rows, 16), _pad(cols, 128), 128 // group

    def strips(t, width, fill):
        out = torch.full((n, R, width), fill, dtype=t.dtype, device=DEV)
        out[:, :rows, :t.shape[2]] = t
        if gate_up:  # strip j: gate rows 8j .. 8j+7, then the matching up rows
            out = out.view(n, 2, R // 16, 8, width).transpose(1, 2)
        return out.reshape(n, R // 16, 16, width)

    q = strips(codes, C, 8 if fmt == "int4" else 0)
    q = q.view(n, R // 16, 2, 8, C // 128, 4, 4, 4, 2)  # strip, row / 8, row % 8, record, c, t, code of the half, half
    q = q.permute(0, 1, 4, 2, 3, 6, 5, 8, 7).to(torch.int16)  # strip, record, row / 8, row % 8, t, c, half, code
    word = torch.zeros(q.shape[:-1], dtype=torch.int16, device=DEV)
    for i in range(4):
        if fmt == "e2m1":
            at = ((8, 7, 6), (5, 4, 3), (2, 1, 0), (13, 10, 11))[i]
            word |= ((q[..., i] >> 3) & 1) << (15, 12, 9, 14)[i]
            for bit, p in zip((2, 1, 0), at):
                word |= ((q[..., i] >> bit) & 1) << p
        else:
            word |= q[..., i] << (4 * i)
    parts = [word.contiguous().view(torch.uint8).reshape(n, R // 16, C // 128, 1024)]
    for t in (scales, zeros):
        if t is not None:
            s = strips(t, C // group, 0).view(n, R // 16, 16, C // 128, per).transpose(2, 3).contiguous()
            parts.append(s.view(torch.uint8).reshape(n, R // 16, C // 128, -1))
    return torch.cat(parts, 3).reshape(n, -1)


def _inputs(case, seed):
    """The inputs in the clear: weights as a checkpoint holds them, token rows, the router."""
    c, f, g = case, case["format"], case["group"]
    gen = _gen(seed)
    if c["kind"] == "quantize":
        w = torch.empty(c["n"], c["rows"], c["cols"], dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 28) // (c["rows"] * c["cols"]))
        for i in range(0, c["n"], step):
            w[i:i + step] = torch.randn(w[i:i + step].shape, generator=gen, device=DEV) / math.sqrt(c["cols"])
        return {"w": w}
    if c["kind"] == "linear":
        s = {"w": _matrix(gen, f, g, 1, c["N"], c["K"])}
        s["x"] = torch.randn(c["T"], c["K"], generator=gen, device=DEV).to(torch.bfloat16)
        s["bias"] = torch.randn(c["N"], generator=gen, device=DEV).to(torch.bfloat16) if c["bias"] else None
        return s
    T, H, E, K, I, Is = (c[k] for k in ("T", "H", "E", "K", "I", "Is"))
    s = {"gate_up": _matrix(gen, f, g, E, 2 * I, H), "down": _matrix(gen, f, g, E, H, I),
         "shared_gate_up": _matrix(gen, f, g, 1, 2 * Is, H), "shared_down": _matrix(gen, f, g, 1, H, Is)}
    s["router_w"] = (torch.randn(E, H, generator=gen, device=DEV) * 0.02).to(torch.bfloat16)
    s["router_b"] = None
    if c["zipf"]:  # expert load skewed toward Zipf(1.1)
        rank = torch.randperm(E, generator=gen, device=DEV).double() + 1
        s["router_b"] = (-0.42 * 1.1 * torch.log(rank)).to(torch.bfloat16)
    s["shared_gate"] = (torch.randn(1, H, generator=gen, device=DEV) / math.sqrt(H)).to(torch.bfloat16)
    s["x"] = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
    s["residual"] = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
    # tokens whose K-th and next score are nearly equal have two right answers: such rows are drawn again
    for _ in range(20):
        top = _scores64(s).sort(dim=1, descending=True).values[:, :K + 1]
        close = ((top[:, :-1] - top[:, 1:]).amin(1) < 1e-4) if top.shape[1] > 1 else torch.zeros(T, dtype=torch.bool, device=DEV)
        if not bool(close.any()):
            break
        fresh = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
        s["x"] = torch.where(close[:, None], fresh, s["x"])
    return s


def _scores64(s):
    l = s["x"].double() @ s["router_w"].double().T
    return l if s["router_b"] is None else l + s["router_b"].double()


def prepare(case, seed):
    case = dict(case)
    case["K"] = min(case["K"], case["E"]) if case["kind"] == "layer" else case.get("K")
    f, g = case["format"], case["group"]
    s = _inputs(case, seed)
    s["case"] = case
    if case["kind"] == "linear":
        s["w"] = _pack(f, g, s["w"], False)[0]
    if case["kind"] == "layer":
        for name, gate_up in (("gate_up", True), ("down", False), ("shared_gate_up", True), ("shared_down", False)):
            s[name] = torch.cat([_pack(f, g, tuple(None if t is None else t[i:i + 16] for t in s[name]), gate_up)
                                 for i in range(0, s[name][0].shape[0], 16)])
        ids = _scores64(s).sort(dim=1, descending=True, stable=True).indices[:, :case["K"]]
        s["most"] = int(torch.bincount(ids.reshape(-1), minlength=case["E"]).max())  # tokens of the busiest expert
    if own:  # what a program makes once: the format, the workspace, the layer's weights as one object
        import sparse_moe_ffn_router_gb300 as moe
        s["format"] = moe.W4Format({"int4": moe.W4_INT4, "int4_zp": moe.W4_INT4_ZP, "e2m1": moe.W4_E2M1}[f], g)
        if case["kind"] == "linear":
            s["workspace"] = moe.new_w4_linear_workspace(s["format"], case["T"], case["N"], case["K"])
        if case["kind"] == "layer":
            s["dims"] = tuple(case[k] for k in ("T", "H", "E", "K", "I", "Is"))
            s["workspace"] = moe.new_workspace(s["dims"])
            s["weights"] = moe.Weights(*(s[k] for k in ("router_w", "router_b", "gate_up", "down", "shared_gate_up",
                                                        "shared_down", "shared_gate")))
        if case["kind"] == "quantize":
            s["layout"] = moe.W4_GATE_UP if case["gate_up"] else moe.W4_ROWS
    return s


# ----------------------------------------------------------------------------------------
# one pass

def run(s):
    return {"quantize": _run_quantize, "linear": _run_linear, "layer": _run_layer}[s["case"]["kind"]](s)


def _unpack(fmt, group, packed, rows, cols, gate_up):
    """Packed matrices [n, bytes] as the fp32 weights they stand for, [n, rows, cols]."""
    n, S, C, per = packed.shape[0], _pad(rows, 16) // 16, _pad(cols, 128) // 128, 128 // group
    rec = packed.view(n, S, C, _record(fmt, group))
    half = rec[..., :1024].contiguous().view(torch.int16).view(n, S, C, 2, 8, 4, 4, 2, 1)
    bit = torch.arange(4, device=packed.device, dtype=torch.int16)
    if fmt == "e2m1":
        at = torch.tensor([[8, 5, 2, 13], [7, 4, 1, 10], [6, 3, 0, 11], [15, 12, 9, 14]], device=packed.device, dtype=torch.int16)
        mag = ((half >> at[0]) & 1) * 4 + ((half >> at[1]) & 1) * 2 + ((half >> at[2]) & 1)
        v = torch.tensor(E2M1, device=packed.device)[mag.int()] * (1 - 2 * ((half >> at[3]) & 1)).float()
    else:
        v = ((half >> (4 * bit)) & 15).float()
    # strip, record, row / 8, row % 8, t, c, half, code -> strip, row, record, c, t, code, half
    v = v.permute(0, 1, 3, 4, 2, 6, 5, 8, 7).reshape(n, S, 16, C * per, group)
    tail = rec[..., 1024:1024 + 32 * per].contiguous().view(torch.bfloat16).view(n, S, C, 16, per)
    scale = tail.transpose(2, 3).reshape(n, S, 16, C * per, 1).float()
    if fmt == "int4":
        v = v - 8.0
    if fmt == "int4_zp":
        z = rec[..., 1024 + 32 * per:].reshape(n, S, C, 16, per).transpose(2, 3).reshape(n, S, 16, C * per, 1)
        v = v - z.float()
    w = (v * scale).view(n, S, 2, 8, C * 128)
    if gate_up:
        w = w.transpose(1, 2)
    return w.reshape(n, S * 16, C * 128)[:, :rows, :cols]


def _run_quantize(s):
    c, w = s["case"], s["w"]
    n, rows, cols = w.shape
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        packed = moe.new_w4(s["format"], rows, cols, n)
        moe.moe_w4_quantize(s["format"], w, packed, s["layout"])
        values = torch.empty_like(w)
        moe.moe_w4_dequantize(s["format"], packed, values, s["layout"])
        return {"values": values}
    v = w.float().view(n, rows, cols // c["group"], c["group"])
    if c["format"] == "int4_zp":
        lo, hi = v.amin(3, keepdim=True).clamp(max=0), v.amax(3, keepdim=True).clamp(min=0)
        sc = (hi / 15 - lo / 15).to(torch.bfloat16).float()
        z = torch.where(sc > 0, (-lo / sc).round().clamp(0, 15), 0.0)
        q = torch.where(sc > 0, ((v / sc).round() + z).clamp(0, 15), z) - z
    else:
        top = 7 if c["format"] == "int4" else 6
        sc = (v.abs().amax(3, keepdim=True) / top).to(torch.bfloat16).float()
        a = torch.where(sc > 0, v / sc, 0.0)
        if c["format"] == "int4":
            q = a.round().clamp(-8, 7)
        else:
            m = a.abs()  # nearest value of the format, halfway cases to the even code
            code = ((m > 0.25).int() + (m >= 0.75).int() + (m > 1.25).int() + (m >= 1.75).int() + (m > 2.5).int()
                    + (m >= 3.5).int() + (m > 5.0).int())
            q = torch.tensor(E2M1, device=w.device)[code] * a.sign()
    return {"values": (q * sc).to(torch.bfloat16).view(n, rows, cols)}


def _run_linear(s):
    c = s["case"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        out = torch.empty(c["T"], c["N"], dtype=torch.bfloat16, device=DEV)
        moe.moe_w4_linear(s["format"], s["x"], s["w"], s["bias"], out, s["workspace"])
        return {"out": out}
    w = _unpack(c["format"], c["group"], s["w"][None], c["N"], c["K"], False)[0]
    out = s["x"].float() @ w.T
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return {"out": out.to(torch.bfloat16)}


def _run_layer(s):
    c = s["case"]
    T, H, E, K, I, Is = (c[k] for k in ("T", "H", "E", "K", "I", "Is"))
    f, g = c["format"], c["group"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        moe.moe_forward_w4(s["dims"], s["format"], s["x"], s["weights"], s["residual"], out, s["workspace"])
        return {"out": out}
    x = s["x"].float()
    score = x @ s["router_w"].float().T
    if s["router_b"] is not None:
        score = score + s["router_b"].float()
    kept, ids = (t[:, :K] for t in score.sort(dim=1, descending=True, stable=True))
    weight = torch.softmax(kept, 1)
    pair = ids.reshape(-1)

    def swiglu(rows, gate_up, down, inner):
        gu = rows @ _unpack(f, g, gate_up, 2 * inner, H, True).transpose(1, 2)
        gate, up = gu.split(inner, 2)
        return (gate * torch.sigmoid(gate) * up) @ _unpack(f, g, down, H, inner, False).transpose(1, 2)

    if T * K <= E:  # few pairs: each with its own expert's weights
        y = swiglu(x.repeat_interleave(K, 0)[:, None], s["gate_up"][pair], s["down"][pair], I)[:, 0]
    else:  # the pairs of each expert side by side, padded to the busiest expert's
        order = pair.argsort(stable=True)
        count = torch.zeros(E, dtype=torch.int64, device=x.device).index_add_(0, pair, torch.ones_like(pair))
        place = torch.empty_like(pair)
        place[order] = torch.arange(T * K, device=x.device) - (count.cumsum(0) - count)[pair[order]]
        rows = torch.zeros(E, s["most"], H, device=x.device)
        rows[pair, place] = x.repeat_interleave(K, 0)
        y = swiglu(rows, s["gate_up"], s["down"], I)[pair, place]
    y = (y.view(T, K, H) * weight[:, :, None]).sum(1)
    shared = swiglu(x[None], s["shared_gate_up"], s["shared_down"], Is)[0]
    gate = torch.sigmoid(x @ s["shared_gate"].float().T)
    return {"out": (s["residual"].float() + gate * shared + y).to(torch.bfloat16)}


# ----------------------------------------------------------------------------------------
# the definition in 64 bits

def _values64(fmt, group, matrix, i):
    """Matrix i of a checkpoint's codes, scales and zero points, as the weights it stands for."""
    codes, scales, zeros = (None if t is None else t[i] for t in matrix)
    rows, cols = codes.shape
    if fmt == "e2m1":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)
        v = table[codes.long()]
    else:
        v = codes.double() - (8.0 if zeros is None else zeros.double().repeat_interleave(group, 1))
    return v * scales.double().repeat_interleave(group, 1)


def exact(case, seed):
    case = dict(case)
    f, g = case["format"], case["group"]
    if case["kind"] == "quantize":
        w = _inputs(case, seed)["w"]
        out = torch.empty(w.shape, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 25) // (case["rows"] * case["cols"]))
        for i in range(0, case["n"], step):  # nearest representable multiple of each group's scale
            v = w[i:i + step].double().unflatten(2, (-1, g))
            if f == "int4_zp":
                lo, hi = torch.clamp(v.min(3, keepdim=True)[0], max=0), torch.clamp(v.max(3, keepdim=True)[0], min=0)
                sc = ((hi - lo) / 15).float().bfloat16().double()
                grid = torch.arange(16, device=DEV, dtype=torch.float64) - torch.round(-lo / sc).clamp(0, 15)
                q = torch.minimum(torch.maximum(torch.round(v / sc), grid[..., :1]), grid[..., -1:])
            else:
                sc = (v.abs().max(3, keepdim=True)[0] / (7 if f == "int4" else 6)).float().bfloat16().double()
                q = v / sc
                if f == "int4":
                    q = torch.round(q).clamp(-8, 7)
                else:  # one mantissa bit: steps of 0.5 below 2, of 1 below 4, of 2 above
                    m = q.abs()
                    unit = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
                    q = torch.copysign((torch.round(m / unit) * unit).clamp(max=6), q)
            out[i:i + step] = torch.nan_to_num(q * sc).flatten(2)
        return {"values": out}
    if case["kind"] == "linear":
        s = _inputs(case, seed)
        out = s["x"].double() @ _values64(f, g, s["w"], 0).T
        return {"out": out if s["bias"] is None else out + s["bias"].double()}
    case["K"] = min(case["K"], case["E"])
    s = _inputs(case, seed)
    T, H, E, K, I, Is = (case[k] for k in ("T", "H", "E", "K", "I", "Is"))
    x = s["x"].double()
    p = torch.softmax(_scores64(s), 1)
    # an expert's rank: the experts ahead of it, equal ones with a lower index among them
    rank = torch.empty(T, E, dtype=torch.int64, device=DEV)
    rank.scatter_(1, p.sort(dim=1, descending=True, stable=True).indices, torch.arange(E, device=DEV).expand(T, E))
    p = torch.where(rank < K, p, 0.0)
    p = p / p.sum(1, keepdim=True)
    out = s["residual"].double()

    def expert(rows, gate_up, down, i, inner):
        gu = rows @ _values64(f, g, gate_up, i).T
        h = gu[:, :inner] / (1 + torch.exp(-gu[:, :inner])) * gu[:, inner:]
        return h @ _values64(f, g, down, i).T

    out = out + torch.sigmoid(x @ s["shared_gate"].double().T) * expert(x, s["shared_gate_up"], s["shared_down"], 0, Is)
    for e in range(E):
        rows = torch.nonzero(rank[:, e] < K)[:, 0]
        if rows.numel():
            out[rows] += p[rows, e][:, None] * expert(x[rows], s["gate_up"], s["down"], e, I)
    return {"out": out}
