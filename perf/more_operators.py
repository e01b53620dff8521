"""Cases of the operators around the sparse Mixture-of-Experts layer when it is trained or put together
from parts: tokens sorted by expert and back with their weights, linear layers with bias, activation
and residual (one matrix, or one for each expert's rows), and the norms before and after a block
with its gate and residual scale; each with its gradient.

  sort      pairs (t, k), t * top + k, ordered by ids[t, k], stable; a slot whose id is no expert is dropped
  dispatch  rows[inv[t, k]] = (w[t, k]) * x[t]
  combine   out[t] = residual[t] + sum_k w[t, k] * rows[inv[t, k]]
  linear    out = act(x . W_e^T + b_e) + residual, e the expert whose rows [offsets[e], offsets[e + 1]) hold x's row
            act: none, relu, silu, gelu (z * Phi(z)), swiglu (W's first half gate, second half up: silu(g) * u)
  norm      s = c * residual + a * gate * N(y; gamma_post), xn = N(s; gamma_pre), N(v; g) = v / sqrt(mean(v^2) + eps) * g
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTS = ("none", "relu", "silu", "gelu", "swiglu")
EPS = 1e-6


# ----------------------------------------------------------------------------------------
# the cases

def listed():
    exchange = dict(E=256, top=8, H=2048, dtype="bf16", weights=False, residual=False, drop=False, skew=False)
    norm = dict(H=2048, dtype="bf16", gate="none", gate_act="none", post=True, branch=1.0, keep=1.0)
    linear = dict(kind="linear", E=0, top=0, dtype="bf16", bias=False, residual=False, keep=False, skew=False)
    return [
        # one decode token on its way to its experts: latency
        dict(exchange, name="dispatch_T1", kind="dispatch", T=1),
        # a prompt, expert load skewed
        dict(exchange, name="dispatch_T4096", kind="dispatch", T=4096, skew=True),
        # a ragged batch in fp32 with dropped slots and an odd row width, back into its residual
        dict(exchange, name="combine_T1003_odd", kind="combine", T=1003, E=60, top=6, H=1541, dtype="fp32",
             weights=True, residual=True, drop=True),
        # a training batch: gradients of the experts' rows and of the routing weights
        dict(exchange, name="combine_backward_T4096", kind="combine_backward", T=4096, weights=True),
        # between two blocks of one decode token: latency
        dict(norm, name="norm_T1", kind="norm", T=1),
        # between two blocks of a prompt, the branch gated element by element
        dict(norm, name="norm_T4096_gated", kind="norm", T=4096, gate="full", gate_act="sigmoid"),
        # a training batch of odd sizes, learned gate for each channel
        dict(norm, name="norm_backward_T2051_odd", kind="norm_backward", T=2051, H=1544, gate="channel", branch=0.5, keep=0.75),
        # one token through a square projection into its residual: latency
        dict(linear, name="linear_T1", T=1, N=2048, K=2048, act="none", residual=True),
        # a prompt through a wide projection
        dict(linear, name="linear_T4096_gelu", T=4096, N=8192, K=2048, act="gelu", bias=True),
        # a training step of a projection of odd sizes in fp16
        dict(linear, name="linear_backward_T1021_odd", kind="linear_backward", T=1021, N=1003, K=1544, act="silu", dtype="fp16", bias=True),
        # a decode batch through its experts' gate_up products
        dict(linear, name="experts_T64", T=64, E=256, top=8, N=1024, K=2048, act="swiglu"),
        # a training step of the experts' gate_up products, expert load skewed
        dict(linear, name="experts_backward_T4096", kind="linear_backward", T=4096, E=256, top=8, N=1024, K=2048, act="swiglu", skew=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("dispatch", "dispatch_backward", "combine", "combine_backward", "norm", "norm", "norm_backward", "norm_backward",
                       "linear", "linear", "linear_backward", "linear_backward", "experts", "experts", "experts_backward"))
    c = dict(kind=kind, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")))
    if kind in ("dispatch", "dispatch_backward", "combine", "combine_backward"):
        c["E"] = _log_int(rng, 2, 256)
        c["top"] = rng.randint(1, min(8, c["E"]))
        c["H"] = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            c["H"] = (c["H"] + 7) // 8 * 8
        c["T"] = min(_log_int(rng, 1, 8192), (1 << 26) // (c["top"] * c["H"]))
        c["weights"] = rng.random() < 0.5 if kind.startswith("dispatch") else rng.random() < 0.8
        c["residual"] = kind == "combine" and rng.random() < 0.5
        c["drop"], c["skew"] = rng.random() < 0.4, rng.random() < 0.4
    elif kind in ("norm", "norm_backward"):
        c["H"] = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            c["H"] = (c["H"] + 7) // 8 * 8
        c["T"] = min(_log_int(rng, 1, 16384), (1 << 25) // c["H"])
        c["gate"] = rng.choice(("none", "token", "channel", "full"))
        c["gate_act"] = "none" if c["gate"] == "none" else rng.choice(("none", "sigmoid", "silu"))
        c["post"] = rng.random() < 0.7
        c["branch"], c["keep"] = rng.choice((1.0, 0.5, 0.22)), rng.choice((1.0, 0.75))
    else:
        c["kind"] = kind.replace("experts", "linear")
        c["dtype"] = rng.choice(("bf16", "bf16", "fp16"))
        c["act"] = rng.choice(ACTS)
        c["bias"] = rng.random() < 0.5
        c["keep"] = kind in ("linear", "experts") and rng.random() < 0.3
        c["residual"] = kind in ("linear", "experts") and rng.random() < 0.4
        c["K"] = 8 * _log_int(rng, 8, 512)
        c["E"], c["top"], c["skew"] = 0, 0, False
        if kind.startswith("experts"):
            c["E"] = _log_int(rng, 2, 256)
            c["top"], c["skew"] = rng.randint(1, min(8, c["E"])), rng.random() < 0.4
            c["N"] = min(_log_int(rng, 64, 2048), (1 << 29) // (c["E"] * c["K"]))
            c["T"] = min(_log_int(rng, 1, 4096), (1 << 36) // (c["top"] * c["K"] * max(64, c["N"])))
        else:
            c["N"] = _log_int(rng, 16, 8192)
            c["T"] = min(_log_int(rng, 1, 8192), (1 << 35) // (c["K"] * c["N"]))
        if c["act"] == "swiglu":  # gate and up halves of 16 features or a multiple
            c["N"] = 32 * max(1, c["N"] // 32)
        if c["E"]:
            c["T"] = max(1, c["T"])
    return c


def _rows(c):
    return c["T"] * c["top"] if c["E"] else c["T"]


def work(case):
    c, b = case, SIZE[case["dtype"]]
    T = c["T"]
    if c["kind"] in ("dispatch", "dispatch_backward", "combine", "combine_backward"):
        P, H = T * c["top"], c["H"]
        move = (P + T) * H * b + 8 * P  # the rows, the tokens, ids or places, weights
        if c["kind"] == "dispatch":
            return {"bytes": move + 8 * P, "flops": P * H}
        if c["kind"] == "combine":
            return {"bytes": move + (T * H * b if c["residual"] else 0), "flops": 2 * P * H}
        if c["kind"] == "combine_backward":
            return {"bytes": move + (P * H * b if c["weights"] else 0), "flops": 3 * P * H}
        return {"bytes": move + (T * H * b if c["weights"] else 0), "flops": 4 * P * H}
    if c["kind"] in ("norm", "norm_backward"):
        n = T * c["H"] * b
        full = c["gate"] == "full"
        if c["kind"] == "norm":
            return {"bytes": (5 if full else 4) * n, "flops": 12 * T * c["H"]}
        return {"bytes": (8 if full else 6) * n, "flops": 30 * T * c["H"]}
    P, N, K, E = _rows(c), c["N"], c["K"], max(1, c["E"])
    touched = E * (1.0 - (1.0 - 1.0 / E) ** P) if E > 1 else 1
    wide = N // 2 if c["act"] == "swiglu" else N
    if c["kind"] == "linear":
        bts = touched * N * K + P * K + P * wide * (2 if c["residual"] else 1) + (P * N if c["keep"] else 0) + (touched * N if c["bias"] else 0)
        return {"bytes": int(b * bts), "flops": 2 * P * N * K}
    bts = touched * N * K + E * N * K + 2 * P * K + P * wide + (0 if c["act"] == "none" else P * N) + (E * N if c["bias"] else 0)
    return {"bytes": int(b * bts), "flops": 4 * P * N * K}


# ----------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ids(gen, T, E, top, skew, drop):
    """Distinct experts for each token, load even or falling with the square root of the rank; dropped slots -1."""
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    if skew:
        score = score - 0.5 * torch.log(torch.randperm(E, generator=gen, device=DEV).float() + 1)
    ids = score.topk(top, dim=1).indices.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(T, top, generator=gen, device=DEV) < 0.1, -1, ids)
    return ids


def _order(ids, E):
    """Counts, offsets, the pairs in order (-1 behind the last) and each pair's place (-1: dropped)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = key.argsort(stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=DEV).index_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts.cumsum(0)])
    at = torch.arange(flat.numel(), device=DEV)
    perm = torch.where(at < offsets[E], order, -1)
    inv = torch.empty_like(order)
    inv[order] = at
    inv = torch.where(key < E, inv, -1)
    return tuple(t.to(torch.int32) for t in (counts, offsets, perm, inv))


def _randn(gen, dt, *shape, scale=1.0):
    out = torch.empty(*shape, dtype=TYPES[dt], device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV) * scale)
    return out


def _inputs(case, seed):
    c, gen, dt = case, _gen(seed), case["dtype"]
    T = c["T"]
    if c["kind"] in ("dispatch", "dispatch_backward", "combine", "combine_backward"):
        H, E, top = c["H"], c["E"], c["top"]
        s = {"ids": _ids(gen, T, E, top, c["skew"], c["drop"])}
        s["w"] = torch.softmax(torch.randn(T, top, generator=gen, device=DEV), 1) if c["weights"] else None
        if c["kind"] != "dispatch":
            s["inv"] = _order(s["ids"], E)[3]
        s["token"] = _randn(gen, dt, T, H)  # x of a dispatch, the gradient of a combine's result, the residual
        if c["kind"] != "dispatch":
            s["rows"] = _randn(gen, dt, T * top, H)
        return s
    if c["kind"] in ("norm", "norm_backward"):
        H = c["H"]
        s = {"y": _randn(gen, dt, T, H, scale=2.0), "residual": _randn(gen, dt, T, H)}
        s["gate"] = None if c["gate"] == "none" else _randn(gen, dt, *{"token": (T,), "channel": (H,), "full": (T, H)}[c["gate"]])
        s["post"] = (1 + _randn(gen, "fp32", H, scale=0.2)).to(TYPES[dt]) if c["post"] else None
        s["pre"] = (1 + _randn(gen, "fp32", H, scale=0.2)).to(TYPES[dt])
        if c["kind"] == "norm_backward":
            s["s"] = s.pop("residual")  # the sum that the forward pass kept
            s["ds"], s["dxn"] = _randn(gen, dt, T, H), _randn(gen, dt, T, H)
        return s
    N, K, E, P = c["N"], c["K"], c["E"], _rows(c)
    wide = N // 2 if c["act"] == "swiglu" else N
    s = {"x": _randn(gen, dt, P, K), "w": _randn(gen, dt, max(1, E), N, K, scale=1 / math.sqrt(K)), "offsets": None}
    if E:
        ids = _ids(gen, T, E, c["top"], c["skew"], False)
        s["offsets"] = _order(ids, E)[1]
    s["bias"] = _randn(gen, dt, max(1, E), N, scale=0.5) if c["bias"] else None
    if c["kind"] == "linear":
        s["residual"] = _randn(gen, dt, P, wide) if c["residual"] else None
    else:
        s["z"] = None if c["act"] == "none" else _randn(gen, dt, P, N)
        s["dout"] = _randn(gen, dt, P, wide)
    return s


def prepare(case, seed):
    case = dict(case)
    s = _inputs(case, seed)
    s["case"] = c = case
    T, dt = c["T"], TYPES[c["dtype"]]
    if c["kind"] in ("dispatch", "combine_backward"):  # the experts' rows: those that no token fills stay as they are
        s["filled"] = torch.zeros(T * c["top"], c["H"], dtype=dt, device=DEV)
    if c["kind"] in ("linear", "linear_backward") and c["E"]:
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the busiest expert
    if own:  # what a program makes once: sizes as one object, workspaces
        import sparse_moe_ffn_router_gb300 as moe
        types = {"bf16": moe.BF16, "fp16": moe.FP16, "fp32": moe.FP32}
        if c["kind"] in ("norm", "norm_backward"):
            s["dims"] = moe.NormDims(T, c["H"], dtype=types[c["dtype"]], post=c["post"],
                                     gate={"none": moe.GATE_NONE, "token": moe.GATE_TOKEN, "channel": moe.GATE_CHANNEL, "full": moe.GATE_FULL}[c["gate"]],
                                     gate_act={"none": moe.ACT_NONE, "sigmoid": moe.ACT_SIGMOID, "silu": moe.ACT_SILU}[c["gate_act"]],
                                     eps=EPS, branch_scale=c["branch"], residual_scale=c["keep"])
            if c["kind"] == "norm_backward":
                s["workspace"] = moe.new_norm_workspace(s["dims"])
        if c["kind"] in ("linear", "linear_backward"):
            act = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "swiglu": moe.ACT_SWIGLU}[c["act"]]
            s["dims"] = moe.LinearDims(_rows(c), c["N"], c["K"], E=max(1, c["E"]), act=act, dtype=types[c["dtype"]])
            s["workspace"] = moe.new_linear_workspace(s["dims"], backward=c["kind"] == "linear_backward")
    return s


# ----------------------------------------------------------------------------------------
# one pass

def run(s):
    return {"dispatch": _dispatch, "dispatch_backward": _dispatch_backward, "combine": _combine, "combine_backward": _combine_backward,
            "norm": _norm, "norm_backward": _norm_backward, "linear": _linear, "linear_backward": _linear_backward}[s["case"]["kind"]](s)


def _dispatch(s):
    c, x, w = s["case"], s["token"], s["w"]
    P = c["T"] * c["top"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        counts, offsets = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (c["E"], c["E"] + 1))
        perm, inv = (torch.empty(P, dtype=torch.int32, device=DEV) for _ in range(2))
        moe.moe_sort_pairs(c["E"], s["ids"], counts, offsets, perm, inv)
        moe.moe_dispatch(x, inv, w, s["filled"])
        return {"counts": counts, "offsets": offsets, "perm": perm, "inv": inv, "rows": s["filled"]}
    counts, offsets, perm, inv = _order(s["ids"], c["E"])
    at = perm.clamp(min=0).long()
    rows = x.float()[at // c["top"]]
    if w is not None:
        rows = rows * w.reshape(-1)[at][:, None]
    rows = torch.where((perm >= 0)[:, None], rows, 0.0).to(x.dtype)
    return {"counts": counts, "offsets": offsets, "perm": perm, "inv": inv, "rows": rows}


def _picked(s):
    """The rows of every pair in fp32, [T, top, H], zero for dropped ones."""
    c, inv = s["case"], s["inv"].long()
    rows = s["rows"][inv.clamp(min=0)].float()
    return torch.where((inv >= 0)[:, None], rows, 0.0).view(c["T"], c["top"], c["H"])


def _combine(s):
    c = s["case"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        out = torch.empty_like(s["token"])
        moe.moe_combine(s["rows"], s["inv"], s["w"], s["token"] if c["residual"] else None, out)
        return {"out": out}
    rows = _picked(s)
    out = (rows if s["w"] is None else rows * s["w"][:, :, None]).sum(1)
    if c["residual"]:
        out = out + s["token"].float()
    return {"out": out.to(TYPES[c["dtype"]])}


def _dispatch_backward(s):
    c, x, w = s["case"], s["token"], s["w"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        dx, dw = torch.empty_like(x), None if w is None else torch.empty_like(w)
        moe.moe_dispatch_backward(s["rows"], s["inv"], w, x, dx, dw)
        return {"dx": dx, "dw": dw}
    rows = _picked(s)
    dx = (rows if w is None else rows * w[:, :, None]).sum(1).to(x.dtype)
    return {"dx": dx, "dw": None if w is None else (rows * x.float()[:, None]).sum(2)}


def _combine_backward(s):
    c, dout, w, inv = s["case"], s["token"], s["w"], s["inv"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        dw = None if w is None else torch.empty_like(w)
        moe.moe_combine_backward(dout, inv, w, s["rows"], s["filled"], dw)
        return {"drows": s["filled"], "dw": dw}
    g = dout.float()[:, None].expand(-1, c["top"], -1)
    spread = (g if w is None else g * w[:, :, None]).reshape(-1, c["H"])
    at = torch.where(inv >= 0, inv.long(), inv.numel())
    drows = torch.zeros(inv.numel() + 1, c["H"], device=DEV).index_copy_(0, at, spread)[:-1].to(dout.dtype)
    return {"drows": drows, "dw": None if w is None else (_picked(s) * g).sum(2)}


def _gate_value(c, gate):
    """The gate's values after their activation, shaped to multiply [T, H]."""
    if gate is None:
        return 1.0
    g = gate[:, None] if c["gate"] == "token" else gate
    return {"none": lambda: g, "sigmoid": lambda: torch.sigmoid(g), "silu": lambda: g * torch.sigmoid(g)}[c["gate_act"]]()


def _gate_slope(c, gate):
    g = gate[:, None] if c["gate"] == "token" else gate
    p = torch.sigmoid(g)
    return {"none": torch.ones_like(g), "sigmoid": p * (1 - p), "silu": p * (1 + g * (1 - p))}[c["gate_act"]]


def _norm_of(v, gamma):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * gamma


def _norm(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        total, xn = torch.empty_like(s["y"]), torch.empty_like(s["y"])
        moe.moe_norm_residual(s["dims"], s["y"], s["residual"], s["gate"], s["post"], s["pre"], total, xn)
        return {"s": total, "xn": xn}
    y = s["y"].float()
    if c["post"]:
        y = _norm_of(y, s["post"].float())
    total = c["keep"] * s["residual"].float() + c["branch"] * _gate_value(c, None if s["gate"] is None else s["gate"].float()) * y
    return {"s": total.to(dt), "xn": _norm_of(total, s["pre"].float()).to(dt)}


def _norm_grad(v, gamma, g):
    """Gradients of N(v; gamma) for the gradient g of its result: of v, and the terms whose sum over rows is gamma's."""
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    gg = g * gamma
    return r * gg - v * (r ** 3) * (gg * v).mean(1, keepdim=True), g * v * r


def _norm_backward(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        dres, dy = torch.empty_like(s["y"]), torch.empty_like(s["y"])
        dgate = None if s["gate"] is None else torch.empty_like(s["gate"])
        dpost, dpre = None if s["post"] is None else torch.empty_like(s["post"]), torch.empty_like(s["pre"])
        moe.moe_norm_residual_backward(s["dims"], s["ds"], s["dxn"], s["s"], s["y"], s["gate"], s["post"], s["pre"],
                                       dres, dy, dgate, dpost, dpre, s["workspace"])
        return {"dresidual": dres, "dy": dy, "dgate": dgate, "dpost": dpost, "dpre": dpre}
    return {k: None if v is None else v.to(dt) for k, v in _norm_gradients(s, torch.float32).items()}


def _norm_gradients(s, wide):
    c = s["case"]
    ds, dxn, total, y = (s[k].to(wide) for k in ("ds", "dxn", "s", "y"))
    gate = None if s["gate"] is None else s["gate"].to(wide)
    through, pre = _norm_grad(total, s["pre"].to(wide), dxn)
    g = ds + through
    n = _norm_of(y, s["post"].to(wide)) if c["post"] else y
    dn = c["branch"] * _gate_value(c, gate) * g
    dgate = None
    if gate is not None:
        dgate = c["branch"] * g * n * _gate_slope(c, gate)
        if c["gate"] != "full":
            dgate = dgate.sum(1 if c["gate"] == "token" else 0)
    dy, dpost = _norm_grad(y, s["post"].to(wide), dn) if c["post"] else (dn, None)
    return {"dresidual": c["keep"] * g, "dy": dy, "dgate": dgate, "dpost": None if dpost is None else dpost.sum(0), "dpre": pre.sum(0)}


def _act(name, z):
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))}[name]()


def _act_grad(name, z, d):
    """The gradient of z for the gradient d of act(z)."""
    if name == "none":
        return d
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        p = torch.sigmoid(g)
        return torch.cat([d * u * p * (1 + g * (1 - p)), d * g * p], -1)
    if name == "relu":
        return torch.where(z > 0, d, 0.0)
    p = torch.sigmoid(z)
    return d * (p * (1 + z * (1 - p)) if name == "silu" else
                0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))


def _places(s):
    """Each row's expert and its place among that expert's rows."""
    at = torch.arange(s["x"].shape[0], device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    return e, at - s["offsets"].long()[e]


def _padded(s, t, places):
    """Rows [P, n] as [E, most, n] in fp32, zero behind each expert's last."""
    out = torch.zeros(s["case"]["E"], s["most"], t.shape[1], device=DEV)
    out[places] = t.float()
    return out


def _linear(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    P, N = _rows(c), c["N"]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        out = torch.empty(P, N // 2 if c["act"] == "swiglu" else N, dtype=dt, device=DEV)
        z = torch.empty(P, N, dtype=dt, device=DEV) if c["keep"] else None
        moe.moe_linear(s["dims"], s["x"], s["w"], s["bias"], s["offsets"], s["residual"], out, z, s["workspace"])
        return {"out": out, "z": z}
    if c["E"]:
        places = _places(s)
        z = (_padded(s, s["x"], places) @ s["w"].float().transpose(1, 2))[places]
        if s["bias"] is not None:
            z = z + s["bias"].float()[places[0]]
    else:
        z = s["x"].float() @ s["w"][0].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
    out = _act(c["act"], z)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return {"out": out.to(dt), "z": z.to(dt) if c["keep"] else None}


def _linear_backward(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    if own:
        import sparse_moe_ffn_router_gb300 as moe
        dx, dw = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        db = None if s["bias"] is None else torch.empty_like(s["bias"])
        moe.moe_linear_backward(s["dims"], s["x"], s["w"], s["offsets"], s["z"], s["dout"], dx, dw, db, s["workspace"])
        return {"dx": dx, "dw": dw, "db": db}
    dz = _act_grad(c["act"], None if s["z"] is None else s["z"].float(), s["dout"].float())
    if not c["E"]:
        dx, dw = dz @ s["w"][0].float(), (dz.T @ s["x"].float())[None]
        return {"dx": dx.to(dt), "dw": dw.to(dt), "db": None if s["bias"] is None else dz.sum(0, keepdim=True).to(dt)}
    places = _places(s)
    dz = _padded(s, dz, places)
    dx = (dz @ s["w"].float())[places].to(dt)
    dw = (dz.transpose(1, 2) @ _padded(s, s["x"], places)).to(dt)
    return {"dx": dx, "dw": dw, "db": None if s["bias"] is None else dz.sum(1).to(dt)}


# ----------------------------------------------------------------------------------------
# the definition in 64 bits

def exact(case, seed):
    c = case = dict(case)
    s = _inputs(case, seed)
    s["case"] = case
    if c["kind"] in ("dispatch", "dispatch_backward", "combine", "combine_backward"):
        T, top, H = c["T"], c["top"], c["H"]
        tok = s["token"].double()
        w = None if s["w"] is None else s["w"].double()
        if c["kind"] == "dispatch":
            _, _, perm, inv = _order(s["ids"], c["E"])
            rows = torch.zeros(T * top, H, dtype=torch.float64, device=DEV)
            for k in range(top):
                at = inv.view(T, top)[:, k].long()
                live = at >= 0
                rows[at[live]] = tok[live] * (1.0 if w is None else w[live, k, None])
            return {"counts": None, "offsets": None, "perm": None, "inv": None, "rows": rows}
        inv = s["inv"].view(T, top).long()
        out = s["token"].double() if c["residual"] else torch.zeros(T, H, dtype=torch.float64, device=DEV)
        drows = torch.zeros(T * top, H, dtype=torch.float64, device=DEV)
        dots = torch.zeros(T, top, dtype=torch.float64, device=DEV)
        for k in range(top):
            live = inv[:, k] >= 0
            rows = s["rows"].double()[inv[live, k]]
            wk = 1.0 if w is None else w[live, k, None]
            out[live] += wk * rows
            drows[inv[live, k]] = wk * tok[live]
            dots[live, k] = torch.einsum("th,th->t", rows, tok[live])
        if c["kind"] == "combine":
            return {"out": out}
        dots = None if w is None else dots
        return {"dx": out, "dw": dots} if c["kind"] == "dispatch_backward" else {"drows": drows, "dw": dots}
    if c["kind"] == "norm":
        y, res, pre = (s[k].double() for k in ("y", "residual", "pre"))
        if c["post"]:
            y = y / (torch.linalg.vector_norm(y, dim=1, keepdim=True) ** 2 / c["H"] + EPS).sqrt() * s["post"].double()
        if s["gate"] is not None:
            g = s["gate"].double()
            g = g.view(-1, 1) if c["gate"] == "token" else g
            if c["gate_act"] != "none":
                p = 1 / (1 + torch.exp(-g))
                g = p if c["gate_act"] == "sigmoid" else g * p
            y = y * g
        total = res * c["keep"] + y * c["branch"]
        return {"s": total, "xn": total / (torch.linalg.vector_norm(total, dim=1, keepdim=True) ** 2 / c["H"] + EPS).sqrt() * pre}
    if c["kind"] == "norm_backward":  # by differentiation of the definition
        s = {k: v for k, v in s.items()}
        leaf = {k: s[k].double().requires_grad_() for k in ("y", "gate", "post") if s[k] is not None}
        y = leaf["y"]
        n = y / (y.square().mean(1, keepdim=True) + EPS).sqrt() * leaf["post"] if c["post"] else y
        if "gate" in leaf:
            g = leaf["gate"].view(-1, 1) if c["gate"] == "token" else leaf["gate"]
            p = 1 / (1 + torch.exp(-g))
            n = n * {"none": g, "sigmoid": p, "silu": g * p}[c["gate_act"]]
        total, pre = s["s"].double().requires_grad_(), s["pre"].double().requires_grad_()
        xn = total / (total.square().mean(1, keepdim=True) + EPS).sqrt() * pre
        dtotal, dpre = torch.autograd.grad(xn, (total, pre), s["dxn"].double())
        g = s["ds"].double() + dtotal
        got = dict(zip(leaf, torch.autograd.grad(c["branch"] * n, list(leaf.values()), g)))
        return {"dresidual": c["keep"] * g, "dy": got["y"], "dgate": got.get("gate"), "dpost": got.get("post"), "dpre": dpre}
    P, N, K = _rows(c), c["N"], c["K"]
    ends = [0, P] if not c["E"] else s["offsets"].tolist()
    wide = N // 2 if c["act"] == "swiglu" else N
    forward = c["kind"] == "linear"
    first = torch.zeros(P, wide if forward else K, dtype=torch.float64, device=DEV)  # out, or dx
    z = torch.zeros(P, N, dtype=torch.float64, device=DEV) if forward else None
    dw = None if forward else torch.zeros(max(1, c["E"]), N, K, dtype=torch.float64, device=DEV)
    db = None if forward else torch.zeros(max(1, c["E"]), N, dtype=torch.float64, device=DEV)
    for e in range(max(1, c["E"])):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        x, w = s["x"][a:b].double(), s["w"][e].double()
        if forward:
            z[a:b] = x @ w.T + (0.0 if s["bias"] is None else s["bias"][e].double())
            first[a:b] = _act64(c["act"], z[a:b])
            continue
        d = s["dout"][a:b].double()
        if c["act"] != "none":
            ze = s["z"][a:b].double().requires_grad_()
            d, = torch.autograd.grad(_act64(c["act"], ze), ze, d)
        first[a:b] = d @ w
        dw[e] = d.T @ x
        db[e] = d.sum(0)
    if forward:
        if s["residual"] is not None:
            first += s["residual"].double()
        return {"out": first, "z": z if c["keep"] else None}
    return {"dx": first, "dw": dw, "db": db if s["bias"] is not None else None}


def _act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    g = z if name == "silu" else z[:, :z.shape[1] // 2]
    h = g / (1 + torch.exp(-g))
    return h if name == "silu" else h * z[:, z.shape[1] // 2:]
