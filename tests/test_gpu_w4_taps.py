"""What the 4-bit layer leaves in the workspace, stage by stage against 64 bits (w4_stages.py)."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import w4_reference as ref
from tests import w4_stages as st
from tests.test_gpu_w4 import W4Layer, check

pytestmark = pytest.mark.gpu


def tap(ws, dims, which, dtype, shape):
    at, n = moe.moe_w4_workspace_tap(dims, which)
    t = ws[at:at + n].view(dtype)
    assert t.numel() == torch.Size(shape).numel()
    return t.view(shape)


def check_routing(L, ws):
    T, H, E, K, I, Is = L.dims
    ids, topw, sgate = st.routing(L.x, L.router_w, L.router_b, L.shared_gate, K)
    got = tap(ws, L.dims, 3, torch.int32, (T, K))
    assert torch.equal(got.long(), ids)
    w, g = tap(ws, L.dims, 4, torch.float32, (T, K)), tap(ws, L.dims, 2, torch.float32, (T,))
    check(w, topw, torch.full_like(topw, 5e-4), "routing weights")
    check(g, sgate, torch.full_like(sgate, 5e-4), "shared gate")
    return got, w, g


def check_activations(L, ws, ids, rounded=False):
    T, H, E, K, I, Is = L.dims
    W = {k: st.weights(L.name, L.group, L.m[k], rounded) for k in ("gate_up", "shared_gate_up")}
    want, bound = st.activations(L.dims, L.x, ids, W["gate_up"], W["shared_gate_up"][0])
    h = tap(ws, L.dims, 0, torch.bfloat16, want.shape)
    live = ~want.isnan()
    check(h[live], want[live], bound[live], "h")
    return h


@pytest.mark.parametrize("dims,name,group", [((1, 512, 32, 4, 128, 128), "int4", 32), ((1, 1024, 64, 2, 512, 64), "e2m1", 64),
                                             ((1, 128, 8, 1, 64, 64), "int4_zp", 64), ((1, 640, 200, 8, 64, 320), "int4", 64),
                                             ((1, 2048, 256, 8, 512, 512), "int4", 32), ((1, 4096, 16, 8, 192, 2048), "e2m1", 32)],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_one_token_leaves_its_activations(dims, name, group):
    """Tap 0 of the one-kernel layer holds the experts' rows in dispatch order, every time; with fewer routed gate_up
    strips (K * I / 8) than SMs, the CTA that writes it has none of its own."""
    for seed in range(4):  # other experts, in other orders
        L = W4Layer(dims, name, group, seed=seed + sum(dims), bias=True)
        ws = moe.new_workspace(L.dims)
        at, n = moe.moe_workspace_tap(L.dims, 0)
        first = None
        for _ in range(40):
            ws[at:at + n] = 255
            L.run(ws=ws)
            if first is None:
                check_activations(L, ws, check_routing(L, ws)[0])
                first = ws[at:at + n].clone()
            assert torch.equal(ws[at:at + n], first)


@pytest.mark.parametrize("dims", [(4000, 256, 6, 1, 64, 64), (700, 1280, 5, 1, 64, 192), (3001, 2048, 40, 1, 128, 256)],
                         ids=lambda v: "x".join(map(str, v)))
def test_one_expert_a_token_leaves_its_outputs(dims):
    """With one expert a token Y is fp32 from 256 tokens too; several tiles to a CTA, every value written by its own
    token and scale, every time, also where Y held NaN before."""
    L = W4Layer(dims, "int4", 64, seed=sum(dims), bias=True)
    T, H, E, K, I, Is = dims
    ws = moe.new_workspace(L.dims)
    y = tap(ws, L.dims, 1, torch.float32, (T, 2, H))
    first = None
    for _ in range(30):
        y.fill_(float("nan"))
        L.run(ws=ws)
        if first is None:
            ids, w, g = check_routing(L, ws)
            h = check_activations(L, ws, ids, rounded=True)
            W = {k: st.weights(L.name, L.group, L.m[k], True) for k in ("down", "shared_down")}
            check(y, *st.outputs(L.dims, h, ids, w, g, W["down"], W["shared_down"][0], 0.0), "Y")
            first = y.clone()
        assert torch.equal(y, first)


@pytest.mark.parametrize("dims", [(300, 512, 4, 1, 128, 64), (1, 2048, 64, 8, 512, 512)], ids=lambda v: "x".join(map(str, v)))
def test_bf16_layer_leaves_the_rest_of_a_shorter_workspace_alone(dims):
    """moe_forward on a workspace without the 4-bit layer's own part: same result, nothing behind it touched."""
    T, H, E, K, I, Is = dims
    L = W4Layer(dims, "int4", 64, seed=5, bias=True)
    dense = [torch.empty(m[0].shape, dtype=torch.bfloat16, device="cuda") for m in L.m.values()]
    for (k, w) in zip(L.m, dense):
        moe.moe_w4_dequantize(ref.fmt("int4", 64), getattr(L.W, k), w, k.endswith("gate_up"))
    W = moe.Weights(L.router_w, L.router_b, *dense, L.shared_gate)
    torch.cuda.synchronize()
    full = moe.new_workspace(dims)
    want, out = torch.empty_like(L.x), torch.empty_like(L.x)
    moe.moe_forward(dims, L.x, W, L.residual, want, full)
    extra = T * 2 * H * 2 if T > 1 else (K + 1) * max(I, Is) // 2 * 8
    ws = torch.zeros_like(full)
    ws[-extra:] = 77
    moe.moe_forward(dims, L.x, W, L.residual, out, ws[:-extra])
    assert moe.moe_last_device_error(ws) == 0 and torch.equal(out, want) and bool((ws[-extra:] == 77).all())


def test_linear_offsets_past_32_bits():
    """More than 2^32 elements of token rows and of results, on the tensor-core path: rows spread over the whole range."""
    T, N, K = (1 << 26) + 77, 66, 64
    assert T * N > 1 << 32 and T * K > 1 << 32 and torch.cuda.mem_get_info()[0] > 24 << 30
    m = ref.matrices("int4", 64, 1, N, K, seed=7)
    w, f = st.weights("int4", 64, m, True)[0], ref.fmt("int4", 64)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(0, 300), torch.randint(0, T, (3000,)), torch.arange(T - 300, T)]).unique().cuda()
    x[rows] = torch.randn(rows.numel(), K, device="cuda").to(torch.bfloat16)
    out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.new_w4_linear_workspace(f, T, N, K)
    moe.moe_w4_linear(f, x, ref.pack("int4", 64, m), None, out, ws)
    assert moe.moe_last_device_error(ws) == 0
    check(out[rows], *ref.linear(x[rows], w, None))
    out[rows] = 0
    assert all(not bool(part.any()) for part in out.split(1 << 24))
