"""What the 4-bit layer leaves in the workspace, stage by stage against 64 bits (w4_stages.py)."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import w4_reference as ref
from tests import w4_stages as st
from tests.test_gpu_w4 import W4Layer, check, run_linear

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


def check_stages(L, ws, out, residual):
    """Every stage of the call that left ws and out: routing, h, Y and the sum."""
    T, H, E, K, I, Is = L.dims
    big = T >= 256
    ids, w, g = check_routing(L, ws)
    h = check_activations(L, ws, ids, rounded=big)
    W = {k: st.weights(L.name, L.group, L.m[k], big) for k in ("down", "shared_down")}
    half = big and K > 1
    Y = tap(ws, L.dims, 1, torch.bfloat16 if half else torch.float32, (T, K + 1, H))
    check(Y, *st.outputs(L.dims, h, ids, w, g, W["down"], W["shared_down"][0], ref.HALF if half else 0.0), "Y")
    check(out, *st.combined(Y, L.residual if residual else None), "out")


@pytest.mark.parametrize("dims,name,group", [
    ((1, 2048, 64, 8, 512, 512), "int4", 64), ((1, 512, 4, 1, 128, 64), "e2m1", 32), ((1, 5120, 16, 4, 128, 128), "int4_zp", 128),
    ((2, 512, 32, 4, 128, 128), "int4_zp", 64), ((7, 2048, 256, 8, 512, 512), "e2m1", 64), ((8, 8192, 8, 2, 64, 192), "int4", 32),
    ((9, 640, 21, 5, 192, 448), "int4", 64), ((64, 2048, 64, 8, 512, 512), "int4_zp", 128), ((130, 384, 3, 3, 2048, 64), "e2m1", 32),
    ((255, 512, 16, 2, 128, 2048), "int4", 64), ((255, 128, 1, 1, 64, 64), "int4", 32),
    ((256, 512, 32, 4, 128, 128), "int4", 32), ((300, 2048, 32, 8, 512, 512), "e2m1", 64), ((777, 640, 11, 3, 192, 320), "int4_zp", 64),
    ((1000, 128, 8, 2, 64, 64), "int4", 32), ((512, 2304, 9, 8, 576, 128), "e2m1", 32), ((300, 512, 4, 1, 128, 64), "e2m1", 64),
    ((2000, 640, 64, 2, 64, 192), "int4_zp", 64), ((1500, 256, 24, 3, 64, 704), "int4", 64), ((260, 8192, 6, 2, 2048, 1024), "int4_zp", 128),
    ((4096, 2048, 256, 8, 512, 512), "int4", 64)],
    ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_layer_stage_by_stage(dims, name, group):
    L = W4Layer(dims, name, group, seed=sum(dims) + 1, bias=dims[0] % 2 == 0)
    ws = moe.new_workspace(L.dims)
    for residual in (True, False):
        for which in (0, 1):
            at, n = moe.moe_w4_workspace_tap(L.dims, which)
            ws[at:at + n] = 255
        check_stages(L, ws, L.run(residual=residual, ws=ws), residual)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("name,group", [("int4", 128), ("int4_zp", 32), ("e2m1", 64)])
@pytest.mark.parametrize("T,N,K", [(64, 1000, 1024), (70, 129, 128), (129, 257, 640), (190, 512, 2048), (300, 384, 512), (1000, 130, 256)])
def test_linear_that_does_not_round_its_weights(name, group, T, N, K):
    """The streaming path's larger token counts, by the bound without a rounding of the weights."""
    assert not ref.linear_rounds(T, N, sms())
    x, w, b, out = run_linear(name, group, T, N, K, bias=N % 2 == 0, seed=3)
    check(out, *ref.linear(x, w, b))


@pytest.mark.parametrize("name,group,cols", [(f, 32, c) for f in ref.FORMATS for c in (32, 96, 160)] + [("int4", 64, 64), ("int4_zp", 64, 1984), ("e2m1", 128, 2048)])
@pytest.mark.parametrize("T,N", [(3000, 640), (9, 24001)])
def test_linear_on_rounded_weights(name, group, cols, T, N):
    """The tensor-core path's weights are s * v rounded to bf16: by the bound of the sums alone, also with columns that
    are no whole record or half of one."""
    assert ref.linear_rounds(T, N, sms())
    m = ref.matrices(name, group, 1, N, cols, seed=cols)
    x = torch.randn(T, cols, device="cuda").to(torch.bfloat16)
    f = ref.fmt(name, group)
    ws, out = moe.new_w4_linear_workspace(f, T, N, cols), torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_linear(f, x, ref.pack(name, group, m), None, out, ws)
    assert moe.moe_last_device_error(ws) == 0
    check(out, *ref.linear(x, st.weights(name, group, m, True)[0], None))


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


@pytest.mark.parametrize("name,group", [("int4", 32), ("int4_zp", 64), ("e2m1", 128)])
@pytest.mark.parametrize("T", [3, 3000])
def test_linear_smallest_scales(name, group, T):
    """Scales from the smallest subnormal bf16 to 2^-118 by token rows of 2^110: the streaming path multiplies by s * v, the
    tensor-core path by s * v rounded to bf16, which for integer codes is rounded at a quarter of its size."""
    N, K = 640, 256
    codes, _, zeros = ref.matrices(name, group, 1, N, K, seed=2)
    g = torch.Generator(device="cuda").manual_seed(4)
    bits = torch.randint(1, 9 << 7, (1, N, K // group), generator=g, device="cuda")  # 2^-133 .. 2^-118
    m = codes, bits.to(torch.int16).view(torch.bfloat16), zeros
    x = (torch.randn(T, K, generator=g, device="cuda") * 2.0 ** 110).to(torch.bfloat16)
    f = ref.fmt(name, group)
    ws, out = moe.new_w4_linear_workspace(f, T, N, K), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_linear(f, x, ref.pack(name, group, m), None, out, ws)
    assert moe.moe_last_device_error(ws) == 0
    w = ref.values(name, group, m)[0]
    if ref.linear_rounds(T, N, sms()):
        part = 1.0 if name == "e2m1" else 4.0
        w = (w / part).float().to(torch.bfloat16).double() * part
    assert ref.linear_rounds(T, N, sms()) == (T == 3000)
    check(out, *ref.linear(x, w, None))


@pytest.mark.parametrize("flags", [0, moe.FLAG_BF16_SCORES])
@pytest.mark.parametrize("T", [1, 5, 8, 40, 300])
def test_layer_routing_with_equal_scores(T, flags):
    """Scores that are exact in fp32 (sums of sixteenths), many of them equal, more so when rounded to bf16: the lower
    expert comes first, and every stage follows."""
    dims = (T, 512, 32, 4, 128, 64)
    L = W4Layer(dims, "int4", 32, seed=T, bias=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    draw = lambda low, high, *shape: torch.randint(low, high, shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    L.x, L.router_w, L.router_b = draw(-1, 2, T, 512), draw(-8, 9, 32, 512) / 16, draw(-2, 3, 32)
    L.W = moe.Weights(L.router_w, L.router_b, L.W.gate_up, L.W.down, L.W.shared_gate_up, L.W.shared_down, L.shared_gate)
    score = L.x.double() @ L.router_w.double().T + L.router_b.double()
    assert float(score.abs().max()) * 16 < 1 << 24
    if flags:
        score = score.float().to(torch.bfloat16).double()
    top = score.sort(dim=1, descending=True, stable=True)
    assert T < 40 or bool((top.values[:, :4] == top.values[:, 1:5]).any())
    ws, out = moe.new_workspace(dims), torch.empty_like(L.x)
    moe.moe_forward_w4((*dims, flags), ref.fmt("int4", 32), L.x, L.W, L.residual, out, ws)
    assert moe.moe_last_device_error(ws) == 0
    ids, w = tap(ws, dims, 3, torch.int32, (T, 4)), tap(ws, dims, 4, torch.float32, (T, 4))
    assert torch.equal(ids.long(), top.indices[:, :4])
    want = torch.softmax(top.values[:, :4], 1)
    # exact differences of scores; expf, three additions and the division: a few fp32 steps
    check(w, want, 2.0 ** -20 * want + 1e-30, "routing weights")
    check_activations(L, ws, ids, rounded=T >= 256)


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_layer_of_large_activations(T):
    """Gate values far into both tails of the sigmoid, where its exponential overflows."""
    L = W4Layer((T, 512, 16, 2, 128, 128), "int4", 32, seed=T)
    L.x = (L.x.float() * 96).to(torch.bfloat16)
    ids = st.routing(L.x, L.router_w, L.router_b, L.shared_gate, 2)[0]
    gate = L.x.double() @ st.weights("int4", 32, L.m["shared_gate_up"], False)[0, :128].T
    assert float(gate.min()) < -90 and float(gate.max()) > 90
    ws = moe.new_workspace(L.dims)
    out = L.run(ws=ws)
    assert torch.equal(tap(ws, L.dims, 3, torch.int32, (T, 2)).long(), ids) and bool(out.isfinite().all())
    check_activations(L, ws, ids, rounded=T >= 256)


def test_layers_on_two_streams_at_once():
    """Layers of two tokens and more in flight together, each with its own workspace and output."""
    layers = [W4Layer((T, 2048, 32, 8, 512, 512), "int4", 64, seed=T) for T in (2, 8, 40, 300)]
    f = ref.fmt("int4", 64)
    spaces = [[moe.new_workspace(L.dims) for L in layers] for _ in range(2)]
    outs = [[torch.empty_like(L.x) for L in layers] for _ in range(2)]
    alone = [L.run() for L in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i, s in enumerate(streams):
            for j in (range(4) if i == 0 else reversed(range(4))):
                L = layers[j]
                moe.moe_forward_w4(L.dims, f, L.x, L.W, L.residual, outs[i][j], spaces[i][j], s)
    torch.cuda.synchronize()
    for i in range(2):
        for j in range(4):
            assert moe.moe_last_device_error(spaces[i][j]) == 0 and torch.equal(outs[i][j], alone[j])
