"""The 4-bit weight operators on the GPU against plain 64-bit forms (w4_reference.py), at the sizes
where they can go wrong, with error bounds derived there."""
from __future__ import annotations

import pytest
import torch

import sparse_moe_ffn_router_gb300 as moe
from tests import w4_reference as ref

pytestmark = pytest.mark.gpu
FG = [(f, g) for f in ref.FORMATS for g in (32, 64, 128)]


def check(got, want, bound, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off / bound).max()):.2f} x the bound"


# ---------------------------------------------------------------------------------------- packing

def test_pack_layout_byte_by_byte():
    """One record of each format against the layout of moe.h, bit by bit."""
    for name, group in FG:
        m = ref.matrices(name, group, 1, 16, 128, seed=3)
        got = ref.pack(name, group, m)[0].cpu().tolist()
        codes, scales, zeros = (None if t is None else t[0].cpu() for t in m)
        per = 128 // group
        for r in range(16):
            for k in range(128):
                c, t, e = k // 32, k % 32 // 8, k % 8
                at = ((r // 8 * 8 + r % 8) * 4 + t) * 16 + c * 4 + 2 * (e & 1)
                half, i = got[at] | got[at + 1] << 8, e // 2
                if name == "e2m1":
                    bits = [(15, 8, 7, 6), (12, 5, 4, 3), (9, 2, 1, 0), (14, 13, 10, 11)][i]
                    code = sum(((half >> b) & 1) << s for b, s in zip(bits, (3, 2, 1, 0)))
                else:
                    code = half >> (4 * i) & 15
                assert code == int(codes[r, k]), (name, group, r, k)
            for i in range(per):
                at = 1024 + 2 * (r * per + i)
                assert got[at] | got[at + 1] << 8 == scales.view(torch.int16)[r, i].item() & 0xffff
                if zeros is not None:
                    assert got[1024 + 32 * per + r * per + i] == int(zeros[r, i])


@pytest.mark.parametrize("name,group", FG)
@pytest.mark.parametrize("n,rows,cols,layout", [(1, 16, 128, 0), (3, 32, 256, 1), (2, 1, 128, 0), (2, 37, 384, 0), (1, 48, 640, 1), (5, 19, 128 * 3, 0)])
def test_pack_and_dequantize(name, group, n, rows, cols, layout):
    m = ref.matrices(name, group, n, rows, cols, seed=rows + cols)
    out = torch.full((n, rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_dequantize(ref.fmt(name, group), ref.pack(name, group, m, layout), out, layout)
    assert torch.equal(out.double(), ref.values(name, group, m).to(torch.bfloat16).double())


@pytest.mark.parametrize("name,group", [(f, 32) for f in ref.FORMATS])
@pytest.mark.parametrize("cols", [32, 96, 160])
def test_columns_that_are_no_whole_record(name, group, cols):
    m = ref.matrices(name, group, 2, 21, cols, seed=cols)
    out = torch.empty(2, 21, cols, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_dequantize(ref.fmt(name, group), ref.pack(name, group, m), out)
    assert torch.equal(out.double(), ref.values(name, group, m).to(torch.bfloat16).double())


@pytest.mark.parametrize("name,group", FG)
@pytest.mark.parametrize("rows,cols,layout", [(32, 512, 1), (33, 384, 0), (1, 128, 0)])
def test_quantize(name, group, rows, cols, layout):
    g = torch.Generator().manual_seed(rows)
    w = torch.randn(3, rows, cols, generator=g) * torch.exp(3 * torch.randn(3, rows, 1, generator=g))
    w[0, 0, :group] = 0.0                                # a group of zeros
    w[1, 0, :group] = w[1, 0, :group].abs()              # one sign only
    w[2, 0, :group] = -w[2, 0, :group].abs()
    w[0, -1, -group:] = torch.arange(group) % 16 * 0.25  # values halfway between codes
    w = w.to(torch.bfloat16).cuda()
    packed = moe.new_w4(ref.fmt(name, group), rows, cols, 3)
    moe.moe_w4_quantize(ref.fmt(name, group), w, packed, layout)
    want = ref.quantize(name, group, w)
    assert torch.equal(packed, ref.pack(name, group, want, layout))


@pytest.mark.parametrize("name", list(ref.FORMATS))
def test_quantize_every_magnitude(name):
    """Every positive normal bf16 as a group's largest value, from the smallest whose scale is normal to 2^126, with
    other values of the group at and between the codes: scales and codes as the definition's divisions give them."""
    bits = torch.arange(0x0200, 0x7e80, dtype=torch.int32)  # 2^-123 .. 2^126
    b = (bits << 16).view(torch.float32)
    n = b.numel() // 16 * 16
    part = torch.tensor([1.0, -1.0, 0.5, 0.25, -0.75, 0.125, 0.375, -0.0625] * 4)
    w = (b[:n, None] * part).to(torch.bfloat16).view(1, n // 4, 128).cuda()
    packed = moe.new_w4(ref.fmt(name, 32), n // 4, 128)
    moe.moe_w4_quantize(ref.fmt(name, 32), w[0], packed)
    assert torch.equal(packed, ref.pack(name, 32, ref.quantize(name, 32, w)))


@pytest.mark.parametrize("name", list(ref.FORMATS))
def test_quantize_extreme_values(name):
    """The largest and smallest finite weights, and a group with an infinity or a NaN."""
    w = torch.zeros(1, 16, 128, dtype=torch.bfloat16, device="cuda")
    big = torch.finfo(torch.bfloat16).max
    w[0, 0, :32] = big
    w[0, 1, :32] = -big
    w[0, 1, 0] = big
    w[0, 2, :32] = 2.0 ** -133  # the smallest subnormal: the scale rounds to it or to zero
    w[0, 3, 0] = float("inf")
    w[0, 4, 40] = float("nan")
    f = ref.fmt(name, 32)
    packed, out = moe.new_w4(f, 16, 128), torch.empty_like(w)
    moe.moe_w4_quantize(f, w, packed)
    moe.moe_w4_dequantize(f, packed, out)
    out = out[0].float()
    assert bool(out[3, :32].isnan().all()) and bool(out[4, 32:64].isnan().all())
    out[3, :32] = 0
    out[4, 32:64] = 0
    # a step of the format at this scale; the largest value times the rounded scale may overflow bf16
    step = {"int4": 1 / 14, "int4_zp": 1 / 15, "e2m1": 1 / 6}[name] * 1.01 + 2.0 ** -7
    fine = out.isfinite()
    assert bool((fine | (w[0].float().abs() == big)).all())
    top = w[0].float().abs().amax(1, keepdim=True)
    top[3:5] = 0
    assert bool(((out - w[0].float().nan_to_num(0, 0, 0)).abs()[fine] <= (step * top + 2.0 ** -133).expand_as(out)[fine]).all())


# ---------------------------------------------------------------------------------------- linear

def run_linear(name, group, T, N, K, bias, seed=0, x=None):
    m = ref.matrices(name, group, 1, N, K, seed=seed + N)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if x is None:
        x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if bias else None
    f = ref.fmt(name, group)
    ws = moe.new_w4_linear_workspace(f, T, N, K)
    out = torch.full((T + 1, N), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_linear(f, x, ref.pack(name, group, m), b, out[:T], ws)
    assert moe.moe_last_device_error(ws) == 0
    assert bool((out[T] == 3.0).all())  # the row behind the last is left as it was
    return x, ref.values(name, group, m)[0], b, out[:T]


@pytest.mark.parametrize("name,group", FG)
@pytest.mark.parametrize("T,N,K", [(1, 64, 128), (1, 2048, 2048), (3, 37, 384), (8, 1, 256), (9, 1003, 1408), (1, 500, 8192)])
def test_linear(name, group, T, N, K):
    x, w, b, out = run_linear(name, group, T, N, K, bias=T != 3)
    check(out, *ref.linear(x, w, b))


@pytest.mark.parametrize("name", list(ref.FORMATS))
@pytest.mark.parametrize("T,N,K", [(1, 20, 32), (5, 33, 160), (2, 100, 1440), (17, 300, 2080), (70, 129, 96)])
def test_linear_odd_columns(name, T, N, K):
    x, w, b, out = run_linear(name, 32, T, N, K, bias=True)
    check(out, *ref.linear(x, w, b, rounded=T >= ref.GEMM_TOKENS))


@pytest.mark.parametrize("name,group", [("int4", 128), ("int4_zp", 32), ("e2m1", 64)])
@pytest.mark.parametrize("T,N,K", [(31, 512, 2048), (64, 1000, 1024), (129, 257, 640), (300, 384, 512), (777, 1100, 1920), (1024, 2048, 4096)])
def test_linear_many_tokens(name, group, T, N, K):
    x, w, b, out = run_linear(name, group, T, N, K, bias=N % 2 == 0)
    check(out, *ref.linear(x, w, b, rounded=T >= ref.GEMM_TOKENS))


@pytest.mark.parametrize("name,group", [("int4", 64), ("int4_zp", 32), ("e2m1", 128)])
@pytest.mark.parametrize("T,N,K", [(9, 20000, 128), (17, 16393, 256), (65, 8200, 384), (1500, 520, 640), (2100, 257, 1152), (4200, 129, 128),
                                   (5000, 640, 896), (10000, 32, 128)])
def test_linear_on_tensor_cores(name, group, T, N, K):
    """Tiles of one row half and of two, several to a CTA, rows past the matrix, ragged token tiles; NaN around the
    result stays."""
    assert ref.linear_rounds(T, N, torch.cuda.get_device_properties(0).multi_processor_count)
    x, w, b, out = run_linear(name, group, T, N, K, bias=N % 2 == 0)
    check(out, *ref.linear(x, w, b, rounded=True))


@pytest.mark.parametrize("T,N,K", [(3000, 640, 384), (5000, 384, 640), (9, 24000, 1152), (777, 5000, 128), (2500, 1000, 2048)])
def test_linear_on_tensor_cores_is_exact_on_integers(T, N, K):
    """Codes -8 .. 7 and tokens with 0, 1 and -1 in at most 32 columns, scales 1: every product, sum and result (at
    most 256) is exact in bf16 and fp32, so the results are equal, whatever the order; and again on every repeat."""
    f = ref.fmt("int4", 128)
    g = torch.Generator(device="cuda").manual_seed(N)
    codes = torch.randint(0, 16, (1, N, K), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.ones(1, N, K // 128, dtype=torch.bfloat16, device="cuda")
    packed = ref.pack("int4", 128, (codes, scales, None))
    w = ref.values("int4", 128, (codes, scales, None))[0]
    x = torch.zeros(T, K, device="cuda")
    cols = torch.randint(0, K, (T, 32), device="cuda", generator=g)
    x.scatter_(1, cols, torch.randint(0, 2, (T, 32), device="cuda", generator=g) * 2.0 - 1)
    want = x.double() @ w.T
    assert float(want.abs().max()) <= 256
    ws = moe.new_w4_linear_workspace(f, T, N, K)
    for _ in range(20):
        out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        moe.moe_w4_linear(f, x.to(torch.bfloat16), packed, None, out, ws)
        assert torch.equal(out.double(), want)
    assert moe.moe_last_device_error(ws) == 0


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_linear_nonfinite_rows_stay_apart(T):
    """NaN and infinities in one token's row reach that row's results only."""
    x = torch.randn(T, 256, device="cuda").to(torch.bfloat16)
    x[T // 2, 5] = float("nan")
    x, w, b, out = run_linear("int4", 32, T, 70, 256, False, x=x)
    keep = torch.arange(T, device="cuda") != T // 2
    assert bool(out[T // 2].isnan().all()) and bool(out[keep].isfinite().all())
    check(out[keep], *ref.linear(x[keep], w, b, rounded=T >= ref.GEMM_TOKENS))


def test_linear_on_tensor_cores_keeps_nonfinite_rows_apart():
    """NaN and infinities in some token rows, those next to tile borders among them, and in one weight row's scale
    reach their own rows and column only."""
    T, N, K = 3000, 640, 256
    f = ref.fmt("e2m1", 64)
    codes, scales, _ = ref.matrices("e2m1", 64, 1, N, K, seed=5)
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    bad = torch.tensor([0, 93, 94, 95, 96, 127, 128, 1500, 2999], device="cuda")
    x[bad, 7] = torch.tensor([float("nan"), float("inf"), float("-inf")] * 3, dtype=torch.bfloat16, device="cuda")
    scales[0, 130, 1] = float("nan")
    ws, out = moe.new_w4_linear_workspace(f, T, N, K), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_w4_linear(f, x, ref.pack("e2m1", 64, (codes, scales, None)), None, out, ws)
    row, col = torch.ones(T, dtype=torch.bool, device="cuda"), torch.ones(N, dtype=torch.bool, device="cuda")
    row[bad], col[130] = False, False
    assert bool(out[:, 130].isnan().all()) and bool((codes[0, :, 7] % 8 == 0).any())
    assert not bool(out[bad][:, codes[0, :, 7] % 8 != 0].isfinite().any())
    w = ref.values("e2m1", 64, (codes, scales, None))[0]
    want, bound = ref.linear(x[row], w[col], None, rounded=True)
    check(out[row][:, col], want, bound)


def test_tensor_core_paths_in_one_graph():
    """A linear layer and a layer of many tokens captured together, replayed on new inputs, and between eager calls on the
    same workspaces."""
    f, T, N, K = ref.fmt("int4", 64), 3000, 640, 512
    packed = ref.pack("int4", 64, ref.matrices("int4", 64, 1, N, K, seed=3))
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    ws, out = moe.new_w4_linear_workspace(f, T, N, K), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    L = W4Layer((400, 640, 9, 2, 192, 64), "int4", 64, seed=11, bias=True)
    lws, lout = moe.new_workspace(L.dims), torch.empty_like(L.x)

    def both(o, lo):
        moe.moe_w4_linear(f, x, packed, None, o, ws)
        moe.moe_forward_w4(L.dims, f, L.x, L.W, L.residual, lo, lws)

    both(out, lout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(2):
            both(out, lout)
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, K, generator=g, device="cuda"))
        L.residual.copy_(torch.randn(L.residual.shape, generator=g, device="cuda"))
        out.fill_(float("nan"))
        lout.fill_(float("nan"))
        graph.replay()
        want, lwant = torch.empty_like(out), torch.empty_like(lout)
        both(want, lwant)
        assert torch.equal(out, want) and torch.equal(lout, lwant)
    assert moe.moe_last_device_error(ws) == 0 and moe.moe_last_device_error(lws) == 0


def test_tensors_of_another_device_are_refused(monkeypatch):
    f = ref.fmt("int4", 32)
    w = torch.zeros(16, 128, dtype=torch.bfloat16, device="cuda")
    packed, ws = moe.new_w4(f, 16, 128), moe.new_w4_linear_workspace(f, 1, 16, 128)
    x, out = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: moe.moe_w4_quantize(f, w, packed), lambda: moe.moe_w4_dequantize(f, packed, w),
                 lambda: moe.moe_w4_linear(f, x, packed, None, out, ws)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_linear_on_two_streams_at_once():
    """Two layers in flight together, each with its own workspace and output, on the streaming and the tensor-core path."""
    f = ref.fmt("int4", 64)
    cases = []
    for T, N, K in ((5, 4096, 2048), (40, 24000, 512), (1000, 2048, 1024), (3000, 640, 512)):
        packed = ref.pack("int4", 64, ref.matrices("int4", 64, 1, N, K, seed=N))
        x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
        ws = [moe.new_w4_linear_workspace(f, T, N, K) for _ in range(2)]
        out = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        alone = torch.empty_like(out[0])
        moe.moe_w4_linear(f, x, packed, None, alone, ws[0])
        cases.append((packed, x, ws, out, alone))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i, s in enumerate(streams):
            for packed, x, ws, out, _ in (cases if i == 0 else cases[::-1]):
                moe.moe_w4_linear(f, x, packed, None, out[i], ws[i], s)
    torch.cuda.synchronize()
    for packed, x, ws, out, alone in cases:
        assert torch.equal(out[0], alone) and torch.equal(out[1], alone)
        assert all(moe.moe_last_device_error(w) == 0 for w in ws)


def test_linear_repeats_bit_for_bit_and_in_graphs():
    f = ref.fmt("int4", 64)
    for T in (1, 7, 33, 260):
        m = ref.matrices("int4", 64, 1, 520, 1024, seed=T)
        p = ref.pack("int4", 64, m)
        x = torch.randn(T, 1024, device="cuda").to(torch.bfloat16)
        ws, out = moe.new_w4_linear_workspace(f, T, 520, 1024), torch.empty(T, 520, dtype=torch.bfloat16, device="cuda")
        moe.moe_w4_linear(f, x, p, None, out, ws)
        first = out.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            moe.moe_w4_linear(f, x, p, None, out, ws)
        out.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_quantize_then_linear_on_one_stream():
    """Weights written and used without any other work between."""
    f = ref.fmt("e2m1", 32)
    x = torch.randn(4, 2048, device="cuda").to(torch.bfloat16)
    ws = moe.new_w4_linear_workspace(f, 4, 4096, 2048)
    packed, out = moe.new_w4(f, 4096, 2048), torch.empty(4, 4096, dtype=torch.bfloat16, device="cuda")
    for i in range(4):
        w = torch.randn(4096, 2048, device="cuda").to(torch.bfloat16)
        torch.cuda.synchronize()
        moe.moe_w4_quantize(f, w, packed)
        moe.moe_w4_linear(f, x, packed, None, out, ws)
        back = torch.empty_like(w)
        moe.moe_w4_dequantize(f, packed, back)
        codes = ref.quantize("e2m1", 32, w[None])
        check(out, *ref.linear(x, ref.values("e2m1", 32, codes)[0], None))


# ---------------------------------------------------------------------------------------- layer

class W4Layer:
    def __init__(self, dims, name, group, seed, bias=False, device="cuda"):
        T, H, E, K, I, Is = dims[:6]
        self.dims, self.name, self.group = dims, name, group
        g = torch.Generator(device=device).manual_seed(seed)
        self.m = {"gate_up": ref.matrices(name, group, E, 2 * I, H, seed + 1), "down": ref.matrices(name, group, E, H, I, seed + 2),
                  "shared_gate_up": ref.matrices(name, group, 1, 2 * Is, H, seed + 3),
                  "shared_down": ref.matrices(name, group, 1, H, Is, seed + 4)}
        self.v = {k: ref.values(name, group, t) for k, t in self.m.items()}
        self.router_w = (torch.randn(E, H, generator=g, device=device) * 0.02).to(torch.bfloat16)
        self.router_b = torch.randn(E, generator=g, device=device).to(torch.bfloat16) if bias else None
        self.shared_gate = (torch.randn(1, H, generator=g, device=device) / H ** 0.5).to(torch.bfloat16)
        self.x = torch.randn(T, H, generator=g, device=device).to(torch.bfloat16)
        self.residual = torch.randn(T, H, generator=g, device=device).to(torch.bfloat16)
        self.W = moe.Weights(self.router_w, self.router_b, *(ref.pack(name, group, self.m[k], k.endswith("gate_up"))
                                                             for k in ("gate_up", "down", "shared_gate_up", "shared_down")),
                             self.shared_gate)
        # tokens whose scores nearly tie have two right answers: drawn again
        for _ in range(50):
            s = self.x.double() @ self.router_w.double().T + (0 if self.router_b is None else self.router_b.double())
            top = s.sort(dim=1, descending=True).values[:, :K + 1]
            bad = (top[:, :-1] - top[:, 1:]).amin(1) < 1e-3 if top.shape[1] > 1 else torch.zeros(T, dtype=torch.bool, device=device)
            if not bool(bad.any()):
                break
            self.x[bad] = torch.randn(int(bad.sum()), H, generator=g, device=device).to(torch.bfloat16)

    def reference(self, residual=True, gemm_tokens=256):
        big = self.dims[0] >= gemm_tokens
        return ref.layer(self.dims, self.x, self.router_w, self.router_b, self.shared_gate, self.v["gate_up"], self.v["down"],
                         self.v["shared_gate_up"][0], self.v["shared_down"][0], self.residual if residual else None,
                         weight_half=ref.HALF if big else 0.0, y_half=ref.HALF if big else 0.0)

    def run(self, residual=True, ws=None, out=None):
        f = ref.fmt(self.name, self.group)
        ws = moe.new_workspace(self.dims) if ws is None else ws
        out = torch.empty_like(self.x) if out is None else out
        moe.moe_forward_w4(self.dims, f, self.x, self.W, self.residual if residual else None, out, ws)
        assert moe.moe_last_device_error(ws) == 0
        return out


@pytest.mark.parametrize("name,group", FG)
@pytest.mark.parametrize("T", [1, 2, 8, 33])
def test_layer_tiny(name, group, T):
    L = W4Layer((T, 512, 32, 4, 128, 128), name, group, seed=T)
    check(L.run(), *L.reference())
    check(L.run(residual=False), *L.reference(residual=False))


@pytest.mark.parametrize("dims,name,group", [
    ((1, 2048, 64, 8, 512, 512), "int4", 32), ((1, 2048, 256, 8, 512, 512), "e2m1", 32), ((1, 2048, 256, 8, 512, 512), "int4_zp", 128),
    ((1, 2048, 16, 1, 512, 512), "int4", 64), ((8, 2048, 64, 8, 512, 512), "e2m1", 32), ((64, 2048, 64, 8, 512, 512), "int4_zp", 128),
    ((255, 2048, 16, 2, 512, 512), "int4", 64), ((255, 128, 8, 8, 64, 64), "int4", 64), ((5, 1280, 21, 3, 192, 448), "int4", 64),
    ((13, 384, 7, 7, 320, 64), "int4_zp", 32), ((3, 4096, 8, 2, 1024, 2048), "e2m1", 128), ((20, 128, 1, 1, 64, 2048), "int4", 32),
    ((256, 512, 32, 4, 128, 128), "int4", 32), ((300, 2048, 32, 8, 512, 512), "e2m1", 64), ((777, 640, 11, 3, 192, 320), "int4_zp", 64),
    ((1000, 128, 8, 2, 64, 64), "int4", 32), ((600, 2048, 256, 8, 512, 512), "int4", 128), ((512, 2304, 9, 8, 576, 128), "e2m1", 32)],
    ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v))
def test_layer_shapes(dims, name, group):
    L = W4Layer(dims, name, group, seed=sum(dims), bias=dims[2] % 2 == 1)
    check(L.run(), *L.reference())


@pytest.mark.parametrize("dims", [(300, 512, 4, 1, 128, 64), (700, 640, 5, 1, 64, 192), (1000, 2048, 16, 1, 512, 512), (256, 128, 1, 1, 64, 64)],
                         ids=lambda v: "x".join(map(str, v)))
def test_layer_of_one_expert_a_token(dims):
    """On the tensor cores Y is not rounded where K is 1: the bound without those roundings holds."""
    L = W4Layer(dims, "e2m1", 64, seed=sum(dims), bias=True)
    want, bound = ref.layer(L.dims, L.x, L.router_w, L.router_b, L.shared_gate, L.v["gate_up"], L.v["down"], L.v["shared_gate_up"][0],
                            L.v["shared_down"][0], L.residual, weight_half=ref.HALF, y_half=0.0)
    ws = moe.new_workspace(L.dims)
    first = L.run(ws=ws)
    check(first, want, bound)
    for _ in range(5):
        assert torch.equal(L.run(ws=ws), first)


@pytest.mark.parametrize("dims", [(777, 640, 11, 3, 192, 320), (300, 384, 7, 7, 64, 64), (2000, 640, 64, 2, 64, 192), (1024, 1408, 40, 4, 704, 128),
                                  (1500, 256, 24, 3, 64, 704), (900, 1280, 11, 4, 192, 320)],
                         ids=lambda v: "x".join(map(str, v)))
def test_layer_repeats_bit_for_bit_with_skewed_experts(dims):
    """Experts of a few tokens next to experts of nearly all, row tiles of one half and of two, several tiles to a
    CTA: the same result every time, also where every intermediate held NaN before."""
    L = W4Layer(dims, "int4_zp", 64, seed=sum(dims), bias=True)
    ws = moe.new_workspace(L.dims)
    first = L.run(ws=ws)
    check(first, *L.reference())
    for _ in range(25):
        for tap in (0, 1):
            at, n = moe.moe_workspace_tap(L.dims, tap)
            ws.view(torch.uint8)[at:at + n] = 255
        assert torch.equal(L.run(ws=ws), first)


@pytest.mark.parametrize("T", [1, 8, 40, 256])
def test_layer_over_its_residual_repeated_and_in_graphs(T):
    L = W4Layer((T, 2048, 32, 8, 512, 512), "int4", 32, seed=T)
    want, bound = L.reference()
    ws = moe.new_workspace(L.dims)
    first = L.run(ws=ws)
    check(first, want, bound)
    for _ in range(3):
        assert torch.equal(L.run(ws=ws), first)
    over = L.residual.clone()
    moe.moe_forward_w4(L.dims, ref.fmt("int4", 32), L.x, L.W, over, over, ws)
    assert torch.equal(over, first)
    out = torch.zeros_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            moe.moe_forward_w4(L.dims, ref.fmt("int4", 32), L.x, L.W, L.residual, out, ws)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and moe.moe_last_device_error(ws) == 0


def test_layer_routes_as_moe_forward_does():
    """Same workspace, same taps: ids, weights and shared gate equal moe_forward's on bf16 weights."""
    T, H, E, K, I, Is = dims = (24, 512, 32, 4, 128, 128)
    L = W4Layer(dims, "int4", 32, seed=5)
    ws = moe.new_workspace(dims)
    got, taps = L.run(ws=ws), {}
    for tap in (2, 3, 4):
        off, nb = moe.moe_workspace_tap(dims, tap)
        taps[tap] = ws[off:off + nb].clone()
    dense = {}
    for k, rows, cols in (("gate_up", 2 * I, H), ("down", H, I), ("shared_gate_up", 2 * Is, H), ("shared_down", H, Is)):
        n = L.m[k][0].shape[0]
        dense[k] = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
        moe.moe_w4_dequantize(ref.fmt("int4", 32), getattr(L.W, k), dense[k], k.endswith("gate_up"))
    W = moe.Weights(L.router_w, None, dense["gate_up"], dense["down"], dense["shared_gate_up"], dense["shared_down"], L.shared_gate)
    out = torch.empty_like(L.x)
    moe.moe_forward(dims, L.x, W, L.residual, out, ws)
    for tap in (2, 3, 4):
        off, nb = moe.moe_workspace_tap(dims, tap)
        assert torch.equal(taps[tap], ws[off:off + nb])
    want, bound = ref.layer(dims, L.x, L.router_w, None, L.shared_gate, L.v["gate_up"], L.v["down"], L.v["shared_gate_up"][0],
                            L.v["shared_down"][0], L.residual, weight_half=ref.HALF)
    check(out, want, bound)  # the bf16 layer on the weights rounded to bf16
    check(got, *L.reference())


def test_layer_flags_nonfinite_scores():
    L = W4Layer((4, 512, 32, 4, 128, 128), "int4", 32, seed=9)
    L.x[2, 7] = float("inf")
    ws, out = moe.new_workspace(L.dims), torch.empty_like(L.x)
    moe.moe_forward_w4(L.dims, ref.fmt("int4", 32), L.x, L.W, L.residual, out, ws)
    assert moe.moe_last_device_error(ws) == 7


def test_quantised_stack_of_layers():
    """bf16 weights quantised, two layers chained by RMSNorm and residual, as a decoder runs them."""
    T, H, E, K, I, Is = dims = (6, 512, 16, 4, 128, 128)
    f = ref.fmt("int4", 32)
    ws = moe.new_workspace(dims)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    for layer in range(2):
        g = torch.Generator(device="cuda").manual_seed(layer)
        rnd = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
        dense = {"gate_up": rnd(E, 2 * I, H, std=H ** -0.5), "down": rnd(E, H, I, std=I ** -0.5),
                 "shared_gate_up": rnd(1, 2 * Is, H, std=H ** -0.5), "shared_down": rnd(1, H, Is, std=Is ** -0.5)}
        router, gate = rnd(E, H, std=0.02), rnd(1, H, std=H ** -0.5)
        packed = {}
        for k, w in dense.items():
            packed[k] = moe.new_w4(f, w.shape[1], w.shape[2], w.shape[0])
            moe.moe_w4_quantize(f, w, packed[k], moe.W4_GATE_UP if k.endswith("gate_up") else moe.W4_ROWS)
        xn, out = torch.empty_like(x), torch.empty_like(x)
        moe.moe_rmsnorm(dims, x, None, 1e-6, xn)
        moe.moe_forward_w4(dims, f, xn, moe.Weights(router, None, packed["gate_up"], packed["down"], packed["shared_gate_up"],
                                                    packed["shared_down"], gate), x, out, ws)
        ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
        off, nb = moe.moe_workspace_tap(dims, 3)
        ids = ws[off:off + nb].view(torch.int32).view(T, K)
        v = {k: ref.values("int4", 32, ref.quantize("int4", 32, w)) for k, w in dense.items()}
        check(out, *ref.layer(dims, xn, router, None, gate, v["gate_up"], v["down"], v["shared_gate_up"][0], v["shared_down"][0], x,
                              ids=ids))
        x = out


def test_layer_one_workspace_for_many_calls():
    """One workspace for calls of several token counts and both kinds of weights, in turn."""
    dims = lambda T: (T, 512, 32, 4, 128, 128)  # noqa: E731
    ws = moe.new_workspace(dims(300))
    layers = {T: W4Layer(dims(T), "int4", 32, seed=70 + T) for T in (1, 3, 8, 20, 300)}
    dense = {}
    L = layers[1]
    for k, rows, cols in (("gate_up", 256, 512), ("down", 512, 128), ("shared_gate_up", 256, 512), ("shared_down", 512, 128)):
        dense[k] = torch.empty(L.m[k][0].shape[0], rows, cols, dtype=torch.bfloat16, device="cuda")
        moe.moe_w4_dequantize(ref.fmt("int4", 32), getattr(L.W, k), dense[k], k.endswith("gate_up"))
    W = moe.Weights(L.router_w, None, dense["gate_up"], dense["down"], dense["shared_gate_up"], dense["shared_down"], L.shared_gate)
    first = {}
    for _ in range(4):
        for T, M in layers.items():
            out = M.run(ws=ws)
            if T not in first:
                check(out, *M.reference())
                first[T] = out
            assert torch.equal(out, first[T])
            moe.moe_forward(dims(1), L.x, W, L.residual, torch.empty_like(L.x), ws)
    assert moe.moe_last_device_error(ws) == 0


def test_layer_wait_timeout_ends_the_call():
    """A CTA that keeps its router scores back: the call ends with the timeout in the workspace."""
    L = W4Layer((1, 512, 32, 4, 128, 128), "int4", 32, seed=1)
    ws, out = moe.new_workspace(L.dims), torch.empty_like(L.x)
    moe.moe_test_set_wait(20_000_000, moe.TEST_SUPPRESS_SCORE)
    try:
        moe.moe_forward_w4(L.dims, ref.fmt("int4", 32), L.x, L.W, L.residual, out, ws)
        assert moe.moe_last_device_error(ws) == 6
    finally:
        moe.moe_test_set_wait()
    moe.moe_workspace_init(ws)
    check(L.run(ws=ws), *L.reference())
