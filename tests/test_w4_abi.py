"""Host-side checks of the 4-bit weight entry points: sizes, and refusals before any launch (the
fake device addresses are never dereferenced)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from sparse_moe_ffn_router_gb300 import binding
from sparse_moe_ffn_router_gb300.binding import CWeights, Dims, W4Format

A = 0x10000000
FULL = (64, 2048, 256, 8, 512, 512)


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def F(fmt=0, group=32):
    return ctypes.byref(W4Format(fmt, group))


@pytest.mark.parametrize("fmt,group,record", [(0, 32, 1152), (0, 64, 1088), (0, 128, 1056), (1, 32, 1216), (1, 64, 1120),
                                              (1, 128, 1072), (2, 32, 1152), (2, 64, 1088), (2, 128, 1056)])
def test_sizes(lib, fmt, group, record):
    assert lib.moe_w4_size(F(fmt, group), 1, 16, 128) == record
    assert lib.moe_w4_size(F(fmt, group), 3, 17, 256) == 3 * 2 * 2 * record  # rows padded to strips
    assert lib.moe_w4_size(F(fmt, group), 0, 16, 128) == 0
    assert lib.moe_w4_size(F(fmt, group), 256, 1024, 2048) == 256 * 64 * 16 * record
    assert lib.moe_w4_size(F(fmt, group), 1, 1, group) == record  # columns padded to records
    assert lib.moe_w4_size(F(fmt, group), 1, 1, 65536) == 512 * record


def test_size_refuses(lib):
    for f, n, r, c in [(F(3), 1, 16, 128), (F(-1), 1, 16, 128), (F(0, 16), 1, 16, 128), (F(0, 256), 1, 16, 256), (None, 1, 16, 128),
                       (F(), -1, 16, 128), (F(), 1, 0, 128), (F(), 1, 16, 0), (F(), 1, 16, 48), (F(0, 128), 1, 16, 192),
                       (F(), 1, 16, 65568), (F(), 1, 2 ** 31 - 1, 65536), (F(), 2 ** 20, 2 ** 20, 2048)]:
        assert lib.moe_w4_size(f, n, r, c) == 0
        assert lib.moe_w4_linear_workspace_size(f, 1, r, c) == 0 or n != 1


def test_largest_row_counts(lib):
    """The largest counts whose roundings to strips and tiles fit 32 bits, and one more."""
    most = 2 ** 31 - 256
    for rows in (most, most - 1, most - 15, most - 16):
        assert lib.moe_w4_size(F(), 1, rows, 32) == -(-rows // 16) * 1152
    for rows in (most + 1, 2 ** 31 - 16, 2 ** 31 - 1):
        assert lib.moe_w4_size(F(), 1, rows, 32) == 0
        assert _quantize(lib, n=1, rows=rows, cols=32) == 2 and _dequantize(lib, n=1, rows=rows, cols=32) == 2
        assert lib.moe_w4_pack(F(), 1, rows, 32, 0, A, A, None, A + 0x1000000, 1 << 60, None) == 2
    ws = lib.moe_w4_linear_workspace_size(F(), most, 16, 32)
    assert ws > 0 and lib.moe_w4_linear_workspace_size(F(), most + 1, 16, 32) == 0

    def linear(T, N):
        return lib.moe_w4_linear(F(), T, N, 32, None, A, 1 << 60, None, A + 0x200000, A + 0x300000, ws, None)

    assert linear(most, 16) == 1 and linear(16, most) == 1  # past the sizes, refused for the missing x
    for big in (most + 1, 2 ** 31 - 128, 2 ** 31 - 1):
        assert linear(big, 16) == 2 and linear(16, big) == 2


def _quantize(lib, f=None, n=2, rows=32, cols=256, layout=0, w=A, packed=A + 0x1000000, nbytes=1 << 20):
    return lib.moe_w4_quantize(f or F(), n, rows, cols, layout, w, packed, nbytes, None)


def _dequantize(lib, f=None, n=2, rows=32, cols=256, layout=0, w=A, packed=A + 0x1000000, nbytes=1 << 20):
    return lib.moe_w4_dequantize(f or F(), n, rows, cols, layout, packed, nbytes, w, None)


@pytest.mark.parametrize("call", [_quantize, _dequantize])
def test_conversions_refuse(lib, call):
    assert call(lib, f=F(3)) == 1 and call(lib, f=F(0, 48)) == 1
    assert call(lib, layout=2) == 1 and call(lib, n=-1) == 1
    assert call(lib, rows=0) == 2 and call(lib, cols=40) == 2 and call(lib, f=F(0, 128), cols=320) == 2
    assert call(lib, layout=1, rows=24) == 2  # gate and up blocks of 8 rows
    assert call(lib, w=None) == 1 and call(lib, packed=None) == 1
    assert call(lib, w=A + 2) == 3 and call(lib, packed=A + 0x1000008) == 3
    need = lib.moe_w4_size(F(), 2, 32, 256)
    assert call(lib, nbytes=need - 1) == 4
    assert call(lib, packed=A + 0x100) == 1  # overlap
    assert call(lib, n=0, w=None, packed=None, nbytes=0) == 0  # nothing to do


def test_pack_refuses(lib):
    def call(f=None, codes=A, scales=A + 0x100000, zeros=None, packed=A + 0x1000000, nbytes=1 << 20, n=2, rows=32):
        return lib.moe_w4_pack(f or F(), n, rows, 256, 0, codes, scales, zeros, packed, nbytes, None)

    assert call(codes=None) == 1 and call(scales=None) == 1 and call(packed=None) == 1
    assert call(zeros=A + 0x200000) == 1          # zero points without the format that has them
    assert call(f=F(1)) == 1                      # and the other way round
    assert call(codes=A + 4) == 3 and call(scales=A + 0x100002) == 3 and call(f=F(1), zeros=A + 0x200001) == 3
    assert call(nbytes=100) == 4 and call(scales=A + 0x1000000) == 1 and call(n=0, codes=None) == 0


def test_linear_refuses(lib):
    size = lib.moe_w4_size(F(), 1, 64, 256)
    ws = lib.moe_w4_linear_workspace_size(F(), 4, 64, 256)
    assert ws > 0 and ws % 256 == 0

    def call(f=None, T=4, N=64, K=256, x=A, packed=A + 0x100000, pb=size, bias=None, out=A + 0x200000, wsp=A + 0x300000, wb=ws):
        return lib.moe_w4_linear(f or F(), T, N, K, x, packed, pb, bias, out, wsp, wb, None)

    assert call(f=F(7)) == 1 and call(T=-1) == 1
    assert call(N=0) == 2 and call(K=100) == 2 and call(K=65568, pb=1 << 30) == 2
    assert call(x=None) == 1 and call(packed=None) == 1 and call(out=None) == 1 and call(wsp=None) == 1
    assert call(x=A + 2) == 3 and call(packed=A + 0x100004) == 3 and call(out=A + 0x200002) == 3 and call(wsp=A + 0x300008) == 3
    assert call(bias=A + 0x400001) == 3
    assert call(pb=size - 1) == 4 and call(wb=ws - 1) == 4
    assert call(out=A + 0x10) == 1 and call(out=A + 0x100010) == 1 and call(bias=A + 0x200000) == 1  # overlaps
    assert call(T=0, x=None, out=None) == 0


def test_forward_refuses(lib):
    names = [f[0] for f in CWeights._fields_]

    def call(dims=FULL, f=None, x=A + 0x100000, w=None, res=None, out=A + 0x800000, ws=A + 0x1000000, wsb=None, **over):
        d = Dims(*dims)
        c = CWeights(*[{**{n: None if n == "router_b" else A for n in names}, **over}[n] for n in names])
        return lib.moe_forward_w4(ctypes.byref(d), f, x, ctypes.byref(c), res, out, ws,
                                  lib.moe_workspace_size(ctypes.byref(d)) if wsb is None else wsb, None)

    assert call(f=None) == 1 and call(f=F(3)) == 1 and call(f=F(0, 33)) == 1
    assert call(f=F(), x=None) == 1 and call(f=F(), down=None) == 1 and call(f=F(), out=None) == 1
    assert call(f=F(), gate_up=A + 8) == 3 and call(f=F(), x=A + 0x100002) == 3
    assert call(f=F(), out=A + 0x100000) == 1 and call(f=F(), wsb=100) == 4
    assert call(f=F(0, 128), dims=(64, 2048, 256, 8, 448, 512)) == 2  # I is no multiple of the group
    assert call(f=F(0, 128), dims=(64, 2048, 256, 8, 512, 320)) == 2
    assert call(f=F(), dims=(64, 2000, 256, 8, 512, 512)) == 2
    assert call(f=F(), dims=(0, 2048, 256, 8, 512, 512), x=None, out=None) == 0


def test_binding_checks():
    f = W4Format(0, 32)
    assert binding.moe_w4_size(f, 16, 128) == 1152
    w = torch.zeros(16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.moe_w4_quantize(f, w, torch.zeros(1152, dtype=torch.uint8))  # not on the GPU
    with pytest.raises(TypeError):
        binding.moe_w4_quantize(f, w.float(), torch.zeros(1152, dtype=torch.uint8))
    with pytest.raises(ValueError):
        binding.moe_w4_linear(f, torch.zeros(3, 128, dtype=torch.bfloat16), w, None, torch.zeros(2, 16, dtype=torch.bfloat16), w)
    with pytest.raises(binding.MoEError):
        binding.new_w4(W4Format(9, 32), 16, 128, device="cpu")
    with pytest.raises(TypeError):  # bf16 weights where packed ones are expected
        binding.moe_forward_w4((1, 128, 8, 2, 64, 64), f, w, binding.Weights(*[w] * 7), None, w, w)
    with pytest.raises(ValueError):  # packed tensors too small for the dims
        binding.moe_forward_w4((1, 128, 8, 2, 64, 64), f, w, binding.Weights(*[torch.zeros(16, dtype=torch.uint8)] * 7), None, w, w)


def test_forward_binding_checks_every_tensor():
    """Rows, types and sizes that do not fit the dims are refused before the library sees a pointer."""
    f, dims = W4Format(0, 32), (5, 128, 8, 2, 64, 64)
    T, H, E, K, I, Is = dims

    def bf16(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16)

    def packed(n, rows, cols):
        return torch.zeros(n, binding.moe_w4_size(f, rows, cols), dtype=torch.uint8)

    def call(residual=None, dims=dims, **over):
        t = dict(x=bf16(T, H), out=bf16(T, H), router_w=bf16(E, H), router_b=bf16(E), shared_gate=bf16(1, H),
                 gate_up=packed(E, 2 * I, H), down=packed(E, H, I), shared_gate_up=packed(1, 2 * Is, H), shared_down=packed(1, H, Is))
        t.update(over)
        x, out = t.pop("x"), t.pop("out")
        binding.moe_forward_w4(dims, f, x, binding.Weights(**t), residual, out, torch.zeros(1 << 20, dtype=torch.uint8))

    for name, t in (("x", bf16(T - 1, H)), ("out", bf16(T, H - 1)), ("residual", bf16(T * H - 1)), ("router_w", bf16(E - 1, H)),
                    ("router_b", bf16(E - 1)), ("shared_gate", bf16(H - 1))):
        with pytest.raises(ValueError, match=f"{name} holds"):
            call(**{name: t})
    for name, t in (("x", bf16(T, H).float()), ("out", bf16(T, H).half()), ("residual", bf16(T, H).float()), ("router_w", bf16(E, H).float()),
                    ("router_b", bf16(E).float()), ("shared_gate", bf16(1, H).float())):
        with pytest.raises(TypeError, match=f"{name} must be"):
            call(**{name: t})
    for name in ("x", "out", "router_w", "shared_gate"):
        with pytest.raises(TypeError, match=f"{name} is missing"):
            call(**{name: None})
    for name in ("gate_up", "down", "shared_gate_up", "shared_down"):
        with pytest.raises(ValueError, match="packed weights of"):
            call(**{name: torch.zeros(1000, dtype=torch.uint8)})
    with pytest.raises(ValueError, match="GPU only"):  # everything fits: only the device is wrong
        call(router_b=None)


@pytest.mark.parametrize("dims,extra", [((300, 512, 4, 1, 128, 64), 300 * 2 * 512 * 2), ((256, 2048, 8, 1, 64, 512), 256 * 2 * 2048 * 2),
                                        ((1, 2048, 256, 8, 512, 512), 9 * 256 * 8), ((64, 2048, 256, 8, 512, 512), 0),
                                        ((1000, 2048, 256, 8, 512, 512), 0), ((255, 512, 4, 1, 128, 64), 0)])
def test_workspace_of_both_layers(lib, dims, extra):
    """The 4-bit layer's own part of the workspace (fp32 Y of one expert a token, exchanged h pairs of one token) lies last and
    is asked of that layer only; its tap 1 has the bytes that it writes."""
    T, H, E, K, I, Is = dims
    d, size = Dims(*dims), lib.moe_workspace_size(ctypes.byref(Dims(*dims)))
    w = CWeights(*[None if f[0] == "router_b" else A for f in CWeights._fields_])

    def bf16(nbytes):  # refused for the missing out once the workspace is large enough
        return lib.moe_forward(ctypes.byref(d), A, ctypes.byref(w), None, None, A + 0x1000000, nbytes, None)

    def w4(nbytes):
        return lib.moe_forward_w4(ctypes.byref(d), F(), A, ctypes.byref(w), None, None, A + 0x1000000, nbytes, None)

    assert bf16(size - extra) == 1 and bf16(size - extra - 1) == 4
    assert w4(size) == 1 and w4(size - 1) == 4
    for tap in (0, 2, 3, 4):
        assert binding.moe_w4_workspace_tap(dims, tap) == binding.moe_workspace_tap(dims, tap)
    (at, nb), (at4, nb4) = binding.moe_workspace_tap(dims, 1), binding.moe_w4_workspace_tap(dims, 1)
    assert at == at4 and at % 256 == 0 and nb == T * (K + 1) * H * (4 if T < 256 else 2)
    assert nb4 == T * (K + 1) * H * (4 if T < 256 or K == 1 else 2) and at4 + nb4 <= size
    assert at + nb <= size - extra
    with pytest.raises(binding.MoEError):
        binding.moe_w4_workspace_tap(dims, 5)
    with pytest.raises(binding.MoEError):
        binding.moe_w4_workspace_tap((T, 100, E, K, I, Is), 1)
