"""The few-token layer and the 4-bit weights without a GPU: refusals of the C
entry points and of the binding, workspace sizes, and the packed layout."""
import ctypes
import importlib.util
import types

import numpy as np
import pytest
import torch

import few_reference as ref
import mixture_experts_layer_36_b200 as moe
from mixture_experts_layer_36_b200 import binding

OK, INVALID, WORKSPACE, CUDA, UNSUPPORTED = 0, 1, 2, 3, 4
F = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
S = ctypes.c_void_p(0)
OUTS = [None] * 5


def test_w4_conversion_refusals():
    L = moe.lib()
    for fn in (L.moe_quantize_weights_w4, L.moe_dequantize_weights_w4):
        # (w, E, K, N, group, q, scale) and (q, scale, E, K, N, group, w)
        def call(a=F, b=F, c=F, E=2, K=128, N=192, group=64, fn=fn):
            if fn is L.moe_quantize_weights_w4:
                return fn(a, E, K, N, group, b, c, S)
            return fn(a, b, E, K, N, group, c, S)
        assert call(E=0) == INVALID
        assert call(E=65536) == INVALID
        assert call(K=0) == INVALID
        assert call(N=-64) == INVALID
        assert call(K=96) == UNSUPPORTED
        assert call(N=32) == UNSUPPORTED
        assert call(K=(1 << 20) + 64) == UNSUPPORTED
        assert call(E=65535, K=1 << 15, N=1 << 10) == INVALID     # E K N >= 2^40
        for group in (0, 1, 16, 48, 96, 256):
            assert call(group=group) == UNSUPPORTED
        for kw in ({"a": None}, {"b": None}, {"c": None}, {"a": ODD}, {"b": ODD}, {"c": ODD}):
            assert call(**kw) == INVALID


def _few(w4, T=4, d=128, E=8, k=2, f=256, cf=0.0, group=64, ptrs=None, y=F, ws=F, ws_bytes=None):
    L = moe.lib()
    need = moe.moe_workspace_size_few(T, d, E, k, f) if ws_bytes is None else ws_bytes
    ptrs = [F, F, None] + [F] * (6 if w4 else 3) if ptrs is None else ptrs
    extra = [group] if w4 else []
    fn = L.moe_layer_forward_few_w4 if w4 else L.moe_layer_forward_few
    return fn(*ptrs, T, d, E, k, f, cf, *extra, y, *OUTS, ws, need, S)


@pytest.mark.parametrize("w4", [False, True], ids=["bf16", "w4"])
def test_few_layer_refusals(w4):
    assert _few(w4, T=0, ws_bytes=0) == OK
    assert _few(w4, T=-1, ws_bytes=0) == INVALID
    assert _few(w4, T=33, ws_bytes=1 << 30) == UNSUPPORTED
    assert _few(w4, E=0, ws_bytes=1 << 30) == INVALID
    assert _few(w4, E=257, ws_bytes=1 << 30) == INVALID
    assert _few(w4, k=0, ws_bytes=1 << 30) == INVALID
    assert _few(w4, k=9, ws_bytes=1 << 30) == INVALID
    assert _few(w4, E=1, k=2, ws_bytes=1 << 30) == INVALID
    assert _few(w4, d=96, ws_bytes=1 << 30) == UNSUPPORTED
    assert _few(w4, f=32, ws_bytes=1 << 30) == UNSUPPORTED
    assert _few(w4, f=0, ws_bytes=1 << 30) == INVALID
    assert _few(w4, cf=-1.0) == INVALID
    assert _few(w4, cf=float("nan")) == INVALID
    assert _few(w4, cf=float("inf")) == INVALID
    need = moe.moe_workspace_size_few(4, 128, 8, 2, 256)
    assert need > 0
    assert _few(w4, ws_bytes=need - 1) == WORKSPACE
    n = 9 if w4 else 6
    for i in [0, 1, *range(3, n)]:
        for bad in (None, ODD):
            ptrs = [F, F, None] + [F] * (n - 3)
            ptrs[i] = bad
            assert _few(w4, ptrs=ptrs) == INVALID, i
    for bad in (None, ODD):
        assert _few(w4, y=bad) == INVALID
        assert _few(w4, ws=bad) == INVALID
    if w4:
        for group in (0, 16, 33, 256, -64):
            assert _few(w4, group=group) == UNSUPPORTED


def test_workspace_sizes():
    size = moe.moe_workspace_size_few
    for bad in ((33, 128, 8, 2, 256), (4, 100, 8, 2, 256), (4, 128, 8, 2, 100),
                (4, 128, 300, 2, 256), (4, 128, 8, 9, 256), (-1, 128, 8, 2, 256)):
        assert size(*bad) == 0, bad
    assert size(1, 7168, 256, 8, 2048) > 0
    # grows with the batch, and stays far below the weights of one expert
    assert size(32, 7168, 256, 8, 2048) >= size(1, 7168, 256, 8, 2048)
    assert size(32, 7168, 256, 8, 2048) < 3 * 7168 * 2048 * 2
    assert binding.MOE_FEW_MAX_TOKENS == 32


def test_packed_places_cover_every_nibble_once():
    for K, N in ((64, 64), (192, 128), (128, 320)):
        kk, nn = np.meshgrid(np.arange(K), np.arange(N), indexing="ij")
        byte, shift = ref.place(kk, nn, K)
        at = np.sort((byte * 2 + shift // 4).reshape(-1))
        assert np.array_equal(at, np.arange(K * N))
        codes = torch.randint(-8, 8, (2, K, N))
        assert torch.equal(ref.unpack(ref.pack(codes)), codes)


def test_binding_refusals_on_cpu_tensors():
    bf, f32 = torch.bfloat16, torch.float32
    x, wr = torch.zeros(2, 64, dtype=bf), torch.zeros(64, 4, dtype=f32)
    w = torch.zeros(4, 64, 64, dtype=bf)
    with pytest.raises(ValueError):
        moe.moe_layer_forward_few(x, wr, None, w, w, w, 2, 0.0)
    with pytest.raises(ValueError):
        moe.moe_quantize_weights_w4(w)
    with pytest.raises(ValueError):
        moe.moe_dequantize_weights_w4(torch.zeros(4, 1, 1, 2048, dtype=torch.uint8),
                                      torch.zeros(4, 1, 64, dtype=bf))


def test_a_stream_of_another_device_is_refused():
    other = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        binding._run_on(torch.device("cuda", 0), other, None)


def test_current_stream_without_the_raw_handle(monkeypatch):
    """A torch that does not have the private function for a stream's handle."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    asked = []

    def current_stream(index):
        asked.append(index)
        return types.SimpleNamespace(cuda_stream=1234)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    spec = importlib.util.spec_from_file_location(binding.__package__ + ".binding_again",
                                                  binding.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._run_on(torch.device("cuda", 1), None, lambda handle: handle) == 1234
    assert asked == [1]


def test_digits_of_a_bf16_value():
    """The fixed point of the layer on codes (v = rint(x 2^(22 - e)), 2^(e-1) <= largest <
    2^e): every bf16 x down to 2^-14 of the largest is a whole number of units, at 2^-15
    not all are, and what is rounded is off by at most 2^-22 of the largest."""
    sig = 1 + np.arange(128) / 128                       # the significands of bf16
    for largest in sig:                                  # e = 1
        for low in range(0, 20):
            x = sig * 2.0 ** -low
            x = x[x <= largest]
            units = x * 2.0 ** 21
            off = np.abs(np.rint(units) - units) * 2.0 ** -21
            assert (off <= 2.0 ** -22 * largest).all()
            assert (off[x >= 2.0 ** -14 * largest] == 0).all()
    x = 2.0 ** -15 * sig                                 # beside a largest value of 1
    assert (np.rint(x * 2.0 ** 21) != x * 2.0 ** 21).any()
    # three balanced digits, as bytes; a block's sum with codes 16 (u - 8)
    v = np.arange(-(1 << 22), (1 << 22) + 1)
    d0 = (v & 255).astype(np.uint8).view(np.int8).astype(np.int64)
    d1 = ((v - d0) >> 8 & 255).astype(np.uint8).view(np.int8).astype(np.int64)
    d2 = ((v - d0) >> 8) - d1 >> 8
    assert (d0 + 256 * d1 + 65536 * d2 == v).all() and np.abs(d2).max() <= 65
    assert 128 * 128 * 128 == 1 << 21                    # digit -128 by code 0, 128 rows
    v = round((1 + 2.0 ** -6) * 2 ** 21)
    assert ((v >> 8) & 255) == 128                       # the middle digit -128
