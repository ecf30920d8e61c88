"""Refusals of the 4-bit quantiser and product (CPU: no compute call is made)."""
import ctypes

import pytest
import torch

import mixture_experts_layer_10_gb300 as moe
from test_grouped_args import INVALID, UNSUPPORTED, WORKSPACE, OnDevice, P, cfg


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def test_scale_stride(lib):
    assert [moe.moe_mx_scale_stride(c) for c in (32, 512, 544, 2880, 4096, 65536)] == [16, 16, 32, 96, 128, 2048]
    n = ctypes.c_int32()
    for bad in (0, 16, 48, -32, 65568):
        assert lib.moe_mx_scale_stride(bad, ctypes.byref(n)) == INVALID
    assert lib.moe_mx_scale_stride(32, None) == INVALID


def test_quantiser_arguments(lib):
    for dtype, rows, cols in ((3, 4, 64), (-1, 4, 64), (0, -1, 64), (0, (1 << 28) + 1, 64), (0, 4, 16), (0, 4, 48), (2, 4, 0),
                              (1, 4, 65568)):
        assert lib.moe_quantize_rows_mxf4(P[0], dtype, rows, cols, P[1], P[2], None) == INVALID
    for i in range(3):
        for v in (None, P[i] + 8):
            a = list(P[:3])
            a[i] = v
            assert lib.moe_quantize_rows_mxf4(a[0], 0, 4, 64, a[1], a[2], None) == INVALID


def test_product_arguments(lib):
    for bad in (dict(n_in=72), dict(n_in=16), dict(n_in=48), dict(in_stride=80), dict(n_out=4), dict(dtype=2), dict(groups=0)):
        assert lib.moe_grouped_mm_mxf4(ctypes.byref(cfg(**bad)), *P, 1 << 20, None) == INVALID
    c = cfg()
    for i in range(8):
        for v in (None, P[i] + (8 if i > 1 else 2)):
            a = list(P)
            a[i] = v
            assert lib.moe_grouped_mm_mxf4(ctypes.byref(c), *a, 1 << 20, None) == INVALID, (i, v)
    assert lib.moe_grouped_mm_mxf4(None, *P, 1 << 20, None) == INVALID
    assert lib.moe_grouped_mm_mxf4(ctypes.byref(c), *P, 255, None) == WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="answers of a machine without the device")
def test_calls_need_the_device(lib):
    assert lib.moe_grouped_mm_mxf4(ctypes.byref(cfg(in_stride=96)), *P, 1 << 20, None) == UNSUPPORTED
    assert lib.moe_quantize_rows_mxf4(P[0], 2, 4, 64, P[1], P[2], None) == UNSUPPORTED


def test_binding_checks_tensors(monkeypatch):
    monkeypatch.setattr(moe, "_current_device", lambda: 1, raising=False)
    called = []
    monkeypatch.setattr(moe, "_call", lambda name, *args: called.append(name))
    u8, i32, bf = torch.uint8, torch.int32, torch.bfloat16
    product = {"row_begin": ((4,), i32), "row_end": ((4,), i32), "codes": ((100, 32), u8), "scales": ((100, 16), u8),
               "Wq": ((4, 128, 32), u8), "W_scale": ((4, 128, 16), u8), "y": ((100, 128), bf), "ws": ((1 << 20,), u8)}
    quantiser = {"src": ((4, 128, 64), bf), "codes": ((4, 128, 32), u8), "scales": ((4, 128, 16), u8)}
    for args, call in ((product, lambda *t: moe.moe_grouped_mm_mxf4(cfg(), *t, stream=0)),
                       (quantiser, lambda *t: moe.moe_quantize_rows_mxf4(*t, stream=0))):
        def go(over=None, at=None):
            call(*(OnDevice(*(over or {}).get(k, a), 0 if k == at else 1) for k, a in args.items()))
        go()
        for name, (shape, dtype) in args.items():
            with pytest.raises(ValueError):
                go(at=name)
            if name not in ("ws", "src"):
                with pytest.raises(ValueError, match=name + ": "):
                    go({name: ((shape[0] + 1, *shape[1:]), dtype)})
                with pytest.raises(ValueError, match=name + ": "):
                    go({name: (shape, torch.float64)})
    assert called == ["moe_grouped_mm_mxf4", "moe_quantize_rows_mxf4"]
    with pytest.raises(ValueError):
        moe.moe_quantize_rows_mxf4(torch.zeros(4, 64, dtype=torch.float64), P[0], P[1])
