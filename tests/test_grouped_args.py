"""Refusals of the grouped products (CPU: no compute call is made, every answer comes from the host's
checks of the arguments)."""
import ctypes
import sys
import types

import pytest
import torch

import mixture_experts_layer_10_gb300 as moe

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = [0x10000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def cfg(**over):
    a = dict(rows=100, n_in=64, n_out=128, groups=4)
    a.update(over)
    return moe.grouped_config(**a)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 28) + 1), dict(n_in=0), dict(n_in=4), dict(n_in=60), dict(n_in=65544), dict(n_out=0),
    dict(n_out=12), dict(n_out=65544), dict(groups=0), dict(groups=1025), dict(dtype=2), dict(dtype=-1), dict(dtype=3),
    dict(dw_dtype=1), dict(dtype=1, dw_dtype=0), dict(dw_dtype=3), dict(accumulate=1),
    dict(accumulate=2, dw_dtype=2), dict(accumulate=-1, dw_dtype=2), dict(in_stride=56), dict(in_stride=68),
    dict(out_stride=120), dict(out_stride=130), dict(in_stride=-64), dict(in_stride=(1 << 31) + 8),
])
def test_bad_descriptions(lib, bad):
    c = cfg(**bad)
    n = ctypes.c_size_t()
    assert lib.moe_grouped_workspace_size(ctypes.byref(c), ctypes.byref(n)) == INVALID
    assert lib.moe_grouped_mm(ctypes.byref(c), *P[:6], 1 << 20, None) == INVALID


@pytest.mark.parametrize("good", [dict(), dict(rows=0), dict(n_in=8, n_out=8), dict(n_in=65536), dict(groups=1024),
                                  dict(dtype=1), dict(dw_dtype=2, accumulate=1), dict(in_stride=72, out_stride=256)])
def test_good_descriptions(good):
    assert moe.moe_grouped_workspace_size(cfg(**good)) >= 256


def test_null_and_misaligned_pointers(lib):
    c = cfg()
    for call in (lib.moe_grouped_mm, lib.moe_grouped_mm_dx, lib.moe_grouped_mm_dw):
        for i in range(6):
            for v in (None, P[i] + 2):
                a = list(P[:6])
                a[i] = v
                assert call(ctypes.byref(c), *a, 1 << 20, None) == INVALID, (call.__name__, i, v)
        assert call(None, *P[:6], 1 << 20, None) == INVALID
        assert call(ctypes.byref(c), *P[:6], 255, None) == WORKSPACE
    for i in range(8):
        for v in (None, P[i] + 2):
            a = list(P)
            a[i] = v
            assert lib.moe_grouped_mm_i8(ctypes.byref(c), *a, 1 << 20, None) == INVALID
    assert lib.moe_grouped_workspace_init(ctypes.byref(c), None, 1 << 20, None) == INVALID
    assert lib.moe_grouped_workspace_init(ctypes.byref(c), P[0], 16, None) == WORKSPACE
    assert lib.moe_grouped_workspace_size(ctypes.byref(c), None) == INVALID


def test_i8_shapes(lib):
    for bad in (dict(n_in=72), dict(in_stride=72)):
        assert lib.moe_grouped_mm_i8(ctypes.byref(cfg(**bad)), *P, 1 << 20, None) == INVALID
    for dtype, rows, cols in ((2, 4, 64), (0, -1, 64), (0, 4, 24), (0, 4, 0), (1, 4, 65552)):
        assert lib.moe_quantize_rows_i8(P[0], dtype, rows, cols, P[1], P[2], None) == INVALID
    assert lib.moe_quantize_rows_i8(P[0] + 8, 0, 4, 64, P[1], P[2], None) == INVALID
    assert lib.moe_quantize_rows_i8(P[0], 0, 4, 64, None, P[2], None) == INVALID


def test_segments_arguments(lib):
    c = moe.config(T=64, d=128, f=256, E=8, k=2)
    ws, _ = moe.moe_workspace_size(c)
    assert lib.moe_segments(ctypes.byref(c), None, P[1], P[2], ws, None) == INVALID
    assert lib.moe_segments(ctypes.byref(c), P[0], P[1] + 1, P[2], ws, None) == INVALID
    assert lib.moe_segments(ctypes.byref(c), P[0], P[1], P[2], ws - 1, None) == WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="answers of a machine without the device")
def test_calls_need_the_device(lib):
    c = cfg()
    assert lib.moe_grouped_mm(ctypes.byref(c), *P[:6], 1 << 20, None) == UNSUPPORTED
    assert lib.moe_grouped_mm_i8(ctypes.byref(c), *P, 1 << 20, None) == UNSUPPORTED


def test_binding_checks_tensors():
    """Shapes, types, strides and the device are checked before a pointer is taken."""
    c = cfg()
    b = torch.zeros(4, dtype=torch.int32)
    x, W, y = torch.zeros(100, 64), torch.zeros(4, 128, 64), torch.zeros(100, 128)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="row_begin"):
        moe.moe_grouped_mm(c, b, b, x, W, y, ws, stream=0)   # a CPU tensor
    with pytest.raises(ValueError, match="x: "):
        moe.moe_grouped_mm(c, P[0], P[1], x, P[2], P[3], ws, stream=0)
    with pytest.raises(ValueError):
        moe.grouped_config(4, 64, 64, 1, dtype=torch.float64)


@pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that no device may be given")
def test_scales_may_start_at_any_float(lib):
    """Scales that are part of a larger array: refused only where they are no floats' addresses."""
    c = cfg()
    for i in (3, 5):
        for off, answer in ((4, UNSUPPORTED), (8, UNSUPPORTED), (1, INVALID), (6, INVALID)):
            a = list(P)
            a[i] += off
            assert lib.moe_grouped_mm_i8(ctypes.byref(c), *a, 1 << 20, None) == answer
    for off, answer in ((4, UNSUPPORTED), (2, INVALID)):
        assert lib.moe_quantize_rows_i8(P[0], 0, 4, 64, P[1], P[2] + off, None) == answer


class OnDevice:
    """What the binding asks of a tensor, of one that lies on a CUDA device (no machine needs to have it)."""
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)
        self.nbytes = 1 << 20

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x10000


def test_operands_lie_on_the_current_device(monkeypatch):
    """Operands and the workspace: on a CUDA device, and on the one that the call runs on."""
    monkeypatch.setattr(moe, "_current_device", lambda: 1, raising=False)
    called = []
    monkeypatch.setattr(moe, "_call", lambda name, *args: called.append(name))
    c, bf = cfg(), torch.bfloat16
    args = {"begin": ((4,), torch.int32), "end": ((4,), torch.int32), "x": ((100, 64), bf), "W": ((4, 128, 64), bf),
            "y": ((100, 128), bf), "ws": ((1 << 20,), torch.uint8)}

    def call(**index):
        moe.moe_grouped_mm(c, *(OnDevice(*a, index.get(k, 1)) for k, a in args.items()), stream=0)

    call()
    assert called == ["moe_grouped_mm"]
    with pytest.raises(ValueError, match="ws: "):
        call(**dict.fromkeys(args, 0))   # all on one device, and not the current one
    with pytest.raises(ValueError, match="src: "):
        moe.moe_quantize_rows_i8(OnDevice((100, 64), bf, 0), OnDevice((100, 64), torch.int8, 0),
                                 OnDevice((100,), torch.float32, 0), stream=0)
    for k in args:
        with pytest.raises(ValueError, match="device"):
            call(**{k: 0})
    ws = torch.zeros(1 << 20, dtype=torch.uint8)   # the host's
    on = [OnDevice(*a, 1) for k, a in args.items() if k != "ws"]
    with pytest.raises(ValueError, match="ws: "):
        moe.moe_grouped_mm(c, *on, ws, stream=0)
    with pytest.raises(ValueError, match="ws: "):
        moe.moe_grouped_workspace_init(c, ws, stream=0)
    with pytest.raises(ValueError, match="ws: "):
        moe.moe_segments(moe.config(T=64, d=128, f=256, E=4, k=2), *on[:2], ws, stream=0)
    assert called == ["moe_grouped_mm"]


@pytest.mark.parametrize("over", [dict(dtype=7), dict(dw_dtype=9), dict(dtype=2)])
def test_unknown_types_are_the_librarys_to_refuse(monkeypatch, over):
    """A description with a type that is none gets the library's answer from the binding, as from C."""
    monkeypatch.setattr(moe, "_current_device", lambda: 1)
    c, bf = cfg(**over), torch.bfloat16
    b, ws = OnDevice((4,), torch.int32, 1), OnDevice((1 << 20,), torch.uint8, 1)
    x, dy, dW = OnDevice((100, 64), bf, 1), OnDevice((100, 128), bf, 1), OnDevice((4, 128, 64), bf, 1)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_grouped_mm_dw(c, b, b, dy, x, dW, ws, stream=0)
    assert e.value.code == INVALID


def test_bindings_to_torch_are_published_whole(monkeypatch):
    """Another thread that finds the table of types finds the other bindings too: a binding that stops half
    way has published no table."""
    for name in ("_holds", "_current_device", "_current_stream"):
        monkeypatch.setattr(moe, name, None)
    half = types.SimpleNamespace(**{n: getattr(torch, n) for n in ("bfloat16", "float16", "float32", "int8", "int16",
                                                                    "uint16", "int32")})   # and no _C
    monkeypatch.setitem(sys.modules, "torch", half)
    with pytest.raises(AttributeError):
        moe._bind_torch()
    assert moe._holds is None and moe._current_stream is None
