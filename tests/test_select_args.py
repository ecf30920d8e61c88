"""Refusals of the expert selection (CPU: no compute call is made, every answer comes from the host's checks of the
arguments)."""
import ctypes

import pytest
import torch

import mixture_experts_layer_10_gb300 as moe
from test_grouped_args import OnDevice

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = [0x10000 * (i + 1) for i in range(8)]


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def cfg(**over):
    a = dict(T=100, E=64, k=6, score="sigmoid", groups=8, top_groups=4, group_top=2, renorm=1, scale=2.5)
    a.update(over)
    return moe.select_config(**a)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=(1 << 24) + 1), dict(E=0, k=1, groups=1, top_groups=1), dict(E=1025, groups=1, top_groups=1), dict(k=0),
    dict(k=33), dict(k=9, top_groups=1), dict(E=4, k=5, groups=1, top_groups=1), dict(groups=0), dict(groups=7), dict(groups=65, E=650),
    dict(groups=-8), dict(top_groups=0), dict(top_groups=9), dict(group_top=0), dict(group_top=3), dict(score=2), dict(score=-1),
    dict(renorm=2), dict(renorm=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(dtype=3), dict(dtype=-1),
])
def test_bad_descriptions(lib, bad):
    c = cfg(**bad)
    assert lib.moe_select(ctypes.byref(c), *P[:4], None) == INVALID
    assert lib.moe_select_bwd(ctypes.byref(c), *P[:4], None) == INVALID


def test_names():
    with pytest.raises(ValueError):
        cfg(score="tanh")
    with pytest.raises(ValueError):
        cfg(dtype=torch.float64)
    assert cfg(top_groups=None).top_groups == 8 and cfg(dtype=torch.bfloat16).dtype == 0


def test_null_and_misaligned_pointers(lib):
    c = cfg()
    for i in range(4):
        for v in (None, P[i] + 2):
            a = list(P[:4])
            a[i] = v
            if not (i == 1 and v is None):   # (there may be no bias)
                assert lib.moe_select(ctypes.byref(c), *a, None) == INVALID, (i, v)
            assert lib.moe_select_bwd(ctypes.byref(c), *a, None) == INVALID, (i, v)
    assert lib.moe_select(ctypes.byref(c), P[0] + 8, *P[1:4], None) == INVALID      # logits: 16 bytes
    assert lib.moe_select_bwd(ctypes.byref(c), *P[:3], P[3] + 4, None) == INVALID   # dlogits: 16 bytes
    assert lib.moe_select(None, *P[:4], None) == INVALID
    assert lib.moe_select_bwd(None, *P[:4], None) == INVALID


def test_router_wgrad_arguments(lib):
    c = moe.config(T=64, d=128, f=256, E=8, k=2)
    ws, _ = moe.moe_workspace_size(c)
    for i in range(3):
        for v in (None, P[i] + 8):
            a = list(P[:5])
            a[i] = v
            assert lib.moe_router_wgrad(ctypes.byref(c), *a, ws, None) == INVALID
    assert lib.moe_router_wgrad(ctypes.byref(c), *P[:3], P[3] + 4, P[4], ws, None) == INVALID
    assert lib.moe_router_wgrad(ctypes.byref(c), *P[:5], ws - 1, None) == WORKSPACE
    assert lib.moe_router_wgrad(None, *P[:5], ws, None) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="answers of a machine without the device")
def test_calls_need_the_device(lib):
    c = cfg()
    assert lib.moe_select(ctypes.byref(c), *P[:4], None) == UNSUPPORTED
    assert lib.moe_select(ctypes.byref(c), P[0], None, P[2] + 4, P[3] + 4, None) == UNSUPPORTED
    assert lib.moe_select_bwd(ctypes.byref(c), *P[:4], None) == UNSUPPORTED
    m = moe.config(T=64, d=128, f=256, E=8, k=2)
    assert lib.moe_router_wgrad(ctypes.byref(m), *P[:3], None, P[4], moe.moe_workspace_size(m)[0], None) == UNSUPPORTED


def test_binding_checks_tensors(monkeypatch):
    """Shapes, types and devices, before a pointer is taken."""
    monkeypatch.setattr(moe, "_current_device", lambda: 1, raising=False)
    called = []
    monkeypatch.setattr(moe, "_call", lambda name, *args: called.append(name))
    f32, i32 = torch.float32, torch.int32
    sel = {"logits": ((100, 64), f32), "bias": ((64,), f32), "idx": ((100, 6), i32), "weights": ((100, 6), f32)}
    bwd = {"logits": ((100, 64), f32), "idx": ((100, 6), i32), "dweights": ((100, 6), f32), "dlogits": ((100, 64), f32)}
    for call, args in ((moe.moe_select, sel), (moe.moe_select_bwd, bwd)):
        def go(over=None, index=1, at=None):
            t = {k: OnDevice(*(over or {}).get(k, a), index if at in (None, k) else 1) for k, a in args.items()}
            call(cfg(), *t.values(), stream=0)
        go()
        with pytest.raises(ValueError, match="logits: "):
            go(index=0)   # all on one device, and not the current one
        for name, (shape, dtype) in args.items():
            with pytest.raises(ValueError):
                go(index=0, at=name)
            with pytest.raises(ValueError, match=name + ": "):
                go({name: ((shape[0] + 1, *shape[1:]), dtype)})
            with pytest.raises(ValueError, match=name + ": "):
                go({name: (shape, torch.float64)})
    assert called == ["moe_select", "moe_select_bwd"]
    with pytest.raises(ValueError, match="logits: "):
        moe.moe_select(cfg(), torch.zeros(100, 64), None, P[0], P[1], stream=0)   # a CPU tensor
