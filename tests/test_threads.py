"""Calls from host threads that have not used CUDA before (GPU): the library's first call in such a thread
builds tensor maps before anything else has made a context current there."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import synth
from test_grouped import dev_i32, rand

pytestmark = pytest.mark.gpu


def in_new_thread(call):
    """call() in a thread of its own, after all work before it; what it raised is raised here."""
    raised = []

    def body():
        try:
            call()
        except Exception as err:   # noqa: BLE001 (handed on)
            raised.append(err)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    if raised:
        raise raised[0]


@pytest.mark.parametrize("op", ["mm", "few rows", "dx", "dw", "i8", "quantise"])
def test_grouped_products(moe, op):
    rows, K, N, G = (6 if op == "few rows" else 600), 256, 256, 2
    b, e = dev_i32([0, rows // 3]), dev_i32([rows // 3, rows])
    cfg = moe.grouped_config(rows, K, N, G)
    ws = moe.grouped_workspace(cfg)
    x, W = rand((rows, K), torch.bfloat16, 1), rand((G, N, K), torch.bfloat16, 2)
    q, qs = torch.ones(rows, K, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    Wq, Ws = torch.ones(G, N, K, dtype=torch.int8, device="cuda"), torch.ones(G, N, device="cuda")
    out = torch.zeros((G, N, K) if op == "dw" else (rows, K), dtype=torch.int8 if op == "quantise" else torch.bfloat16,
                      device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    call = {"mm": lambda: moe.moe_grouped_mm(cfg, b, e, x, W, out, ws, stream),
            "few rows": lambda: moe.moe_grouped_mm(cfg, b, e, x, W, out, ws, stream),
            "dx": lambda: moe.moe_grouped_mm_dx(cfg, b, e, x, W, out, ws, stream),
            "dw": lambda: moe.moe_grouped_mm_dw(cfg, b, e, x, x, out, ws, stream),
            "i8": lambda: moe.moe_grouped_mm_i8(cfg, b, e, q, qs, Wq, Ws, out, ws, stream),
            "quantise": lambda: moe.moe_quantize_rows_i8(x, out, qs, stream)}[op]
    in_new_thread(call)
    assert moe.moe_check_error(ws) == 0
    got = out.clone()
    assert bool((got != 0).any())
    out.zero_()
    call()
    assert moe.moe_check_error(ws) == 0
    assert torch.equal(got, out)


def test_expert_ffn(moe):
    T, d, f, E, k = 300, 128, 192, 8, 2
    cfg = moe.config(T=T, d=d, f=f, E=E, k=k)
    buf = moe.Buffers.allocate(cfg)
    idx = torch.from_numpy(synth.random_assignments(0, T, E, k, 1.0)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    xp = torch.zeros(buf.rows, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch(cfg, idx, rand((T, d), torch.bfloat16, 1), torch.empty(E, **i32), torch.empty(E + 1, **i32),
                     torch.empty(T, k, **i32), torch.empty(T * k, **i32), xp, buf.ws)
    Wg, Wu, Wd = rand((E, f, d), torch.bfloat16, 2), rand((E, f, d), torch.bfloat16, 3), rand((E, d, f), torch.bfloat16, 4)
    out = torch.zeros_like(xp)
    stream = torch.cuda.current_stream().cuda_stream
    in_new_thread(lambda: moe.moe_expert_ffn_fwd(cfg, xp, Wg, Wu, Wd, out, buf.ws, stream))
    assert moe.moe_check_error(buf.ws) == 0
    got = out.clone()
    out.zero_()
    moe.moe_expert_ffn_fwd(cfg, xp, Wg, Wu, Wd, out, buf.ws, stream)
    assert moe.moe_check_error(buf.ws) == 0
    assert bool((got != 0).any()) and torch.equal(got, out)


FIRST_CALLS = """
import threading, torch
import mixture_experts_layer_10_gb300 as moe
rows, K, N, G, n = 600, 256, 320, 2, 8
moe.load()
g = torch.Generator("cuda").manual_seed(1)
x, dy, W = (torch.empty(s, device="cuda").normal_(generator=g).bfloat16() for s in ((rows, K), (rows, N), (G, N, K)))
b, e = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 250], [250, 600]))
cfg = moe.grouped_config(rows, K, N, G)
outs = [[torch.zeros_like(t) for t in (dy, x, W)] for _ in range(n)]
ws = [moe.grouped_workspace(cfg) for _ in range(n)]
streams = [torch.cuda.Stream() for _ in range(n)]
torch.cuda.synchronize()
start, failed = threading.Barrier(n), []

def calls(i):
    try:
        y, dx, dW = outs[i]
        start.wait()
        moe.moe_grouped_mm(cfg, b, e, x, W, y, ws[i], streams[i])
        moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx, ws[i], streams[i])
        moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws[i], streams[i])
        assert moe.moe_check_error(ws[i], streams[i]) == 0
    except Exception as err:
        failed.append(repr(err))

threads = [threading.Thread(target=calls, args=(i,)) for i in range(n)]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not failed, failed
ref = [[x[p:q].float() @ W[i].float().T for i, (p, q) in enumerate(((0, 250), (250, 600)))]]
assert torch.allclose(outs[0][0].float(), torch.cat(ref[0]), atol=0.5, rtol=0.02)
for o in outs[1:]:
    assert all(torch.equal(u, v) for u, v in zip(o, outs[0]))
print("same")
"""


def test_first_calls_of_several_threads():
    """A new process's first calls, made by eight threads at once on streams and workspaces of their own."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
