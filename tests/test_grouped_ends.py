"""Grouped products (GPU) where sums are long: rows or columns by the ten thousand.

A tensor-core accumulator drops up to one unit of its last place, 2^-23 of the running sum, at each step of
16 products, always towards zero, so with values of one sign the losses add up.  A weight gradient is summed
2048 rows at a time (128 steps) and the parts are added in fp32, rounded to nearest (2^-24 each).
"""
import pytest
import torch

from test_grouped import TYPES, dev_i32, layout, rand, run_all, run_i8

pytestmark = pytest.mark.gpu


def positive(shape, dtype, seed, scale):
    """Values of one sign in [scale / 2, scale]."""
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") * 0.5 + 0.5).mul_(scale).to(dtype)


@pytest.mark.parametrize("rows", [[2049], [65536, 3, 16384], [262144]])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_long_group_16bit_weight_gradient(moe, dtype, rows):
    """dW in the operands' type over many rows of one sign: each output within half a step of its type and
    the sums' own error of 64 bits, and no bias of all outputs together."""
    t = TYPES[dtype]
    K, N, n, G = 72, 136, sum(rows), len(rows)
    begin = [sum(rows[:g]) for g in range(G)]
    end = [b + r for b, r in zip(begin, rows)]
    # columns of different size, so that the outputs lie anywhere between two 16-bit values
    x = positive((n, K), t, 1, 4 * max(rows) ** -0.5) * torch.linspace(0.5, 1, K, device="cuda").to(t)
    dy = positive((n, N), t, 2, 4 * max(rows) ** -0.5)
    cfg = moe.grouped_config(n, K, N, G, dtype=t)
    ws = moe.grouped_workspace(cfg)
    dW = torch.empty(G, N, K, dtype=t, device="cuda")
    moe.moe_grouped_mm_dw(cfg, dev_i32(begin), dev_i32(end), dy, x, dW, ws)
    assert moe.moe_check_error(ws) == 0
    eps = torch.finfo(t).eps
    for g in range(G):
        ref = dy[begin[g]:end[g]].double().T @ x[begin[g]:end[g]].double()
        off = (dW[g].double() - ref) / ref
        runs = (rows[g] + 2047) // 2048
        sums = (128 + 1) * 2.0 ** -23 + runs * 2.0 ** -24
        assert off.abs().max().item() <= sums + eps / 2 * (1 + sums)
        if rows[g] > 2048:
            # the roundings of N K outputs average out: eps / 2 / sqrt(3) each at most, five deviations
            assert off.mean().abs().item() <= sums + 5 * eps / 2 / (3 * N * K) ** 0.5


# few rows a group: a cluster of blocks splits the contraction, with a tile for every cluster at most.
# Spreads of the rows that make the most tiles of 8 or 32 rows, and the fewest.
SPREADS = {
    "8 rows": [[8, 0, 0, 0], [5, 1, 1, 1], [2, 2, 2, 2], [0, 0, 0, 8], [0, 0, 0, 0]],
    "32 rows": [[32, 0, 0, 0], [29, 1, 1, 1], [0, 31, 0, 1], [8, 8, 8, 8]],
    "200 rows": [[200, 0, 0, 0, 0, 0, 0, 0], [193, 1, 1, 1, 1, 1, 1, 1], [97, 33, 65, 1, 1, 1, 1, 1],
                 [25, 25, 25, 25, 25, 25, 25, 25], [0, 199, 0, 0, 0, 0, 0, 1]],
}


@pytest.mark.parametrize("name", list(SPREADS))
def test_few_rows_spreads(moe, name):
    for groups in SPREADS[name]:
        begin, end, _ = layout(groups)
        rows = int(name.split()[0])   # of the buffer: what the call is planned for
        run_all(moe, begin, end, rows, 2048, 136, torch.bfloat16)
        run_i8(moe, begin, end, rows, 4096, 136, torch.float16, codes=(-32, 33))


@pytest.mark.parametrize("rows", [5, 300])
def test_scales_in_a_larger_array(moe, rows):
    """Scales that start at any float of an array: the same results to the bit, nothing written beside them."""
    K, N, G = 256, 136, 3
    x, W = rand((rows, K), torch.bfloat16, 1), rand((G, N, K), torch.bfloat16, 2)
    cfg = moe.grouped_config(rows, K, N, G)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32([0, 2, 4]), dev_i32([2, 4, rows])
    q, Wq = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(G, N, K, dtype=torch.int8, device="cuda")
    out = []
    for at in (0, 1, 2, 3):
        qs, Ws = torch.full((rows + 8,), 7.0, device="cuda"), torch.full((G * N + 8,), 7.0, device="cuda")
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        s, t = qs[at:at + rows], Ws[at:at + G * N].view(G, N)
        moe.moe_quantize_rows_i8(x, q, s)
        moe.moe_quantize_rows_i8(W, Wq, t)
        moe.moe_grouped_mm_i8(cfg, b, e, q, s, Wq, t, y, ws)
        assert moe.moe_check_error(ws) == 0
        assert bool((qs[:at] == 7).all()) and bool((qs[at + rows:] == 7).all())
        out.append((y, s.clone(), t.clone()))
    for other in out[1:]:
        assert all(torch.equal(u, v) for u, v in zip(other, out[0]))


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_widest_contraction(moe, dtype, rows):
    """65536 columns of one sign, on few rows and on many: y, dx and 8-bit products lose at most 2^-23 of the
    sum at each 16 products, and one rounding of the type."""
    t, L, N = TYPES[dtype], 65536, 136
    steps = (L // 16 + 1) * 2.0 ** -23
    eps = torch.finfo(t).eps
    x = positive((rows, L), t, 1, 4 * L ** -0.5)
    W = positive((N, L), t, 2, 4 * L ** -0.5) * torch.linspace(0.5, 1, N, device="cuda").to(t)[:, None]
    b, e = dev_i32([0]), dev_i32([rows])
    ref = x.double() @ W.double().T
    wide, back = moe.grouped_config(rows, L, N, 1, dtype=t), moe.grouped_config(rows, N, L, 1, dtype=t)
    ws = moe.grouped_workspace(wide)
    y, dx = (torch.empty(rows, N, dtype=t, device="cuda") for _ in range(2))
    moe.moe_grouped_mm(wide, b, e, x, W[None], y, ws)
    moe.moe_grouped_mm_dx(back, b, e, x, W.T.contiguous()[None], dx, ws)
    assert moe.moe_check_error(ws) == 0
    for out in (y, dx):
        assert ((out.double() - ref) / ref).abs().max().item() <= steps + eps / 2 * (1 + steps)
    q, P = ((positive(s, torch.float32, i, 127)).round().to(torch.int8) for i, s in ((3, (rows, L)), (4, (1, N, L))))
    qs = torch.linspace(0.5, 1, rows, device="cuda") * 2.0 ** -14
    Ps = torch.linspace(0.5, 1, N, device="cuda")[None] * 2.0 ** -14
    moe.moe_grouped_mm_i8(wide, b, e, q, qs, P, Ps, y, ws)
    assert moe.moe_check_error(ws) == 0
    ref = q.double() @ P[0].double().T * qs.double()[:, None] * Ps.double()
    before = steps + 3 * 2.0 ** -24
    assert ((y.double() - ref) / ref).abs().max().item() <= before + eps / 2 * (1 + before)


def test_profile_counts_every_launch(moe):
    """Every kernel that the grouped products launch is timed and counted, under a name of its own."""
    rows, K, N, G = 600, 256, 136, 2
    b, e = dev_i32([0, 250]), dev_i32([250, 600])
    cfg = moe.grouped_config(rows, K, N, G)
    ws = moe.grouped_workspace(cfg)
    x, dy, W = rand((rows, K), torch.bfloat16, 1), rand((rows, N), torch.bfloat16, 2), rand((G, N, K), torch.bfloat16, 3)
    q, qs = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    P, Ps = torch.empty(G, N, K, dtype=torch.int8, device="cuda"), torch.empty(G, N, device="cuda")
    y, dx, dW = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(W)
    layer = moe.config(T=64, d=128, f=128, E=2, k=1)
    buf = moe.Buffers.allocate(layer)
    idx = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    moe.moe_dispatch(layer, idx, rand((64, 128), torch.bfloat16, 4), torch.empty(2, **i32), torch.empty(3, **i32),
                     torch.empty(64, 1, **i32), torch.empty(64, **i32),
                     torch.empty(buf.rows, 128, dtype=torch.bfloat16, device="cuda"), buf.ws)
    calls = {"grouped_mm": lambda: moe.moe_grouped_mm(cfg, b, e, x, W, y, ws),
             "grouped_mm_dx": lambda: moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx, ws),
             "grouped_maps grouped_mm_dw": lambda: moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws),
             "quantize_i8": lambda: (moe.moe_quantize_rows_i8(x, q, qs), moe.moe_quantize_rows_i8(W, P, Ps)),
             "grouped_mm_i8": lambda: moe.moe_grouped_mm_i8(cfg, b, e, q, qs, P, Ps, y, ws),
             "segments": lambda: moe.moe_segments(layer, torch.empty(2, **i32), torch.empty(2, **i32), buf.ws)}
    for names, call in calls.items():
        moe.moe_profile_enable(True)
        call()
        prof = moe.moe_profile_read()
        moe.moe_profile_enable(False)
        ran = {n: launches for n, (ms, launches) in prof.items() if launches}
        assert ran == {n: 2 if n == "quantize_i8" else 1 for n in names.split()}
        assert all(prof[n][0] > 0 for n in ran)
    assert moe.moe_check_error(ws) == 0 and moe.moe_check_error(buf.ws) == 0
