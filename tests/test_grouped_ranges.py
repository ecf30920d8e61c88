"""Grouped products (GPU) at the ends of what they take: exact sums over long contractions, the most groups,
every pair of forms that the weight gradient's copies have, elements past 32 bits of offset, one group that
holds all rows.

Exact sums: operands of -1, 0 and 1 (8-bit: codes up to 32 in magnitude) make every product and every partial
sum an integer below 2^24, and outputs that the tests have asserted to be below the type's own integers are
equal to the sums in 64 bits, to the bit: one product lost or taken twice shows.
"""
import pytest
import torch

from test_grouped import TYPES, check, dev_i32, exact_dw, exact_mm, in_groups, layout, rand, run_all, run_i8

pytestmark = pytest.mark.gpu

INTEGERS = {torch.bfloat16: 2 ** 8, torch.float16: 2 ** 11}   # up to here each is a value of the type
LONG = [4700, None, 0, 300, 2049]   # more than 16 row tiles, runs of 2048 rows that do and do not come out even


def signs(shape, dtype, seed):
    """-1, 0, 0 or 1."""
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.randint(0, 4, shape, generator=g, device="cuda")
    return ((v == 3).int() - (v == 0).int()).to(dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("groups,K,N", [(LONG, 4096, 520), (LONG, 520, 1032), ([3, 0, None, 5, 1], 4096, 520)])
def test_exact_sums(moe, groups, K, N, dtype):
    t = TYPES[dtype]
    begin, end, rows = layout(groups)
    G, live = len(begin), in_groups(begin, end, rows)
    x, dy, W = signs((rows, K), t, 1), signs((rows, N), t, 2), signs((G, N, K), t, 3)
    b, e = dev_i32(begin), dev_i32(end)
    cfg = moe.grouped_config(rows, K, N, G, dtype=t)
    ws = moe.grouped_workspace(cfg)
    y, dx, dW = torch.zeros_like(dy), torch.zeros_like(x), torch.empty_like(W)
    moe.moe_grouped_mm(cfg, b, e, x, W, y, ws)
    moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx, ws)
    moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws)
    add = moe.grouped_config(rows, K, N, G, dtype=t, dw_dtype=torch.float32, accumulate=1)
    dW32 = torch.arange(G * N * K, device="cuda").remainder_(100).float().view(G, N, K)
    before = dW32.double()
    moe.moe_grouped_mm_dw(add, b, e, dy, x, dW32, ws)
    assert moe.moe_check_error(ws) == 0
    ref_y, ref_dx = exact_mm(begin, end, x, W)[0], exact_mm(begin, end, dy, W.transpose(1, 2))[0]
    ref_dW = exact_dw(begin, end, dy, x)[0]
    for out, ref in ((y, ref_y), (dx, ref_dx), (dW, ref_dW)):
        assert ref.abs().max().item() <= INTEGERS[t]
        assert torch.equal(out.double(), ref)
    assert bool((y[~live] == 0).all())
    assert torch.equal(dW32.double(), ref_dW + before)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("groups,K,N", [(LONG, 4096, 520), (LONG, 1040, 264), ([3, 0, None, 5, 1], 4096, 520)])
def test_exact_8bit_sums(moe, groups, K, N, dtype):
    t = TYPES[dtype]
    begin, end, rows = layout(groups)
    G, live = len(begin), in_groups(begin, end, rows)
    g = torch.Generator("cuda").manual_seed(K)
    q, P = (torch.randint(-32, 33, s, generator=g, device="cuda").to(torch.int8) for s in ((rows, K), (G, N, K)))
    qs = 2.0 ** -torch.randint(4, 8, (rows,), generator=g, device="cuda").float()
    Ps = 2.0 ** -torch.randint(4, 8, (G, N), generator=g, device="cuda").float()
    cfg = moe.grouped_config(rows, K, N, G, dtype=t)
    ws = moe.grouped_workspace(cfg)
    y = torch.zeros(rows, N, dtype=t, device="cuda")
    moe.moe_grouped_mm_i8(cfg, dev_i32(begin), dev_i32(end), q, qs, P, Ps, y, ws)
    assert moe.moe_check_error(ws) == 0
    ref, S = exact_mm(begin, end, q, P)
    assert S.max().item() < 2 ** 24
    for gi, (a, z) in enumerate(zip(begin, end)):
        ref[a:z] *= qs[a:z].double()[:, None] * Ps[gi].double()   # powers of two
    assert torch.equal(y[live], ref[live].to(t))


@pytest.mark.parametrize("step", [3, 20, 40])
def test_most_groups(moe, step):
    """1024 groups, on few rows (3), more than the few-row kernels take (20; in 8 bits 40)."""
    begin, end, rows = layout([i * 7 % step for i in range(1024)])
    run_all(moe, begin, end, rows, 64, 72, torch.bfloat16)
    run_i8(moe, begin, end, rows, 64, 72, torch.float16)


@pytest.mark.parametrize("dw_dtype", [None, torch.float32])
@pytest.mark.parametrize("K,N", [(128, 192), (136, 192), (128, 200), (136, 200)])
def test_weight_gradient_copies(moe, K, N, dw_dtype):
    """Either operand's width a multiple of 64 or not."""
    begin, end, rows = layout([5, 0, None, 130, 2100, 64, 1])
    run_all(moe, begin, end, rows, K, N, torch.bfloat16, dw_dtype=dw_dtype)
    run_all(moe, begin, end, rows, K, N, torch.float16, dw_dtype=dw_dtype, pad=8)


@pytest.mark.parametrize("G,each", [(64, 8), (64, 16), (1024, 8)])
def test_all_rows_in_one_group(moe, G, each):
    """As many rows as few-row kernels take for G groups, all of one group: its weight serves every row tile."""
    groups = [0] * G
    groups[G // 3] = each * G
    begin, end, rows = layout(groups)
    if each == 8:
        run_all(moe, begin, end, rows, 72, 136, torch.bfloat16)
    run_i8(moe, begin, end, rows, 80, 136, torch.float16)


def far(rows, width, stride, dtype):
    """[rows, width] whose rows are `stride` elements apart."""
    return torch.empty(rows * stride, dtype=dtype, device="cuda").view(rows, stride)[:, :width]


@pytest.mark.parametrize("G", [2, 40])
@pytest.mark.parametrize("op", ["mm", "dx", "dw", "i8"])
def test_far_rows_of_every_product(moe, op, G):
    """Rows 2^24 elements apart, 300 of them: offsets past 32 bits, on few rows a group (40 groups) and many."""
    rows, K, N, stride = 300, 64, 80, 1 << 24
    if torch.cuda.mem_get_info()[0] < 2 * 2 * rows * stride + (4 << 30):
        pytest.skip("not enough free memory")
    begin, end, _ = layout([20] + [0] * (G - 2) + [280])
    b, e, t = dev_i32(begin), dev_i32(end), torch.bfloat16
    cfg = moe.grouped_config(rows, K, N, G, in_stride=stride, out_stride=stride)
    ws = moe.grouped_workspace(cfg)
    W = rand((G, N, K), t, 2)
    x0, dy0 = rand((rows, K), t, 1), rand((rows, N), t, 3)
    if op == "i8":
        q, qs = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
        P, Ps = torch.empty(G, N, K, dtype=torch.int8, device="cuda"), torch.empty(G, N, device="cuda")
        moe.moe_quantize_rows_i8(x0, q, qs)
        moe.moe_quantize_rows_i8(W, P, Ps)
        codes, y = far(rows, K, stride, torch.int8), far(rows, N, stride, t)
        codes.copy_(q)
        moe.moe_grouped_mm_i8(cfg, b, e, codes, qs, P, Ps, y, ws)
        ref, S = exact_mm(begin, end, q.double() * qs.double()[:, None], P.double() * Ps.double()[..., None])
        out, terms, extra = y, 0, 3 * 2.0 ** -24
    elif op == "dw":
        x, dy, out = far(rows, K, stride, t), far(rows, N, stride, t), torch.empty_like(W)
        x.copy_(x0)
        dy.copy_(dy0)
        moe.moe_grouped_mm_dw(cfg, b, e, dy, x, out, ws)
        ref, S = exact_dw(begin, end, dy0, x0)
        terms, extra = 280, 0.0
    else:
        width_in, width_out, v = (K, N, x0) if op == "mm" else (N, K, dy0)
        src, out = far(rows, width_in, stride, t), far(rows, width_out, stride, t)
        src.copy_(v)
        (moe.moe_grouped_mm if op == "mm" else moe.moe_grouped_mm_dx)(cfg, b, e, src, W, out, ws)
        ref, S = exact_mm(begin, end, v, W if op == "mm" else W.transpose(1, 2))
        terms, extra = width_in, 0.0
    assert moe.moe_check_error(ws) == 0
    check(op, out, ref, S, terms, extra)


@pytest.mark.parametrize("rows", [40, 1200])
@pytest.mark.parametrize("op", ["mm", "dx", "dw", "dw32", "i8"])
def test_far_weights(moe, op, rows):
    """Weights of more than 2^32 elements; the first and the last group have the rows."""
    G, K, N, t = 66, 8192, 8192, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 5 * G * K * N + (8 << 30):
        pytest.skip("not enough free memory")
    groups = [rows // 4] + [0] * (G - 2) + [rows - rows // 4]
    begin, end, _ = layout(groups)
    b, e = dev_i32(begin), dev_i32(end)
    cfg = moe.grouped_config(rows, K, N, G, dw_dtype=torch.float32 if op == "dw32" else t)
    ws = moe.grouped_workspace(cfg)
    x, dy = rand((rows, K), t, 1), rand((rows, N), t, 2)
    parts = ((0, begin[0], end[0]), (G - 1, begin[-1], end[-1]))
    if op in ("dw", "dw32"):
        dW = torch.full((G, N, K), 7.0, dtype=torch.float32 if op == "dw32" else t, device="cuda")
        moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws)
        assert moe.moe_check_error(ws) == 0
        for g, a, z in parts:
            ref, S = exact_dw([a], [z], dy, x)
            check(op, dW[g][None], ref, S, z - a)
        for g in range(1, G - 1):
            assert not bool(dW[g].any())
        return
    W = torch.empty(G, N, K, dtype=torch.int8 if op == "i8" else t, device="cuda")
    for g in (0, G - 1):
        W[g] = rand((N, K), t, 3 + g) if op != "i8" else torch.randint(-20, 21, (N, K), device="cuda").to(torch.int8)
    out = torch.empty(rows, N, dtype=t, device="cuda")
    if op == "i8":
        q = torch.randint(-20, 21, (rows, K), device="cuda").to(torch.int8)
        one, ones = torch.full((rows,), 2.0 ** -8, device="cuda"), torch.ones(G, N, device="cuda")
        moe.moe_grouped_mm_i8(cfg, b, e, q, one, W, ones, out, ws)
        src, Wt, scale = q, lambda g: W[g], 2.0 ** -8
    elif op == "mm":
        moe.moe_grouped_mm(cfg, b, e, x, W, out, ws)
        src, Wt, scale = x, lambda g: W[g], 1.0
    else:
        moe.moe_grouped_mm_dx(cfg, b, e, dy, W, out, ws)
        src, Wt, scale = dy, lambda g: W[g].T, 1.0
    assert moe.moe_check_error(ws) == 0
    for g, a, z in parts:
        ref, S = exact_mm([0], [z - a], src[a:z], Wt(g)[None])
        check(op, out[a:z], ref * scale, S * scale, 0 if op == "i8" else K, 0.0)
