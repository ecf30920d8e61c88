"""Grouped products (GPU): moe_grouped_mm, its gradients and the 8-bit integer form against the
definition in 64 bits, over group lengths, widths, types, strides and gaps.

Tolerance: an output is rounded once to its type (half a step, eps / 2 relative, or half the smallest
fp16 step); before that each of the L products and L / 16 partial sums of a result loses at most one
unit of 2^-23 of the largest partial sum, which the sum S of the products' magnitudes bounds.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# rows of every group (None: 5 rows that belong to no group)
GROUPS = {
    "one_row": [1],
    "one": [37],
    "none": [0, 0],
    "mixed": [5, 0, 1, 130, None, 64, 0, 257, 33],
    "tile_ends": [256, 255, None, 128, 31, 32, 96, 16, 15, 8, 63, 65],
    "many_short": [i % 4 for i in range(300)],
    "long": [3, 1500, 0, 700],
    "gap_first": [None, 40, None, 300, None],
}
WIDTHS = [(8, 8), (64, 128), (72, 264), (520, 136), (1024, 24), (136, 1032)]


def layout(groups):
    """(begin, end, rows) of the test's groups."""
    begin, end, at = [], [], 0
    for n in groups:
        if n is None:
            at += 5
            continue
        begin.append(at)
        at += n
        end.append(at)
    return begin, end, at


def dev_i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rand(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def exact_mm(begin, end, x, W):
    """(y, S) in 64 bits, zero in rows of no group."""
    y = torch.zeros(x.shape[0], W.shape[1], dtype=torch.float64, device="cuda")
    S = torch.zeros_like(y)
    for g, (a, b) in enumerate(zip(begin, end)):
        y[a:b] = x[a:b].double() @ W[g].double().T
        S[a:b] = x[a:b].double().abs() @ W[g].double().abs().T
    return y, S


def exact_dw(begin, end, dy, x):
    dW = torch.stack([dy[a:b].double().T @ x[a:b].double() for a, b in zip(begin, end)])
    S = torch.stack([dy[a:b].double().abs().T @ x[a:b].double().abs() for a, b in zip(begin, end)])
    return dW, S


def check(what, got, ref, S, terms, extra=0.0):
    """got against ref: `terms` products a result, `extra` further relative roundings."""
    eps = torch.finfo(got.dtype).eps
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    pre = (terms + terms // 16 + 1) * 2.0 ** -23 * S + extra * ref.abs()
    bound = pre + eps / 2 * (ref.abs() + pre) + tiny
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got.float()).all()), f"{what}: not finite"
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {int((err > bound).sum())} of {err.numel()} outside, worst by {worst:.3e}"


def in_groups(begin, end, rows):
    m = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, b in zip(begin, end):
        m[a:b] = True
    return m


def run_all(moe, begin, end, rows, K, N, dtype, dw_dtype=None, accumulate=0, seed=0, pad=0):
    """Forward and both gradients of one layout, checked; rows of no group hold NaN on the way in and
    a mark on the way out.  `pad`: extra elements between rows."""
    G = len(begin)
    dw_dtype = dw_dtype or dtype
    cfg = moe.grouped_config(rows, K, N, G, dtype=dtype, dw_dtype=dw_dtype, accumulate=accumulate,
                             in_stride=K + pad if pad else 0, out_stride=N + pad if pad else 0)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32(begin), dev_i32(end)
    live = in_groups(begin, end, rows)
    x = rand((rows, K + pad), dtype, seed)[:, :K]
    dy = rand((rows, N + pad), dtype, seed + 1)[:, :N]
    W = rand((G, N, K), dtype, seed + 2) * K ** -0.5
    x[~live] = float("nan")
    dy[~live] = float("nan")
    y = torch.full((rows, N + pad), 7.0, dtype=dtype, device="cuda")
    dx = torch.full((rows, K + pad), 7.0, dtype=dtype, device="cuda")
    dW = rand((G, N, K), dw_dtype, seed + 3)
    dW0 = dW.double() if accumulate else torch.zeros(1, dtype=torch.float64, device="cuda")
    moe.moe_grouped_mm(cfg, b, e, x, W, y[:, :N], ws)
    moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx[:, :K], ws)
    moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws)
    assert moe.moe_check_error(ws) == 0
    for what, out, width in (("y", y, N), ("dx", dx, K)):
        assert bool((out[~live] == 7).all()), f"{what}: a row of no group was written"
        assert bool((out[:, width:] == 7).all()), f"{what}: the space between rows was written"
    x0, dy0 = torch.where(live[:, None], x, 0), torch.where(live[:, None], dy, 0)
    ref, S = exact_mm(begin, end, x0, W)
    check("y", y[:, :N][live], ref[live], S[live], K)
    ref, S = exact_mm(begin, end, dy0, W.transpose(1, 2))
    check("dx", dx[:, :K][live], ref[live], S[live], N)
    ref, S = exact_dw(begin, end, dy0, x0)
    terms = max(bb - aa for aa, bb in zip(begin, end))
    check("dW", dW, ref + dW0, S + dW0.abs(), terms)
    return x0, dy0, dW


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("name", list(GROUPS))
def test_group_lengths(moe, name, dtype):
    begin, end, rows = layout(GROUPS[name])
    run_all(moe, begin, end, rows, 192, 320, TYPES[dtype])


@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("name", ["mixed", "many_short"])
def test_widths(moe, name, K, N):
    begin, end, rows = layout(GROUPS[name])
    run_all(moe, begin, end, rows, K, N, torch.bfloat16, seed=K)


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("name,K,N", [("mixed", 200, 264), ("many_short", 64, 72), ("long", 256, 256), ("none", 64, 64)])
def test_fp32_weight_gradient(moe, name, K, N, dtype, accumulate):
    begin, end, rows = layout(GROUPS[name])
    run_all(moe, begin, end, rows, K, N, TYPES[dtype], dw_dtype=torch.float32, accumulate=accumulate)


def test_long_group_fp32_weight_gradient(moe):
    """A contraction of many thousand rows stays an fp32 sum: relative error as of 32 bits."""
    begin, end, rows = layout([9001, 0, 4097])
    x, dy, dW = run_all(moe, begin, end, rows, 128, 136, torch.bfloat16, dw_dtype=torch.float32)
    ref, _ = exact_dw(begin, end, dy, x)
    assert (dW.double() - ref).norm() / ref.norm() < 1e-5


@pytest.mark.parametrize("name", ["mixed", "tile_ends", "many_short"])
def test_row_strides(moe, name):
    begin, end, rows = layout(GROUPS[name])
    run_all(moe, begin, end, rows, 136, 264, torch.float16, pad=24)
    run_all(moe, begin, end, rows, 128, 192, torch.bfloat16, pad=64)


@pytest.mark.parametrize("K,N", [(2048, 768), (768, 2048), (4096, 1408)])
@pytest.mark.parametrize("sizes", [[1] * 8 + [0] * 24, [3, 0, 9, 17, 40, 1, 2, 70], [300, 500, 120, 90]])
def test_expert_shapes(moe, sizes, K, N):
    begin, end, rows = layout(sizes)
    run_all(moe, begin, end, rows, K, N, torch.bfloat16, seed=5)


def test_no_rows(moe):
    """A call without rows writes zero weight gradients and nothing else."""
    for acc in (0, 1):
        cfg = moe.grouped_config(0, 64, 128, 3, dw_dtype=torch.float32, accumulate=acc)
        ws = moe.grouped_workspace(cfg)
        z = dev_i32([0, 0, 0])
        x, dy = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 128, dtype=torch.bfloat16,
                                                                                       device="cuda")
        W = rand((3, 128, 64), torch.bfloat16, 0)
        dW = torch.full((3, 128, 64), 2.0, device="cuda")
        moe.moe_grouped_mm(cfg, z, z, x, W, dy, ws)
        moe.moe_grouped_mm_dx(cfg, z, z, dy, W, x, ws)
        moe.moe_grouped_mm_dw(cfg, z, z, dy, x, dW, ws)
        assert moe.moe_check_error(ws) == 0
        assert bool((dW == (2.0 if acc else 0.0)).all())


@pytest.mark.parametrize("bad", ["nan", "inf", "lowest"])
def test_values_stay_in_their_group(moe, bad):
    """NaN, infinities and lowest values in one group (and between groups) leave every other group's
    outputs as they are, to the bit."""
    begin, end, rows = layout([40, 7, None, 70, 300, 1])
    K, N, G = 136, 200, 5
    v = {"nan": float("nan"), "inf": float("inf"), "lowest": torch.finfo(torch.bfloat16).min}[bad]
    cfg = moe.grouped_config(rows, K, N, G)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32(begin), dev_i32(end)
    x, dy, W = rand((rows, K), torch.bfloat16, 1), rand((rows, N), torch.bfloat16, 2), rand((G, N, K), torch.bfloat16, 3)
    out = []
    for spoil in (False, True):
        if spoil:   # group 1 and the rows of no group after it
            x[begin[1]:begin[2]] = v
            dy[begin[1]:begin[2]] = v
        y, dx, dW = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(W)
        moe.moe_grouped_mm(cfg, b, e, x, W, y, ws)
        moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx, ws)
        moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws)
        assert moe.moe_check_error(ws) == 0
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[begin[1]:end[1]] = False
        out.append((y[keep], dx[keep], dW[[0, 2, 3, 4]]))
    for a, c in zip(*out):
        assert torch.equal(a.view(torch.int16), c.view(torch.int16))


def test_a_row_of_nan_stays_a_row(moe):
    begin, end, rows = layout([300, 5])
    cfg = moe.grouped_config(rows, 128, 64, 2)
    ws = moe.grouped_workspace(cfg)
    x, W = rand((rows, 128), torch.bfloat16, 1), rand((2, 64, 128), torch.bfloat16, 2)
    y0, y1 = (torch.empty(rows, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_grouped_mm(cfg, dev_i32(begin), dev_i32(end), x, W, y0, ws)
    x[7, 3] = float("nan")
    moe.moe_grouped_mm(cfg, dev_i32(begin), dev_i32(end), x, W, y1, ws)
    assert bool(torch.isnan(y1[7]).all())
    keep = torch.arange(rows, device="cuda") != 7
    assert torch.equal(y0[keep], y1[keep])


@pytest.mark.parametrize("begin,end", [([0, 5], [6, 10]), ([0, 5], [5, 11]), ([-1, 5], [5, 10]), ([0, 5], [5, 4]),
                                       ([4, 0], [10, 4]), ([0, 2 ** 31 - 1], [5, 2 ** 31 - 1])])
def test_bad_groups_write_nothing(moe, begin, end):
    """Groups out of range or out of order are reported, and no output is touched; the next call with
    good groups runs."""
    rows, K, N = 10, 64, 64
    cfg = moe.grouped_config(rows, K, N, 2)
    ws = moe.grouped_workspace(cfg)
    x, W = rand((rows, K), torch.bfloat16, 1), rand((2, N, K), torch.bfloat16, 2)
    q, qs = torch.ones(rows, K, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    Wq, Ws = torch.ones(2, N, K, dtype=torch.int8, device="cuda"), torch.ones(2, N, device="cuda")
    b, e = dev_i32(begin), dev_i32(end)

    def calls():
        yield lambda o: moe.moe_grouped_mm(cfg, b, e, x, W, o, ws), (rows, N)
        yield lambda o: moe.moe_grouped_mm_dx(cfg, b, e, x, W, o, ws), (rows, K)
        yield lambda o: moe.moe_grouped_mm_dw(cfg, b, e, x, x, o, ws), (2, N, K)
        yield lambda o: moe.moe_grouped_mm_i8(cfg, b, e, q, qs, Wq, Ws, o, ws), (rows, N)

    for call, shape in calls():
        out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        call(out)
        assert moe.moe_check_error(ws) == 5
        assert bool((out == 7).all())
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm(cfg, dev_i32([0, 5]), dev_i32([5, 10]), x, W, out, ws)
    assert moe.moe_check_error(ws) == 0 and not bool((out == 7).all())


@pytest.mark.parametrize("sizes", [[6, 0, 3], [200, 60, 300]])
def test_gradients_are_the_differences(moe, sizes):
    """Small integers, so that every product and sum is exact: the change of <c, y> when one x or one W
    changes by one is the gradient there, to the bit."""
    begin, end, rows = layout(sizes)
    K, N, G = 16, 24, len(sizes)
    cfg = moe.grouped_config(rows, K, N, G, dw_dtype=torch.float32)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32(begin), dev_i32(end)
    g = torch.Generator("cuda").manual_seed(3)
    x, c, W = (torch.randint(-1, 2, s, generator=g, device="cuda").to(torch.bfloat16)
               for s in ((rows, K), (rows, N), (G, N, K)))

    def value():
        y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_mm(cfg, b, e, x, W, y, ws)
        return (y.double() * c.double()).sum().item()

    dx, dW = torch.zeros_like(x), torch.zeros(G, N, K, device="cuda")
    moe.moe_grouped_mm_dx(cfg, b, e, c, W, dx, ws)
    moe.moe_grouped_mm_dw(cfg, b, e, c, x, dW, ws)
    base = value()
    for r, k in ((0, 0), (rows - 1, K - 1), (rows // 2, 5)):
        x[r, k] += 1
        assert value() - base == dx[r, k].item()
        x[r, k] -= 1
    for gi, n, k in ((0, 0, 0), (2, N - 1, K - 1), (2, 7, 3)):
        W[gi, n, k] += 1
        assert value() - base == dW[gi, n, k].item()
        W[gi, n, k] -= 1
    assert moe.moe_check_error(ws) == 0


@pytest.mark.parametrize("sizes", [[2, 0, 1], [40, 300, 7]])
def test_repeats_streams_and_graphs(moe, sizes):
    """The same bits from call to call, on another stream, and from a captured graph replayed on new
    inputs."""
    begin, end, rows = layout(sizes)
    K, N, G = 256, 320, 3
    cfg = moe.grouped_config(rows, K, N, G, dw_dtype=torch.float32, accumulate=1)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32(begin), dev_i32(end)
    x, dy, W = rand((rows, K), torch.bfloat16, 1), rand((rows, N), torch.bfloat16, 2), rand((G, N, K), torch.bfloat16, 3)
    q, qs = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    Wq, Ws = torch.empty(G, N, K, dtype=torch.int8, device="cuda"), torch.empty(G, N, device="cuda")
    moe.moe_quantize_rows_i8(W, Wq, Ws)
    y, yi, dx, dW = torch.zeros_like(dy), torch.zeros_like(dy), torch.zeros_like(x), torch.zeros(G, N, K, device="cuda")

    def step():
        dW.zero_()
        moe.moe_grouped_mm(cfg, b, e, x, W, y, ws)
        moe.moe_grouped_mm_dx(cfg, b, e, dy, W, dx, ws)
        moe.moe_grouped_mm_dw(cfg, b, e, dy, x, dW, ws)
        moe.moe_quantize_rows_i8(x, q, qs)
        moe.moe_grouped_mm_i8(cfg, b, e, q, qs, Wq, Ws, yi, ws)

    def result():
        torch.cuda.synchronize()
        r = [t.clone() for t in (y, dx, dW, yi)]
        for t in (y, dx, dW, yi):
            t.zero_()
        torch.cuda.synchronize()
        return r

    def same(p, r):
        return all(torch.equal(u, v) for u, v in zip(p, r))

    step()
    first = result()
    step()
    assert same(first, result())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    assert same(first, result())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    result()
    graph.replay()
    assert same(first, result())
    x.mul_(-1)
    graph.replay()
    replayed = result()
    step()
    assert same(replayed, result()) and not same(first, replayed)
    assert moe.moe_check_error(ws) == 0


@pytest.mark.parametrize("op,sizes,K,N", [("mm", [600, 70], 256, 256), ("dx", [600, 70], 256, 256),
                                          ("dw", [600, 70], 256, 256), ("i8", [600, 70], 256, 256),
                                          ("mm", [9, 3], 2048, 2048), ("i8", [1, 1], 2048, 2048)])
def test_a_wait_that_runs_out_is_reported(moe, op, sizes, K, N):
    """A fill of the operand ring that never comes ends in MOE_ERR_TIMEOUT, and the next call runs."""
    begin, end, rows = layout(sizes)
    cfg = moe.grouped_config(rows, K, N, 2)
    ws = moe.grouped_workspace(cfg)
    b, e = dev_i32(begin), dev_i32(end)
    x, W = rand((rows, K), torch.bfloat16, 1), rand((2, N, K), torch.bfloat16, 2)
    q, qs = torch.ones(rows, K, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    Wq, Ws = torch.ones(2, N, K, dtype=torch.int8, device="cuda"), torch.ones(2, N, device="cuda")
    out = torch.zeros((2, N, K) if op == "dw" else (rows, K), dtype=torch.bfloat16, device="cuda")
    call = {"mm": lambda: moe.moe_grouped_mm(cfg, b, e, x, W, out, ws),
            "dx": lambda: moe.moe_grouped_mm_dx(cfg, b, e, x, W, out, ws),
            "dw": lambda: moe.moe_grouped_mm_dw(cfg, b, e, x, x, out, ws),
            "i8": lambda: moe.moe_grouped_mm_i8(cfg, b, e, q, qs, Wq, Ws, out, ws)}[op]
    call()
    assert moe.moe_check_error(ws) == 0
    good = out.clone()
    moe.moe_debug_inject(ws, -1, 20_000_000, stall_fill=1)
    call()
    assert moe.moe_check_error(ws) == 6
    moe.moe_debug_inject(ws, -1, 0)
    out.zero_()
    call()
    assert moe.moe_check_error(ws) == 0
    assert torch.equal(out, good)


def test_far_rows(moe):
    """Element offsets past 32 bits: rows far apart in a large buffer."""
    rows, K, N, stride = 300, 64, 72, 1 << 24   # 300 rows x 16 Mi elements
    need = rows * stride * 2 * 2
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough free memory")
    xb = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    yb = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x, y = xb.view(rows, stride)[:, :K], yb.view(rows, stride)[:, :N]
    x.copy_(rand((rows, K), torch.bfloat16, 1))
    W = rand((2, N, K), torch.bfloat16, 2)
    cfg = moe.grouped_config(rows, K, N, 2, in_stride=stride, out_stride=stride)
    ws = moe.grouped_workspace(cfg)
    begin, end = [0, 20], [20, 300]
    moe.moe_grouped_mm(cfg, dev_i32(begin), dev_i32(end), x, W, y, ws)
    assert moe.moe_check_error(ws) == 0
    ref, S = exact_mm(begin, end, x, W)
    check("y", y, ref, S, K)


# ---- 8-bit integers ------------------------------------------------------------------------------

def exact_codes(v):
    """Codes and scales of the rows of v by the definition (v finite): the scale in fp32, the quotient
    rounded to fp32 and then to the nearest integer."""
    scale = (v.float().abs().amax(-1).double() / 127).float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return torch.round((v.double() / scale[..., None].double()).float()).clamp(-127, 127).to(torch.int8), scale


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (257, 4096), (5, 14336), (2, 65536), (1000, 528)])
def test_quantize_rows(moe, rows, cols, dtype):
    v = rand((rows, cols), TYPES[dtype], rows)
    v[:, ::17] *= 20
    v[rows // 2] = 0
    v[-1, 0] = torch.finfo(TYPES[dtype]).max
    v[0] *= 2.0 ** -14 if dtype == "fp16" else 2.0 ** -120
    codes, scales = torch.empty(rows, cols, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_quantize_rows_i8(v, codes, scales)
    c, s = exact_codes(v)
    assert torch.equal(scales, s)
    assert torch.equal(codes, c)


def test_quantize_ties_and_extremes(moe):
    """A largest value of 254 makes the scale 2: odd values lie halfway and go to the even code."""
    v = torch.arange(-254, 255, device="cuda").to(torch.float16)
    v = torch.cat([v, torch.zeros(-len(v) % 16, dtype=torch.float16, device="cuda")])[None].contiguous()
    v = torch.cat([v, torch.zeros_like(v), torch.full_like(v, float("nan")), torch.zeros_like(v)])
    v[3, 5] = float("inf")
    v[1, 9] = -0.0
    codes, scales = torch.empty(v.shape, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    moe.moe_quantize_rows_i8(v, codes, scales)
    assert scales[0].item() == 2 and scales[1].item() == 1
    assert torch.equal(codes[0].float(), torch.round(v[0].float() / 2))
    assert bool((codes[1] == 0).all())
    assert bool(torch.isnan(scales[2:]).all())


def test_quantize_tiny_rows(moe):
    """Rows whose scale underflows or is subnormal stay finite and in range."""
    v = torch.zeros(3, 32, dtype=torch.bfloat16, device="cuda")
    v[0, 3] = 2.0 ** -133    # the smallest bf16: amax / 127 rounds to a subnormal
    v[1, 3] = -(2.0 ** -126)
    v[2, 3] = 2.0 ** -140    # rounds to zero in bf16
    codes, scales = torch.empty(3, 32, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    moe.moe_quantize_rows_i8(v, codes, scales)
    c, s = exact_codes(v)
    assert torch.equal(scales, s) and torch.equal(codes, c)


def run_i8(moe, begin, end, rows, K, N, dtype, seed=0, pad=0, codes=None):
    G = len(begin)
    cfg = moe.grouped_config(rows, K, N, G, dtype=dtype, in_stride=K + pad if pad else 0, out_stride=N + 8 if pad else 0)
    ws = moe.grouped_workspace(cfg)
    g = torch.Generator("cuda").manual_seed(seed)
    lo, hi = codes or (-128, 128)
    qb = torch.randint(lo, hi, (rows, K + pad), dtype=torch.int8, device="cuda", generator=g)
    Wq = torch.randint(lo, hi, (G, N, K), dtype=torch.int8, device="cuda", generator=g)
    qs = torch.rand(rows, device="cuda", generator=g) + 0.01
    Ws = (torch.rand(G, N, device="cuda", generator=g) + 0.01) * 2.0 ** -14
    y = torch.full((rows, N + (8 if pad else 0)), 7.0, dtype=dtype, device="cuda")
    moe.moe_grouped_mm_i8(cfg, dev_i32(begin), dev_i32(end), qb[:, :K], qs, Wq, Ws, y[:, :N], ws)
    assert moe.moe_check_error(ws) == 0
    live = in_groups(begin, end, rows)
    assert bool((y[~live] == 7).all()) and bool((y[:, N:] == 7).all())
    ref, S = exact_mm(begin, end, qb[:, :K], Wq)
    scale = torch.zeros_like(ref)
    for gi, (a, b) in enumerate(zip(begin, end)):
        scale[a:b] = qs[a:b].double()[:, None] * Ws[gi].double()
    # integer sums are exact below 2^24; past that they are fp32 sums
    terms = 0 if S.numel() == 0 or float(S.max()) < 2 ** 24 else K
    pre = (terms + terms // 16) * 2.0 ** -23 * S * scale
    ref = ref * scale
    got = y[:, :N][live].double()
    eps = torch.finfo(dtype).eps
    pre = (pre + 3 * 2.0 ** -24 * ref.abs())[live]
    bound = pre + eps / 2 * (ref[live].abs() + pre) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert bool(((got - ref[live]).abs() <= bound).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("name", list(GROUPS))
def test_i8_group_lengths(moe, name, dtype):
    begin, end, rows = layout(GROUPS[name])
    run_i8(moe, begin, end, rows, 192, 320, TYPES[dtype])


@pytest.mark.parametrize("K,N", [(16, 8), (48, 264), (528, 136), (2048, 768), (4096, 24), (144, 1032)])
@pytest.mark.parametrize("name", ["mixed", "many_short", "one_row"])
def test_i8_widths(moe, name, K, N):
    begin, end, rows = layout(GROUPS[name])
    run_i8(moe, begin, end, rows, K, N, torch.bfloat16, seed=N)


def test_i8_strides_and_extreme_codes(moe):
    begin, end, rows = layout(GROUPS["mixed"])
    run_i8(moe, begin, end, rows, 208, 136, torch.bfloat16, pad=48)
    run_i8(moe, begin, end, rows, 2048, 136, torch.bfloat16, codes=(126, 128))
    run_i8(moe, begin, end, rows, 2048, 136, torch.bfloat16, codes=(-128, -126))


def test_i8_bad_rows_stay_rows(moe):
    """A NaN scale makes its own row NaN and no other."""
    rows, K, N = 40, 64, 64
    cfg = moe.grouped_config(rows, K, N, 1)
    ws = moe.grouped_workspace(cfg)
    x = rand((rows, K), torch.bfloat16, 1)
    x[3, 3], x[9, 0] = float("nan"), float("-inf")
    q, qs = torch.empty(rows, K, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    Wq, Ws = torch.ones(1, N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_quantize_rows_i8(x, q, qs)
    moe.moe_grouped_mm_i8(cfg, dev_i32([0]), dev_i32([rows]), q, qs, Wq, Ws, y, ws)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[3, 9]] = True
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())


# ---- on the layer's dispatched rows ----------------------------------------------------------------

def test_segments_and_products_on_dispatched_rows(moe):
    """moe_segments gives the padded layout of moe_dispatch, and the expert FFN built from grouped
    products of those rows gives moe_expert_ffn_fwd's output rows."""
    from harness import padded_starts
    import synth
    T, d, f, E, k, S = 300, 128, 192, 8, 2, 1
    mc = moe.config(T=T, d=d, f=f, E=E, k=k, S=S)
    buf = moe.Buffers.allocate(mc)
    idx = torch.from_numpy(synth.random_assignments(0, T, E, k, 1.0)).cuda()
    x = rand((T, d), torch.bfloat16, 1)
    counts, offsets = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ros, tor = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    xp = torch.empty(buf.rows, d, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch(mc, idx, x, counts, offsets, ros, tor, xp, buf.ws)
    b, e = (torch.empty(E + S, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.moe_segments(mc, b, e, buf.ws)
    n = counts.cpu().numpy().tolist() + [T] * S
    P = padded_starts(n)
    assert b.tolist() == P[:-1].tolist()
    assert e.tolist() == [int(p) + m for p, m in zip(P, n)]
    Wg, Wu = (rand((E + S, f, d), torch.bfloat16, i) * d ** -0.5 for i in (2, 3))
    Wd = rand((E + S, d, f), torch.bfloat16, 4) * f ** -0.5
    op = torch.empty_like(xp)
    moe.moe_expert_ffn_fwd(mc, xp, Wg, Wu, Wd, op, buf.ws)
    up = moe.grouped_config(buf.rows, d, f, E + S)
    down = moe.grouped_config(buf.rows, f, d, E + S)
    ws = moe.grouped_workspace(up)
    a, u = (torch.zeros(buf.rows, f, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o = torch.zeros_like(xp)
    moe.moe_grouped_mm(up, b, e, xp, Wg, a, ws)
    moe.moe_grouped_mm(up, b, e, xp, Wu, u, ws)
    h = (torch.nn.functional.silu(a.float()) * u.float()).to(torch.bfloat16)
    moe.moe_grouped_mm(down, b, e, h, Wd, o, ws)
    assert moe.moe_check_error(ws) == 0 and moe.moe_check_error(buf.ws) == 0
    live = in_groups(b.tolist(), e.tolist(), buf.rows)
    # the layer keeps a and b in fp32 where this path rounds them: three bf16 roundings a hidden value
    # (silu's derivative is below 1.1, and |silu(a)| >= |a| / 4 where that matters), one more an output
    S_ = exact_mm(b.tolist(), e.tolist(), a.abs() * u.abs() + h.abs(), Wd.abs())[0][live]
    err = (o[live].double() - op[live].double()).abs()
    assert bool((err <= 4 * 2.0 ** -8 * S_ + 2.0 ** -7 * op[live].double().abs()).all())
