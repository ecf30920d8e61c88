"""Microscaled 4-bit floating point (GPU): the quantiser against the format's definition, bit for bit, and the grouped
product against the definition in 64 bits, over group lengths, widths, types, strides and gaps.

Tolerance of the product: as of the other grouped products, an output is rounded once to its type, and before that
each of the L products and L / 16 partial sums of a result loses at most one unit of 2^-23 of the sum of the products'
magnitudes.
"""
import pytest
import torch

from test_grouped import GROUPS, TYPES, check, dev_i32, in_groups, layout, rand

pytestmark = pytest.mark.gpu

LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
WIDTHS = [(32, 8), (64, 128), (96, 264), (512, 136), (1056, 24), (160, 1032), (2880, 72)]
SOURCES = {**TYPES, "fp32": torch.float32}


def stride(cols):
    return (cols // 32 + 15) // 16 * 16


def values(codes, scales):
    """The values in 64 bits; NaN where a scale is 255."""
    level = torch.tensor(LEVELS + [-v for v in LEVELS], dtype=torch.float64, device=codes.device)
    q = level[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()].unflatten(-1, (-1, 32))
    x = scales[..., : q.shape[-2]].double()
    x = torch.where(x == 255, float("nan"), torch.exp2(x - 127))
    return (q * x[..., None]).flatten(-2)


def definition(v):
    """Codes (4 bits, unpacked) and scale bytes of v [.., cols], by distance to the levels."""
    b = v.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    e = torch.floor(torch.log2(torch.where(bad | (top == 0), 1.0, top)))
    e = torch.where(torch.exp2(e) > top, e - 1, e)      # (log2 near a power of two)
    e = torch.where(torch.exp2(e + 1) <= top, e + 1, e)
    x = torch.where(top == 0, -127.0, (e - 2).clamp(-127, 127))
    q = b / torch.exp2(x)[..., None]
    even_first = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=v.device)
    far = (q.abs()[..., None] - torch.tensor(LEVELS, dtype=torch.float64, device=v.device)[even_first]).abs()
    code = even_first[far.argmin(-1)] + 8 * (torch.signbit(b)).long()
    code = torch.where(bad[..., None], 0, code)
    return code.flatten(-2), torch.where(bad, 255, (x + 127).long())


def quantise(moe, v, stream=None):
    codes = torch.full((*v.shape[:-1], v.shape[-1] // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((*v.shape[:-1], stride(v.shape[-1])), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows_mxf4(v, codes, scales, stream)
    return codes, scales


def same_as_definition(moe, v):
    codes, scales = quantise(moe, v)
    want, x = definition(v)
    got = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    assert torch.equal(scales[..., : x.shape[-1]].long(), x)
    assert bool((scales[..., x.shape[-1]:] == 0).all())
    # (the sign of a zero is its value's, or none)
    zero = (want & 7) == 0
    assert torch.equal(torch.where(zero, 0, want), torch.where(zero & ((got & 7) == 0), 0, got))


@pytest.mark.parametrize("dtype", list(SOURCES))
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 96), (100, 2880), (33, 4096), (5, 65536), (1000, 160), (257, 512),
                                       (129, 1056), (0, 64)])
def test_quantiser(moe, rows, cols, dtype):
    v = rand((rows, cols), SOURCES[dtype], 3)
    v[:, ::7] *= 16
    same_as_definition(moe, v)


@pytest.mark.parametrize("dtype", list(SOURCES))
def test_quantiser_ends(moe, dtype):
    """Every half step between levels at many exponents, zeros, subnormal and largest numbers, NaN and infinities."""
    t = SOURCES[dtype]
    half = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.5, 7.75], device="cuda")
    row = torch.cat([half, -half, half[:14] * 1.0625, torch.zeros(14, device="cuda")])[:64]
    row = torch.stack([row, row.flip(0)]).flatten()
    lo, hi = (-14, 12) if t == torch.float16 else (-120, 120)
    v = torch.cat([row[None] * 2.0 ** e for e in range(lo, hi, 3)]).to(t)
    same_as_definition(moe, v)
    f = torch.finfo(t)
    ends = torch.zeros(10, 64, dtype=t, device="cuda")
    ends[1, 3] = f.max
    ends[2] = -f.max
    ends[3, 40] = f.smallest_normal
    ends[4] = f.smallest_normal / 4
    ends[5, 7], ends[6, 7], ends[7, 40] = float("nan"), float("inf"), -float("inf")
    ends[8] = -0.0
    ends[9, :32] = torch.linspace(-1, 1, 32, device="cuda").to(t) * f.smallest_normal
    same_as_definition(moe, ends)


def operands(moe, rows, G, K, N, pad=0, seed=0):
    x = rand((rows, K), torch.bfloat16, seed)
    x[:, ::37] *= 8
    W = rand((G, N, K), torch.bfloat16, seed + 1) * K ** -0.5
    q, s = quantise(moe, x)
    if pad:
        room = torch.full((rows, (K + pad) // 2), 0x77, dtype=torch.uint8, device="cuda")
        room[:, : K // 2] = q
        q = room[:, : K // 2]
    return q, s, *quantise(moe, W)


def exact(begin, end, x, W):
    y = torch.zeros(x.shape[0], W.shape[1], dtype=torch.float64, device="cuda")
    S = torch.zeros_like(y)
    for g, (a, b) in enumerate(zip(begin, end)):
        y[a:b] = x[a:b] @ W[g].T
        S[a:b] = x[a:b].abs() @ W[g].abs().T
    return y, S


def run(moe, begin, end, rows, K, N, dtype, pad=0, seed=0, extra_rows=0):
    rows += extra_rows
    G = len(begin)
    q, s, Wq, Ws = operands(moe, rows, G, K, N, pad, seed)
    cfg = moe.grouped_config(rows, K, N, G, dtype=dtype, in_stride=K + pad if pad else 0, out_stride=N + 8 if pad else 0)
    ws = moe.grouped_workspace(cfg)
    live = in_groups(begin, end, rows)
    s[~live] = 255   # rows of no group are NaN
    s[:, K // 32:] = 255   # and nothing reads the bytes behind a row's scales
    Ws[..., K // 32:] = 255
    y = torch.full((rows, N + (8 if pad else 0)), 7.0, dtype=dtype, device="cuda")
    moe.moe_grouped_mm_mxf4(cfg, dev_i32(begin), dev_i32(end), q, s, Wq, Ws, y[:, :N], ws)
    assert moe.moe_check_error(ws) == 0
    assert bool((y[~live] == 7).all()) and bool((y[:, N:] == 7).all())
    ref, S = exact(begin, end, torch.nan_to_num(values(q, s)), values(Wq, Ws))
    check("y", y[live][:, :N], ref[live], S[live], K)
    return y


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("groups", list(GROUPS))
def test_product(moe, groups, K, N, dtype):
    begin, end, rows = layout(GROUPS[groups])
    run(moe, begin, end, rows, K, N, TYPES[dtype])


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159, 160, 161, 191, 192, 193,
                               224, 225, 255, 256, 257, 383, 384, 385, 400])
def test_row_tiles(moe, n):
    """A group of every length around the tiles' borders, alone and among others."""
    run(moe, [0], [n], n, 320, 136, torch.bfloat16)
    run(moe, [3, 3 + n + 2], [3 + n, 3 + n + 2 + 40], n + 50, 320, 136, torch.bfloat16)


@pytest.mark.parametrize("n", [5, 300])
def test_strides(moe, n):
    run(moe, [1, n], [n - 1, n + 30], n + 32, 224, 200, torch.float16, pad=32)


@pytest.mark.parametrize("rows,K,N,G", [(700, 14336, 64, 3), (64, 65536, 8, 2), (3, 8192, 40, 2), (2000, 4096, 4096, 3),
                                        (1024, 64, 65536, 2), (40, 4096, 4096, 1)])
def test_wide_and_long(moe, rows, K, N, G):
    cut = [rows * i // G for i in range(G + 1)]
    run(moe, cut[:-1], cut[1:], rows, K, N, torch.bfloat16)


@pytest.mark.parametrize("K", [512, 544, 1024, 1056, 1280, 1824, 2048, 2080, 2336, 4096, 4128, 14336])
def test_split_contractions(moe, K):
    """Few tiles of a contraction that pairs share: whole and broken blocks, one group, groups without rows, every
    length of a tile's rows."""
    run(moe, [0], [1], 1, K, 264, torch.bfloat16)
    run(moe, [2, 9, 9, 40], [7, 9, 33, 232], 240, K, 136, torch.float16)
    run(moe, [0, 40], [33, 500], 520, K, 520, torch.bfloat16, pad=32)


def test_split_sums_are_the_same_every_time(moe):
    rows, K, N = 24, 14336, 520
    q, s, Wq, Ws = operands(moe, rows, 1, K, N)
    cfg = moe.grouped_config(rows, K, N, 1)
    ws = moe.grouped_workspace(cfg)
    out = []
    for _ in range(20):
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_mm_mxf4(cfg, dev_i32([0]), dev_i32([rows]), q, s, Wq, Ws, y, ws)
        out.append(y)
    assert all(torch.equal(out[0], y) for y in out)


def test_long_sums_of_one_sign(moe):
    """Rows of one sign, 65536 columns: what the accumulator drops, at most a unit of 2^-23 of the sum at every 16
    products and always towards zero, shows in the mean over many outputs, where the roundings to fp16
    (half a step, 2^-11, either way) mostly cancel: 24576 of them leave at most 5 standard deviations of
    2^-11 / sqrt(3) / sqrt(24576).  A split of the contraction drops less."""
    for rows, N in ((192, 128), (192, 4096)):
        K = 65536
        x, W = (torch.rand(shape, device="cuda") + 0.25 for shape in ((rows, K), (1, N, K)))
        (q, s), (Wq, Ws) = quantise(moe, x), quantise(moe, W / K)
        cfg = moe.grouped_config(rows, K, N, 1, dtype=torch.float16)
        ws = moe.grouped_workspace(cfg)
        y = torch.empty(rows, N, dtype=torch.float16, device="cuda")
        moe.moe_grouped_mm_mxf4(cfg, dev_i32([0]), dev_i32([rows]), q, s, Wq, Ws, y, ws)
        vx, vw = values(q, s), values(Wq, Ws)[0]
        off = (y.double() - vx @ vw.T) / (vx @ vw.T)
        assert -K / 16 * 2.0 ** -23 - 9e-6 <= off.mean().item() <= 9e-6, off.mean().item()


def test_many_groups(moe):
    n = [(i * 7) % 11 for i in range(1024)]
    begin, end, rows = layout(n)
    run(moe, begin, end, rows, 128, 72, torch.bfloat16)


def test_rows_in_a_larger_buffer(moe):
    run(moe, [0, 256, 768], [3, 300, 780], 1024, 512, 264, torch.bfloat16, extra_rows=5000)


def test_range_of_scales(moe):
    """Rows and channels of very small and large values; the product's own range is fp32's."""
    K, N, rows = 256, 64, 40
    x = rand((rows, K), torch.float32, 1) * torch.exp2(torch.linspace(-60, 60, rows, device="cuda"))[:, None]
    W = rand((1, N, K), torch.float32, 2) * torch.exp2(torch.linspace(-50, 50, N, device="cuda"))[None, :, None]
    x[5], W[0, 7] = 0, 0
    (q, s), (Wq, Ws) = quantise(moe, x), quantise(moe, W)
    cfg = moe.grouped_config(rows, K, N, 1)
    ws = moe.grouped_workspace(cfg)
    y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_mm_mxf4(cfg, dev_i32([0]), dev_i32([rows]), q, s, Wq, Ws, y, ws)
    ref, S = exact([0], [rows], values(q, s), values(Wq, Ws))
    check("y", y, ref, S, K)
    assert bool((y[5] == 0).all()) and bool((y[:, 7] == 0).all())


@pytest.mark.parametrize("rows", [6, 300])
def test_nan_stays_in_its_row_and_channel(moe, rows):
    K, N, G = 256, 40, 2
    q, s, Wq, Ws = operands(moe, rows, G, K, N)
    s[1, 3] = 255
    Ws[1, 9, 7] = 255
    cfg = moe.grouped_config(rows, K, N, G)
    ws = moe.grouped_workspace(cfg)
    y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    cut = rows // 2
    moe.moe_grouped_mm_mxf4(cfg, dev_i32([0, cut]), dev_i32([cut, rows]), q, s, Wq, Ws, y, ws)
    nan = torch.zeros(rows, N, dtype=torch.bool, device="cuda")
    nan[1] = True
    nan[cut:, 9] = True
    assert torch.equal(y.isnan(), nan)


@pytest.mark.parametrize("rows", [20, 600])
def test_bad_groups(moe, rows):
    K, N = 64, 64
    q, s, Wq, Ws = operands(moe, rows, 2, K, N)
    cfg = moe.grouped_config(rows, K, N, 2)
    ws = moe.grouped_workspace(cfg)
    for begin, end in (([0, 5], [6, 9]), ([0, 5], [4, rows + 1]), ([-1, 5], [4, 9]), ([0, 9], [4, 5]), ([5, 0], [9, 4])):
        y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_mm_mxf4(cfg, dev_i32(begin), dev_i32(end), q, s, Wq, Ws, y, ws)
        assert moe.moe_check_error(ws) == 5 and bool((y == 7).all())
    moe.moe_grouped_mm_mxf4(cfg, dev_i32([0, 3]), dev_i32([3, rows]), q, s, Wq, Ws, y, ws)
    assert moe.moe_check_error(ws) == 0 and not bool((y == 7).all(1).any())


@pytest.mark.parametrize("rows", [20, 600, 9000])
def test_a_wait_that_runs_out(moe, rows):
    """One stage is never filled: the call reports it, and the next one is right."""
    K, N = 2048, 264
    q, s, Wq, Ws = operands(moe, rows, 2, K, N)
    cfg = moe.grouped_config(rows, K, N, 2)
    ws = moe.grouped_workspace(cfg)
    begin, end = dev_i32([0, rows // 2]), dev_i32([rows // 2, rows])
    y, z = (torch.empty(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_grouped_mm_mxf4(cfg, begin, end, q, s, Wq, Ws, y, ws)
    moe.moe_debug_inject(ws, -1, 20_000_000, stall_fill=1)
    moe.moe_grouped_mm_mxf4(cfg, begin, end, q, s, Wq, Ws, z, ws)
    assert moe.moe_check_error(ws) == 6
    moe.moe_debug_inject(ws, -1, 0)
    moe.moe_grouped_mm_mxf4(cfg, begin, end, q, s, Wq, Ws, z, ws)
    assert moe.moe_check_error(ws) == 0 and torch.equal(y, z)


@pytest.mark.parametrize("rows", [24, 900])
def test_captured_and_on_streams(moe, rows):
    """Two products at once on two streams with workspaces of their own; quantiser and product captured and
    replayed on new values; the same bits each time."""
    K, N, G = 1024, 520, 3
    cut = [0, rows // 4, rows // 4, rows]
    begin, end = dev_i32(cut[:-1]), dev_i32(cut[1:])
    cfg = moe.grouped_config(rows, K, N, G)
    x = [rand((rows, K), torch.bfloat16, i) for i in (1, 2)]
    W = rand((G, N, K), torch.bfloat16, 3)
    Wq, Ws = quantise(moe, W)
    qs = [quantise(moe, v) for v in x]
    y = [torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    wss = [moe.grouped_workspace(cfg) for _ in range(2)]
    for i in range(2):
        moe.moe_grouped_mm_mxf4(cfg, begin, end, *qs[i], Wq, Ws, y[i], wss[i])
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            st = torch.cuda.Stream()
            moe.moe_grouped_mm_mxf4(cfg, begin, end, *qs[i], Wq, Ws, y[2 + i], wss[i], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[3])
    buf, q, s = x[0].clone(), torch.empty_like(qs[0][0]), torch.empty_like(qs[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quantize_rows_mxf4(buf, q, s)
        moe.moe_grouped_mm_mxf4(cfg, begin, end, q, s, Wq, Ws, y[2], wss[0])
    buf.copy_(x[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[2], y[1]) and moe.moe_check_error(wss[0]) == 0


def test_serving_chain(moe):
    """A SwiGLU layer's experts in 4 bits on a selection of one's own: route, select, dispatch, quantise, gate and up as
    one product, SwiGLU, quantise, down, combine; against the same steps in 64 bits on the same codes (two bf16
    roundings on the way, and the second quantisation sees the first's: so it is taken from the kernels' own h)."""
    T, d, f, E, k = 200, 256, 192, 16, 4
    cfg = moe.config(T, d, f, E, k)
    buf = moe.Buffers.allocate(cfg)
    rows = buf.rows
    i32 = dict(dtype=torch.int32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, W_r, b = rand((T, d), torch.bfloat16, 1), rand((d, E), torch.float32, 2) * d ** -0.5, rand((E,), torch.float32, 3) * 0.05
    W1, W2 = rand((E, 2 * f, d), torch.bfloat16, 4) * d ** -0.5, rand((E, d, f), torch.bfloat16, 5) * f ** -0.5
    (q1, s1), (q2, s2) = quantise(moe, W1), quantise(moe, W2)
    idx, w, logits = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    row_of_slot, token_of_row = torch.empty(T, k, **i32), torch.empty(T * k, **i32)
    x_perm, o, y = torch.empty(rows, d, **bf), torch.zeros(rows, d, **bf), torch.empty(T, d, **bf)
    sel = moe.select_config(T, E, k, "sigmoid", groups=4, top_groups=2, group_top=2, renorm=1, scale=2.5)
    moe.moe_route(cfg, x, W_r, None, idx, w, logits, buf.ws)
    moe.moe_select(sel, logits, b, idx, w)
    moe.moe_dispatch(cfg, idx, x, counts, offsets, row_of_slot, token_of_row, x_perm, buf.ws)
    begin, end = torch.empty(E, **i32), torch.empty(E, **i32)
    moe.moe_segments(cfg, begin, end, buf.ws)
    up, down = moe.grouped_config(rows, d, 2 * f, E), moe.grouped_config(rows, f, d, E)
    ws = moe.grouped_workspace(up)
    a = torch.zeros(rows, 2 * f, **bf)
    qx = quantise(moe, x_perm)
    moe.moe_grouped_mm_mxf4(up, begin, end, *qx, q1, s1, a, ws)
    h = torch.nn.functional.silu(a[:, :f].float()).mul(a[:, f:].float()).bfloat16()
    qh = quantise(moe, h)
    moe.moe_grouped_mm_mxf4(down, begin, end, *qh, q2, s2, o, ws)
    moe.moe_combine(cfg, o, w, y, buf.ws)
    assert moe.moe_check_error(ws) == 0 and moe.moe_check_error(buf.ws) == 0
    B, N = begin.tolist(), end.tolist()
    vx, vh, v1, v2 = values(*qx), values(*qh), values(q1, s1), values(q2, s2)
    live = in_groups(B, N, rows)
    ra, Sa = exact(B, N, vx, v1)
    check("a", a[live], ra[live], Sa[live], d)
    ro, So = exact(B, N, vh, v2)
    check("o", o[live], ro[live], So[live], f)
    # y: k rows of o, each weighted, summed in 32 bits and rounded once
    chosen = torch.nn.functional.one_hot(idx.long(), E).flatten(0, 1)
    at = begin.long()[idx.long()] + (chosen.cumsum(0) - 1).gather(1, idx.long().view(-1, 1)).view(T, k)
    rows64 = o.double()[at] * w.double()[..., None]
    ref, mass = rows64.sum(1), rows64.abs().sum(1)
    assert bool(((y.double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.001 + 8 * 2.0 ** -24 * mass).all())


def test_profiler_counts_the_kernels(moe):
    rows, K, N, G = 64, 256, 64, 2
    x = rand((rows, K), torch.bfloat16, 1)
    l = rand((rows, 16), torch.float32, 2)
    cfg, mc = moe.grouped_config(rows, K, N, G), moe.config(rows, K, 64, 16, 2)
    ws, ws_layer = moe.grouped_workspace(cfg), moe.Buffers.allocate(mc).ws
    sel = moe.select_config(rows, 16, 2, "sigmoid")
    idx, w = torch.empty(rows, 2, dtype=torch.int32, device="cuda"), torch.empty(rows, 2, device="cuda")
    q, s, Wq, Ws = operands(moe, rows, G, K, N)
    moe.moe_profile_enable(True)
    moe.moe_select(sel, l, None, idx, w)
    moe.moe_select_bwd(sel, l, idx, w, torch.empty_like(l))
    moe.moe_router_wgrad(mc, x, l, torch.empty(K, 16, device="cuda"), None, ws_layer)
    quantise(moe, x)
    moe.moe_grouped_mm_mxf4(cfg, dev_i32([0, 20]), dev_i32([20, rows]), q, s, Wq, Ws, torch.empty(rows, N, dtype=torch.bfloat16, device="cuda"), ws)
    ran = {n: c for n, (ms, c) in moe.moe_profile_read().items() if c}
    moe.moe_profile_enable(False)
    assert ran == {"select": 1, "select_bwd": 1, "router_dlogits_rows": 1, "router_dwr": 1, "router_reduce": 1, "quantize_mxf4": 1,
                   "grouped_mm_mxf4": 1}


def test_offsets_past_32_bits(moe):
    """Codes, scales' rows, weights and outputs behind the 2^32nd byte: the same bits as of those rows by themselves."""
    n, K, N = 300, 8192, 72
    rows = (1 << 20) + n                         # 4.3 GB of codes
    head = rand((n, K), torch.bfloat16, 1)
    q, s = quantise(moe, head)
    W = rand((2, N, K), torch.bfloat16, 2)
    Wq, Ws = quantise(moe, W)
    codes = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(rows, stride(K), dtype=torch.uint8, device="cuda")
    codes[-n:], scales[-n:] = q, s
    wide = 4096                                  # y rows far apart: 8.6 GB
    y = torch.full((rows, wide), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = moe.grouped_config(rows, K, N, 2, out_stride=wide)
    ws = moe.grouped_workspace(cfg)
    moe.moe_grouped_mm_mxf4(cfg, dev_i32([rows - n, rows - 9]), dev_i32([rows - 9, rows]), codes, scales, Wq, Ws, y[:, :N], ws)
    assert moe.moe_check_error(ws) == 0
    ref, S = exact([0, n - 9], [n - 9, n], values(q, s), values(Wq, Ws))
    check("y", y[-n:, :N], ref, S, K)
    assert bool((y[: rows - n] == 7).all()) and bool((y[-n:, N:] == 7).all())
    del codes, scales, y
    G = 1024                                     # 4.8 GB of weights
    big = torch.zeros(G, 2304, 2048, dtype=torch.uint8, device="cuda")
    bs = torch.zeros(G, 2304, stride(4096), dtype=torch.uint8, device="cuda")
    W = rand((1, 2304, 4096), torch.bfloat16, 3)
    big[-1:], bs[-1:] = quantise(moe, W)
    x = rand((40, 4096), torch.bfloat16, 4)
    q, s = quantise(moe, x)
    cfg = moe.grouped_config(40, 4096, 2304, G)
    ws = moe.grouped_workspace(cfg)
    y = torch.empty(40, 2304, dtype=torch.bfloat16, device="cuda")
    cut = [0] * G + [40]
    moe.moe_grouped_mm_mxf4(cfg, dev_i32(cut[:-1]), dev_i32(cut[1:]), q, s, big, bs, y, ws)
    assert moe.moe_check_error(ws) == 0
    ref, S = exact([0], [40], values(q, s), values(big[-1:], bs[-1:]))
    check("y", y, ref, S, 4096)


def test_quantiser_past_32_bits(moe):
    rows, cols, n = (1 << 22) + 37, 544, 500     # 4.6 GB
    v = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    v[-n:] = rand((n, cols), torch.bfloat16, 1)
    codes, scales = quantise(moe, v)
    q, s = quantise(moe, v[-n:].clone())
    assert torch.equal(codes[-n:], q) and torch.equal(scales[-n:], s)
    assert not bool(codes[: rows - n].any()) and not bool(scales[: rows - n].any())
