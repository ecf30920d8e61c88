"""Workloads of the grouped matrix products, for timing and for comparing outputs.

The operators work on rows grouped by expert: group g is rows ``begin[g] .. end[g] - 1``, and has a
weight of its own.

``mm``   y = x W[g]^T for the rows of every group (bf16 or fp16)
``bwd``  its gradients: dx = dy W[g], and dW[g] = dy^T x over the rows of the group, either written in
         the operands' type or added to a running fp32 gradient
``i8``   the rows quantised to 8-bit integers with one scale each, times weights in 8-bit integers
         with one scale per output channel

With ``own`` false they run in a plain form of elementary torch operations in 32 bits, with ``own``
true through the framework's entry points.  ``exact`` computes them in 64 bits, group by group.

A case: ``rows`` rows spread over ``groups`` groups in proportion to rank ** -skew, the last ``idle``
groups (before the order of the groups is shuffled) left without rows; ``padded`` starts every group
on a multiple of 256 rows, as the layer's dispatch lays them out, and leaves gaps between them.
"""
import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    def case(name, op, rows, n_in, n_out, groups, skew=0.0, idle=0, padded=False, dtype="bf16", dw="same"):
        return dict(name=name, op=op, rows=rows, n_in=n_in, n_out=n_out, groups=groups, skew=skew, idle=idle,
                    padded=padded, dtype=dtype, dw=dw)

    return [
        # one token of a decode step, top 8 of 128 fine-grained experts: only 8 weights are read
        case("mm 1 token", "mm", 8, 2048, 768, 128),
        # a decode batch of 64 sequences, top 6 of 64 experts: a few rows for every weight
        case("mm 64 tokens", "mm", 384, 2048, 1408, 64, skew=0.5),
        # a prompt of about 4096 tokens, top 4 of 128 wide experts, an odd number of rows
        case("mm 4096 tokens", "mm", 16381, 2880, 2880, 128, skew=0.7, dtype="fp16"),
        # a training batch of 8192 tokens, top 2 of 8 large experts, on the dispatch's padded rows
        case("mm 8192 tokens", "mm", 16384, 4096, 14336, 8, skew=0.2, padded=True),
        # a small layer with odd sizes and an expert without rows
        case("bwd 1000 rows", "bwd", 1000, 520, 264, 5, skew=1.0, idle=1, dtype="fp16"),
        # a micro-batch of 1024 tokens, top 8 of 128, added to the fp32 gradient of the step
        case("bwd 1024 tokens", "bwd", 8192, 2048, 768, 128, skew=1.0, idle=9, dw="fp32"),
        # a training batch of 16384 tokens, top 6 of 64 experts
        case("bwd 16384 tokens", "bwd", 98304, 2048, 1408, 64, skew=0.4),
        # the down projection of 8 large experts, 4096 tokens, top 2
        case("bwd 4096 tokens", "bwd", 8192, 14336, 4096, 8, skew=0.3),
        # one token of a decode step, top 2 of 8 large experts
        case("i8 1 token", "i8", 2, 4096, 14336, 8),
        # a dense projection (one group) for a small decode batch
        case("i8 dense 37 rows", "i8", 37, 4096, 4096, 1),
        # a prompt of 4096 tokens, top 6 of 64 experts
        case("i8 4096 tokens", "i8", 24576, 2048, 1408, 64, skew=0.5),
        # a batch of 8192 tokens, top 2 of 8 large experts
        case("i8 8192 tokens", "i8", 16384, 4096, 14336, 8, skew=0.2, dtype="fp16"),
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        return max(lo, int(round(lo * (hi / lo) ** rng.random() / step)) * step)

    op = rng.choice(["mm", "bwd", "i8"])
    step = 16 if op == "i8" else 8
    while True:
        groups = spread(1, 128)
        case = dict(op=op, rows=spread(1, 65536), n_in=spread(128, 14336, step), n_out=spread(128, 14336, step),
                    groups=groups, skew=round(rng.choice([0.0, rng.random()]), 3),
                    idle=rng.randrange(0, max(1, groups // 4)), padded=rng.random() < 0.25,
                    dtype=rng.choice(["bf16", "fp16"]), dw=rng.choice(["same", "fp32"]))
        # no larger than the largest listed cases: their operations, weights, and rows of the plain
        # form, which computes every group at the size of the largest
        weight, most = case["n_in"] * case["n_out"], groups * int(_sizes(case).max())
        times = 4 if op == "bwd" else 2
        if (times * case["rows"] * weight <= 1.9e12 and times * most * weight <= 3.7e12 and groups * weight <= 4.7e8
                and most * max(case["n_in"], case["n_out"]) <= 6e8):
            return case


def _sizes(case):
    """Rows of every group, largest first."""
    live = case["groups"] - case["idle"]
    p = np.arange(1, live + 1, dtype=np.float64) ** -case["skew"]
    share = case["rows"] * p / p.sum()
    n = np.floor(share).astype(np.int64)
    n[np.argsort(-(share - n), kind="stable")[: case["rows"] - int(n.sum())]] += 1
    return np.concatenate([n, np.zeros(case["idle"], np.int64)])


def _segments(case, seed):
    """(begin, end, rows of the buffers) with the groups in an order of the seed."""
    n = np.random.default_rng(seed).permutation(_sizes(case))
    room = (n + 255) // 256 * 256 if case["padded"] else n
    begin = np.cumsum(room) - room
    return begin, begin + n, int(room.sum())


def _quantised(w):
    """Codes in [-127, 127] and one scale for each row of w [.., rows, cols], in place of a checkpoint's."""
    scale = w.abs().amax(-1) / 127
    return torch.round(w / scale[..., None]).to(torch.int8), scale


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, G, K, N, t = case["op"], case["groups"], case["n_in"], case["n_out"], _TYPES[case["dtype"]]
    begin, end, rows = _segments(case, seed)

    def normal(*shape, std=1.0, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    s = dict(op=op, most=int((end - begin).max()), dw=case["dw"],
             begin=torch.tensor(begin, dtype=torch.int32, device="cuda"),
             end=torch.tensor(end, dtype=torch.int32, device="cuda"))
    s["x"] = normal(rows, K)
    if op == "i8":
        s["x"][:, :: 97] *= 8   # the large channels that trained models have
        s["wq"] = torch.empty(G, N, K, dtype=torch.int8, device="cuda")
        s["ws"] = torch.empty(G, N, dtype=torch.float32, device="cuda")
        for e in range(G):
            s["wq"][e], s["ws"][e] = _quantised(normal(N, K, std=K ** -0.5, dtype=torch.float32))
    else:
        s["w"] = normal(G, N, K, std=K ** -0.5)
    if op == "bwd":
        s["dy"] = normal(rows, N)
        if case["dw"] == "fp32":
            s["dw0"] = normal(G, N, K, dtype=torch.float32)
    if own:
        import mixture_experts_layer_10_gb300 as moe
        fp32 = case["dw"] == "fp32" and op == "bwd"
        s["cfg"] = moe.grouped_config(rows, K, N, G, dtype=t, dw_dtype=torch.float32 if fp32 else t,
                                      accumulate=int(fp32))
        s["work"] = moe.grouped_workspace(s["cfg"])
        if op == "bwd":
            s["dx"] = torch.zeros(rows, K, dtype=t, device="cuda")
            if not fp32:
                s["dwo"] = torch.empty(G, N, K, dtype=t, device="cuda")
        else:
            s["y"] = torch.zeros(rows, N, dtype=t, device="cuda")
        if op == "i8":
            s["codes"] = torch.empty(rows, K, dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    return s


def _by_group(s, v):
    """v [rows, width] as [G, most, width] in 32 bits, zero past the end of a group."""
    at = s["begin"].long()[:, None] + torch.arange(s["most"], device="cuda")
    live = at < s["end"].long()[:, None]
    return v.float()[torch.where(live, at, 0)] * live[..., None]


def _by_row(s, v, rows):
    """The inverse: v [G, most, width] as [rows, width], zero in rows of no group."""
    r = torch.arange(rows, device="cuda")
    g = torch.searchsorted(s["end"].long(), r, right=True).clamp(max=len(s["end"]) - 1)
    at = r - s["begin"].long()[g]
    live = (at >= 0) & (r < s["end"].long()[g])
    return torch.where(live[:, None], v[g, at.clamp(0, s["most"] - 1)], 0)


def _plain(s):
    x, t = s["x"], s["x"].dtype
    if s["op"] == "i8":
        scale = x.float().abs().amax(1) / 127
        scale = torch.where(scale > 0, scale, 1.0)
        codes = torch.round(x.float() / scale[:, None])
        y = _by_row(s, torch.bmm(_by_group(s, codes), s["wq"].float().transpose(1, 2)) * s["ws"][:, None, :], len(x))
        return (y * scale[:, None]).to(t)
    w = s["w"].float()
    if s["op"] == "mm":
        return _by_row(s, torch.bmm(_by_group(s, x), w.transpose(1, 2)), len(x)).to(t)
    dy = _by_group(s, s["dy"])
    dx = _by_row(s, torch.bmm(dy, w), len(x)).to(t)
    dw = torch.bmm(dy.transpose(1, 2), _by_group(s, x))
    return dx, s["dw0"].add_(dw) if s["dw"] == "fp32" else dw.to(t)


def run(s):
    if not own:
        return _plain(s)
    import mixture_experts_layer_10_gb300 as moe
    cfg, b, e, work = s["cfg"], s["begin"], s["end"], s["work"]
    if s["op"] == "mm":
        moe.moe_grouped_mm(cfg, b, e, s["x"], s["w"], s["y"], work)
        return s["y"]
    if s["op"] == "bwd":
        dw = s["dw0"] if s["dw"] == "fp32" else s["dwo"]
        moe.moe_grouped_mm_dx(cfg, b, e, s["dy"], s["w"], s["dx"], work)
        moe.moe_grouped_mm_dw(cfg, b, e, s["dy"], s["x"], dw, work)
        return s["dx"], dw
    moe.moe_quantize_rows_i8(s["x"], s["codes"], s["scales"])
    moe.moe_grouped_mm_i8(cfg, b, e, s["codes"], s["scales"], s["wq"], s["ws"], s["y"], work)
    return s["y"]


def work(case):
    n = _sizes(case)
    rows, live, G, K, N = int(n.sum()), int((n > 0).sum()), case["groups"], case["n_in"], case["n_out"]
    if case["op"] == "mm":
        return {"bytes": 2 * (rows * (K + N) + live * K * N), "flops": 2 * rows * K * N}
    if case["op"] == "i8":
        return {"bytes": 2 * rows * (K + N) + live * N * (K + 4), "flops": 2 * rows * K * N}
    dw = 8 * live * K * N if case["dw"] == "fp32" else 2 * G * K * N
    return {"bytes": 2 * (rows * (2 * K + N) + live * K * N) + dw, "flops": 4 * rows * K * N}


def exact(case, seed):
    s = prepare(case, seed)
    begin, end, rows = _segments(case, seed)
    x, op = s["x"].double(), s["op"]
    if op == "i8":
        step = x.abs().max(dim=1, keepdim=True).values / 127.0
        step[step == 0] = 1.0
        x = torch.round(x / step)
    y = x.new_zeros(rows, case["n_in"] if op == "bwd" else case["n_out"])
    dw = x.new_zeros(case["groups"], case["n_out"], case["n_in"]) if op == "bwd" else None
    for g, (a, b) in enumerate(zip(begin.tolist(), end.tolist())):
        if op == "mm":
            y[a:b] = x[a:b] @ s["w"][g].double().mT
        elif op == "i8":
            y[a:b] = step[a:b] * (x[a:b] @ (s["wq"][g].double() * s["ws"][g].double()[:, None]).mT)
        else:
            d = s["dy"][a:b].double()
            y[a:b] = d @ s["w"][g].double()
            dw[g] = d.mT @ x[a:b]
    if op != "bwd":
        return y
    return y, dw + s["dw0"].double() if case["dw"] == "fp32" else dw
