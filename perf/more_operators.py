"""Workloads of the expert selection and of the 4-bit grouped product, for timing and for comparing outputs.

``select``  tokens to experts from router logits: softmax or sigmoid scores, a balance bias that only the
            selection sees, groups of experts, top-k, weights renormalised and scaled
``bwd``     its gradient: dlogits from the gradient of the weights, the selection held
``mx``      rows quantised to microscaled 4-bit floating point (e2m1 codes, a power-of-two scale for every 32
            values), times the weights of each row's group, which are kept in that form

With ``own`` false they run in a plain form of elementary torch operations, with ``own`` true through the
framework's entry points.  ``exact`` computes them in 64 bits from the definitions.  The selection's keys are
formed in 64 bits in the plain form too: the order of two experts may hang on their last bits.

An ``mx`` case: ``rows`` rows spread over ``groups`` groups in proportion to rank ** -skew, the last ``idle``
groups (before the order of the groups is shuffled) left without rows; ``padded`` starts every group on a
multiple of 256 rows, as the layer's dispatch lays them out, and leaves gaps between them.
"""
import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BLOCK = 32
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    def sel(name, op, T, E, k, score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, bias=False,
            masked=False, dtype="fp32"):
        return dict(name=name, op=op, T=T, E=E, k=k, score=score, groups=groups, top_groups=top_groups,
                    group_top=group_top, renorm=renorm, scale=scale, bias=bias, masked=masked, dtype=dtype)

    def mx(name, rows, n_in, n_out, groups, skew=0.0, idle=0, padded=False, dtype="bf16"):
        return dict(name=name, op="mx", rows=rows, n_in=n_in, n_out=n_out, groups=groups, skew=skew, idle=idle,
                    padded=padded, dtype=dtype)

    deep = dict(groups=8, top_groups=4, group_top=2, scale=2.5, bias=True)
    return [
        # one token of a decode step, fine-grained experts in groups
        sel("select 1 token", "select", 1, 256, 8, "sigmoid", **deep),
        # a decode batch, some experts out of service
        sel("select 61 tokens", "select", 61, 64, 6, "softmax", bias=True, masked=True, dtype="bf16"),
        # a training batch of a layer with few large experts
        sel("select 8192 tokens", "select", 8192, 8, 2, "softmax"),
        # a training batch, fine-grained experts in groups
        sel("select 65536 tokens", "select", 65536, 256, 8, "sigmoid", **deep),
        # a small batch with an odd number of experts, gates as the softmax gives them
        sel("bwd 1000 tokens", "bwd", 1000, 40, 5, "softmax", renorm=False, dtype="fp16"),
        # the training batches' gradients
        sel("bwd 16384 tokens", "bwd", 16384, 128, 8, "softmax", renorm=False),
        sel("bwd 65536 tokens", "bwd", 65536, 256, 8, "sigmoid", **deep),
        # one token of a decode step, top 8 of 128 fine-grained experts: only 8 weights are read
        mx("mx 1 token", 8, 2048, 768, 128),
        # a decode batch of 64 sequences, top 6 of 64 experts: a few rows for every weight
        mx("mx 64 tokens", 384, 2048, 1408, 64, skew=0.5),
        # a prompt of about 4096 tokens, top 4 of 128 wide experts, an odd number of rows
        mx("mx 4096 tokens", 16381, 2880, 2880, 128, skew=0.7, idle=3, dtype="fp16"),
        # a prompt of 4096 tokens, top 6 of 64 experts
        mx("mx 4096 fine tokens", 24576, 2048, 1408, 64, skew=0.5),
        # a batch of 8192 tokens, top 2 of 8 large experts, on the dispatch's padded rows
        mx("mx 8192 tokens", 16384, 4096, 14336, 8, skew=0.2, padded=True),
    ]


def draw(rng):
    def spread(lo, hi, step=1):
        return max(lo, int(round(lo * (hi / lo) ** rng.random() / step)) * step)

    op = rng.choice(["select", "bwd", "mx"])
    if op != "mx":
        while True:
            groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
            E = groups * max(1, round(spread(2, 512) / groups))
            top = rng.randint(1, groups)
            most = top * (E // groups)
            k = spread(1, min(16, most))
            case = dict(op=op, T=spread(1, 65536), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                        top_groups=top, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                        scale=rng.choice([1.0, 2.5, 16.0]), bias=rng.random() < 0.5, masked=rng.random() < 0.25,
                        dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
            # (one weight of a renormalised token is 1, and has no gradient)
            if case["T"] * E <= 65536 * 256 and not (op == "bwd" and case["renorm"] and k == 1):
                return case
    while True:
        groups = spread(1, 128)
        case = dict(op=op, rows=spread(1, 65536), n_in=spread(128, 14336, 32), n_out=spread(128, 14336, 8),
                    groups=groups, skew=round(rng.choice([0.0, rng.random()]), 3),
                    idle=rng.randrange(0, max(1, groups // 4)), padded=rng.random() < 0.25,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
        # no larger than the largest listed cases: their operations, weights, and rows of the plain
        # form, which computes every group at the size of the largest
        weight, most = case["n_in"] * case["n_out"], groups * int(_sizes(case).max())
        if (2 * case["rows"] * weight <= 1.9e12 and 2 * most * weight <= 3.7e12 and groups * weight <= 1.1e9
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


def _levels(v):
    """v [.., K] in 32 bits as the levels of e2m1 codes [.., K / 32, 32] and scale exponents [.., K / 32]:
    2 ** (floor(log2(largest)) - 2), and v over it to the nearest level, ties to the even code, 6 at most."""
    b = v.float().unflatten(-1, (-1, _BLOCK))
    top = b.abs().amax(-1)
    x = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    q = torch.ldexp(b, -x[..., None])
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0) * torch.sign(q), x


def _packed(v):
    """v [.., K] as codes [.., K / 2], two to a byte, the even one low, and scale bytes [.., K / 32], which lie in
    rows of a multiple of 16."""
    q, x = _levels(v)
    level = torch.tensor(_LEVELS, device=v.device)
    code = torch.searchsorted(level, q.abs()) + 8 * (q < 0)
    code = code.flatten(-2).unflatten(-1, (-1, 2)).to(torch.uint8)
    scales = torch.zeros(*x.shape[:-1], (x.shape[-1] + 15) // 16 * 16, dtype=torch.uint8, device=v.device)
    scales[..., : x.shape[-1]] = (x + 127).to(torch.uint8)
    return code[..., 0] | code[..., 1] << 4, scales


def _values(codes, scales, dtype=torch.float32):
    """The inverse: [.., K] in the type given."""
    level = torch.tensor([*_LEVELS, *(-v for v in _LEVELS)], dtype=dtype, device=codes.device)
    q = level[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()].unflatten(-1, (-1, _BLOCK))
    x = scales[..., : q.shape[-2]].int() - 127
    return torch.ldexp(q, x[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    t = _TYPES[case["dtype"]]
    if case["op"] == "mx":
        G, K, N = case["groups"], case["n_in"], case["n_out"]
        begin, end, rows = _segments(case, seed)
        s = dict(op="mx", most=int((end - begin).max()), begin=torch.tensor(begin, dtype=torch.int32, device="cuda"),
                 end=torch.tensor(end, dtype=torch.int32, device="cuda"), x=normal(rows, K, dtype=t))
        s["x"][:, :: 97] *= 8   # the large channels that trained models have
        s["out"] = torch.bfloat16 if t == torch.float32 else t
        s["wq"] = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
        s["ws"] = torch.empty(G, N, (K // _BLOCK + 15) // 16 * 16, dtype=torch.uint8, device="cuda")
        for e in range(G):
            s["wq"][e], s["ws"][e] = _packed(normal(N, K, std=K ** -0.5))
        if own:
            import mixture_experts_layer_10_gb300 as moe
            s["cfg"] = moe.grouped_config(rows, K, N, G, dtype=s["out"])
            s["work"] = moe.grouped_workspace(s["cfg"])
            s["codes"] = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(rows, s["ws"].shape[2], dtype=torch.uint8, device="cuda")
            s["y"] = torch.zeros(rows, N, dtype=s["out"], device="cuda")
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s = dict(case)
    # a router's logits: every token's own, around the experts' popularity
    s["logits"] = (normal(T, E, std=1.5) + normal(E, std=0.5)).to(t)
    if case["masked"]:
        s["logits"][:, torch.randperm(E, generator=g, device="cuda")[: E // 8]] = float("-inf")
        s["logits"][1::50] = float("-inf")   # tokens that may go nowhere
    s["b"] = normal(E, std=0.05) if case["bias"] else None
    if case["op"] == "bwd":
        s["idx"] = _select(s)[0]
        s["dw"] = normal(T, k)
    if own:
        import mixture_experts_layer_10_gb300 as moe
        s["cfg"] = moe.select_config(T, E, k, score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                     group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"], dtype=t)
        if case["op"] == "select":
            s["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["w"] = torch.empty(T, k, device="cuda")
        else:
            s["dl"] = torch.empty(T, E, dtype=t, device="cuda")
    return s


def _scores(s, dtype):
    """Scores of all experts, 0 where the logit is -inf."""
    l = s["logits"].to(dtype)
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-1e30))
    return e / e.sum(1, keepdim=True).clamp(min=1e-300 if dtype == torch.float64 else 1e-37)


def _select(s):
    """Experts of every slot, and their weights in 64 bits."""
    p = _scores(s, torch.float64)
    key = p if s["b"] is None else p + s["b"].double()
    out = s["logits"] == float("-inf")
    key = torch.where(out, float("-inf"), key)
    n, E = s["groups"], s["E"]
    if s["top_groups"] < n:
        top = torch.sort(key.view(-1, n, E // n), dim=2, descending=True).values[:, :, : s["group_top"]]
        score = torch.where(top[:, :, 0] == float("-inf"), float("-inf"), torch.where(top == float("-inf"), 0, top).sum(2))
        rank = torch.sort(score, dim=1, descending=True, stable=True).indices
        stay = torch.zeros_like(score, dtype=torch.bool).scatter_(1, rank[:, : s["top_groups"]], True)
        # below every key and every masked one: not to be chosen at all
        order = torch.where(out, -1e300, key)
        key = torch.where(stay[:, :, None], order.view(-1, n, E // n), float("-inf")).view(-1, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, : s["k"]]
    w = p.gather(1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return idx.int(), w * s["scale"]


def _select_bwd(s):
    p, idx, c = _scores(s, torch.float32), s["idx"].long(), s["dw"]
    ps = p.gather(1, idx)
    h = ps / ps.sum(1, keepdim=True).clamp(min=1e-37) if s["renorm"] else ps
    if s["renorm"]:
        d = h * (c - (c * h).sum(1, keepdim=True))
    else:
        d = h * c
    if s["score"] == "sigmoid":
        d = d * (1 - ps)
    dl = torch.zeros_like(p).scatter_add_(1, idx, d)
    if s["score"] == "softmax" and not s["renorm"]:
        dl = dl - p * (c * ps).sum(1, keepdim=True)
    return (dl * s["scale"]).to(s["logits"].dtype)


def _mx(s):
    q, x = _levels(s["x"])
    v = torch.ldexp(q, x[..., None]).flatten(-2)
    at = s["begin"].long()[:, None] + torch.arange(s["most"], device="cuda")
    live = at < s["end"].long()[:, None]
    by_group = v[torch.where(live, at, 0)] * live[..., None]
    y = torch.bmm(by_group, _values(s["wq"], s["ws"]).transpose(1, 2))
    # back to rows, zero in those of no group
    r = torch.arange(len(v), device="cuda")
    g = torch.searchsorted(s["end"].long(), r, right=True).clamp(max=len(s["end"]) - 1)
    at = r - s["begin"].long()[g]
    live = (at >= 0) & (r < s["end"].long()[g])
    return torch.where(live[:, None], y[g, at.clamp(0, s["most"] - 1)], 0).to(s["out"])


def run(s):
    if not own:
        if s["op"] == "select":
            idx, w = _select(s)
            return idx, w.float()
        return _select_bwd(s) if s["op"] == "bwd" else _mx(s)
    import mixture_experts_layer_10_gb300 as moe
    if s["op"] == "select":
        moe.moe_select(s["cfg"], s["logits"], s["b"], s["idx"], s["w"])
        return s["idx"], s["w"]
    if s["op"] == "bwd":
        moe.moe_select_bwd(s["cfg"], s["logits"], s["idx"], s["dw"], s["dl"])
        return s["dl"]
    moe.moe_quantize_rows_mxf4(s["x"], s["codes"], s["scales"])
    moe.moe_grouped_mm_mxf4(s["cfg"], s["begin"], s["end"], s["codes"], s["scales"], s["wq"], s["ws"], s["y"], s["work"])
    return s["y"]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "mx":
        n = _sizes(case)
        rows, live, K, N = int(n.sum()), int((n > 0).sum()), case["n_in"], case["n_out"]
        return {"bytes": rows * (size * K + 2 * N) + live * N * (K // 2 + K // _BLOCK), "flops": 2 * rows * K * N}
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "select":
        return {"bytes": T * (E * size + 8 * k) + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    reads = E if case["score"] == "softmax" and not case["renorm"] else k
    return {"bytes": T * ((E + reads) * size + 8 * k), "flops": T * (4 * reads + 8 * k)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "mx":
        begin, end, rows = _segments(case, seed)
        v = s["x"].double().cpu().numpy() if s["x"].numel() < 1 << 22 else None
        if v is None:
            q, x = _levels(s["x"])
            v = torch.ldexp(q.double(), x[..., None]).flatten(-2)
        else:   # the levels by distance, on the host
            b = v.reshape(rows, -1, _BLOCK)
            top = np.abs(b).max(2)
            x = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 2, -127)
            q = np.abs(b) / np.exp2(x)[..., None]
            level = np.array([0, 2, 4, 6, 1, 3, 5, 7])   # the even codes first: they win ties
            far = np.abs(q[..., None] - np.array(_LEVELS)[level])
            q = np.array(_LEVELS)[level[far.argmin(-1)]] * np.sign(b)
            v = torch.tensor((q * np.exp2(x)[..., None]).reshape(rows, -1), device="cuda")
        y = v.new_zeros(rows, case["n_out"])
        for e, (a, b) in enumerate(zip(begin.tolist(), end.tolist())):
            if b > a:
                y[a:b] = v[a:b] @ _values(s["wq"][e], s["ws"][e], torch.float64).mT
        return y
    l, scale = s["logits"].double(), case["scale"]
    masked = torch.isinf(l)
    if case["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
    if case["op"] == "bwd":
        p = p.clone().requires_grad_()
        w = p.gather(1, s["idx"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        w.backward(scale * s["dw"].double())
        d = p.grad * p.detach()
        p = p.detach()
        return d * (1 - p) if case["score"] == "sigmoid" else d - p * d.sum(1, keepdim=True)
    idx, _ = _select(s)
    w = p.gather(1, idx.long())
    w = torch.where(masked.gather(1, idx.long()), 0.0, w)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return None, w * scale
