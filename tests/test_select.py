"""Expert selection (GPU): moe_select, its gradient and the router's weight gradient against the definitions in
64 bits, over scores, groups, masks, types and sizes.

Experts have to be equal.  Tolerances of the weights: exp and the sums of at most 1024 exponentials (32 a lane and
5 steps between lanes, each addition 2^-24) are within 2^-18 of the value, and a difference x - M that goes into exp
is off by |x - M| 2^-24, which is as much of exp.  A gradient is a product of such values with c_j - sum c h, whose
terms may cancel: their magnitudes are what the error is a part of.  Each output is rounded once, by half a step.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF = float("inf")


def scores64(l, score):
    l = l.double()
    if score == "sigmoid":
        return torch.where(l == -INF, 0.0, torch.sigmoid(l))
    m = l.amax(1, keepdim=True).clamp(min=-1e300)
    e = torch.exp(l - m)
    z = e.sum(1, keepdim=True)
    return torch.where(z == 0, 0.0, e / z)


def weights64(l, idx, score, renorm, scale):
    """Weights in 64 bits of the experts given; differentiable in l."""
    if not renorm:
        return scores64(l, score).gather(1, idx) * scale
    x = l.double().gather(1, idx)
    x = torch.nn.functional.logsigmoid(x) if score == "sigmoid" else x
    live = x > -INF
    m = x.masked_fill(~live, -1e300).amax(1, keepdim=True).detach()
    e = torch.where(live, torch.exp(torch.where(live, x, m) - m), 0.0)
    z = e.sum(1, keepdim=True)
    return torch.where(z == 0, 0.0, e / z.clamp(min=1e-300)) * scale


def select64(l, b, k, score, groups, top, group_top):
    """Experts of every slot, by sorting keys in 64 bits."""
    T, E = l.shape
    # (scores rise with their logits: without anything added, the order is the logits', also where 64 bits hold
    # the scores as one number)
    key = scores64(l, score) if b is not None or (top < groups and group_top == 2) else l.double()
    if b is not None:
        key = key + b.double()
    dead = ~(l.double() > -INF) | ~(key > -INF)
    rank = torch.where(dead, -INF, key)
    if top < groups:
        per = E // groups
        best = rank.view(T, groups, per).sort(2, descending=True).values[:, :, :group_top]
        score_g = torch.where(best[:, :, 0] == -INF, -INF, torch.where(best == -INF, 0.0, best).sum(2))
        order = score_g.sort(dim=1, descending=True, stable=True).indices
        gone = torch.ones(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order[:, :top], False)
        gone = gone.repeat_interleave(per, 1)
        # (masked ones of a group that stays come before any of a group that is gone)
        rank = torch.where(gone, -INF, torch.where(dead, -1e300, rank))
    return rank.sort(dim=1, descending=True, stable=True).indices[:, :k]


def rand(shape, seed, std=1.5):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)


def run(moe, l, b, k, score="softmax", groups=1, top=None, group_top=1, renorm=0, scale=1.0, pad=3):
    """idx and weights, with the rows behind the last token checked to be left as they were."""
    T, E = l.shape
    cfg = moe.select_config(T, E, k, score, groups, top, group_top, renorm, scale, l.dtype)
    idx = torch.full((T + pad, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + pad, k), -7.0, device="cuda")
    moe.moe_select(cfg, l, b, idx[:T], w[:T])
    assert bool((idx[T:] == -7).all()) and bool((w[T:] == -7).all())
    return cfg, idx[:T], w[:T]


def check(moe, l, b, k, score="softmax", groups=1, top=None, group_top=1, renorm=0, scale=1.0, seed=0):
    T, E = l.shape
    top = groups if top is None else top
    cfg, idx, w = run(moe, l, b, k, score, groups, top, group_top, renorm, scale)
    want = select64(l, b, k, score, groups, top, group_top)
    assert torch.equal(idx.long(), want), f"{int((idx.long() != want).any(1).sum())} of {T} tokens differ"
    x = l.double()
    if renorm:
        x = torch.where(want >= 0, x.gather(1, want), 0.0)
    else:
        x = x.gather(1, want)
    m = (l.double().amax(1, keepdim=True) if not renorm else x.amax(1, keepdim=True)).clamp(min=-1e30)
    far = torch.where(x == -INF, 0.0, (x - m).abs()).clamp(max=1e4)
    ref = weights64(l, want, score, renorm, scale)
    bound = (2.0 ** -18 + far * 2.0 ** -23) * ref.abs() + 1e-36
    err = (w.double() - ref).abs()
    assert bool((err <= bound).all()), f"weights: {(err - bound).max().item():.3e}"

    # the gradient: of the reference's weights by autograd
    c = rand((T, k), seed + 77, 1.0)
    dl = torch.full((T + 2, E), -7.0, dtype=l.dtype, device="cuda")
    moe.moe_select_bwd(cfg, l, idx, c, dl[:T])
    assert bool((dl[T:] == -7).all())
    leaf = l.double().requires_grad_()
    weights64(torch.where(l == -INF, -INF, leaf), want, score, renorm, scale).backward(c.double())
    g = torch.where(l == -INF, 0.0, torch.nan_to_num(leaf.grad))
    h = (ref / scale).abs()
    mass = (c.abs() * h).sum(1, keepdim=True)
    terms = torch.zeros_like(g).scatter_add_(1, want, abs(scale) * h * (c.abs() + (mass if renorm else 0.0)))
    if score == "softmax" and not renorm:
        terms = terms + abs(scale) * scores64(l, score) * mass
    spread = far.amax(1, keepdim=True) if renorm else (l.double() - m).abs().clamp(max=1e4)
    pre = (2.0 ** -17 + spread * 2.0 ** -22) * terms + 1e-36
    bound = pre + torch.finfo(l.dtype).eps / 2 * (g.abs() + pre) + (2.0 ** -25 if l.dtype == torch.float16 else 0.0)
    err = (dl[:T].double() - g).abs()
    assert bool((err <= bound).all()), f"dlogits: {(err - bound).max().item():.3e}"


CASES = [
    (1, 1, 1, {}), (1, 2, 1, {}), (5, 7, 3, {}), (33, 8, 8, {}), (129, 9, 2, {}), (64, 16, 16, {}), (100, 24, 4, {}),
    (77, 32, 32, {}), (31, 33, 32, {}), (200, 40, 5, {}), (200, 64, 6, {}), (65, 100, 8, {}), (300, 128, 8, {}),
    (130, 129, 17, {}), (257, 256, 8, {}), (64, 320, 10, {}), (41, 512, 32, {}), (29, 777, 9, {}), (50, 1024, 8, {}),
    (257, 256, 8, dict(groups=8, top=4, group_top=2)), (100, 256, 8, dict(groups=8, top=3, group_top=1)),
    (100, 64, 6, dict(groups=4, top=2, group_top=2)), (100, 32, 4, dict(groups=4, top=1, group_top=2)),
    (100, 16, 2, dict(groups=16, top=3, group_top=2)), (90, 60, 5, dict(groups=5, top=2, group_top=2)),
    (60, 1024, 16, dict(groups=64, top=5, group_top=2)), (60, 100, 7, dict(groups=10, top=9, group_top=1)),
    (60, 512, 12, dict(groups=2, top=1, group_top=2)), (60, 8, 2, dict(groups=2, top=1, group_top=1)),
    (60, 160, 6, dict(groups=8, top=3, group_top=2)), (37, 24, 6, dict(groups=3, top=2, group_top=2)),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups", CASES)
def test_select_and_gradient(moe, T, E, k, groups, score, dtype):
    for i, (bias, renorm, scale) in enumerate([(False, 0, 1.0), (True, 1, 2.5), (True, 0, 1.0), (False, 1, 0.5)]):
        seed = 1000 * T + E + i
        l = rand((T, E), seed).to(TYPES[dtype])
        check(moe, l, rand((E,), seed + 1, 0.1) if bias else None, k, score, renorm=renorm, scale=scale, seed=seed, **groups)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(groups=8, top=3, group_top=2), dict(groups=3, top=2, group_top=2)])
def test_masks(moe, score, dtype, groups):
    """Experts out, tokens with few, one or none left, and masks of the type's lowest value."""
    T, E, k = 96, 96, 6
    for bias in (False, True):
        l = rand((T, E), 5).to(TYPES[dtype])
        l[:, ::5] = -INF
        l[1] = -INF
        l[2] = -INF
        l[2, 50] = 1.0
        l[3, :90] = -INF
        l[4, 8:] = -INF
        l[5] = torch.finfo(l.dtype).min
        l[6, 1:] = torch.finfo(l.dtype).min
        b = rand((E,), 6, 0.1) if bias else None
        if bias:
            b[7] = -INF
        for renorm in (0, 1):
            check(moe, l, b, k, score, renorm=renorm, scale=2.0, **groups)
    _, idx, w = run(moe, l, b, k, score, renorm=1, **groups)
    assert bool((w[1] == 0).all()) and len(set(idx[1].tolist())) == k
    assert bool((w[2] == torch.tensor([1.0] + [0.0] * 5, device="cuda")).all()) and int(idx[2, 0]) == 50


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(8, dict()), (64, dict(groups=8, top=4, group_top=2)), (256, dict(groups=8, top=4, group_top=2)),
                                      (120, dict(groups=5, top=2, group_top=2)), (32, dict(groups=16, top=11, group_top=2)),
                                      (25, dict(groups=5, top=1, group_top=2)), (96, dict())])
@pytest.mark.parametrize("k", [4, 13, 20])
def test_ties_and_near_ties(moe, score, E, groups, k):
    T = 200
    if k > E // groups.get("groups", 1) * groups.get("top", 1):
        pytest.skip("more slots than experts of the groups that stay")
    l = (rand((T, E), 3) * 2).round() / 4                       # equal logits in every row
    check(moe, l, None, k, score, renorm=1, **groups)
    check(moe, l, torch.zeros(E, device="cuda"), k, score, renorm=1, **groups)
    check(moe, torch.zeros(T, E, device="cuda"), None, k, score, **groups)
    check(moe, l + 30, torch.zeros(E, device="cuda"), k, score, **groups)   # sigmoids that round to 1
    check(moe, -0.0 * l.sign(), None, k, score, **groups)       # zeros of both signs
    # keys that differ by less than a step of fp32: the bias makes up for the first token's scores
    l = rand((T, E), 4)
    l[1:] = l[0] + rand((T - 1, E), 5, 1e-6)
    p = scores64(l, score)[0]
    check(moe, l, (p.max() - p).float(), k, score, renorm=1, **groups)
    # most logits equal and a few the least bit above them, at either end of the experts
    l = torch.zeros(T, E, device="cuda")
    l.scatter_(1, torch.randint(0, E, (T, 3), device="cuda", generator=torch.Generator("cuda").manual_seed(6)), 2.0 ** -24)
    check(moe, l, torch.zeros(E, device="cuda"), k, score, renorm=1)
    l[:, : E // 2] -= 1.0
    check(moe, l, torch.zeros(E, device="cuda"), k, score, renorm=1)
    # scores far below the bias's last place: the order is the bias's, then theirs
    check(moe, l - 40, torch.ones(E, device="cuda"), k, score, renorm=1, **groups)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_flat_tokens(moe, score, dtype):
    """Tokens whose logits are all one number (padding, an untrained router), some of their experts masked, one of them
    the least bit larger: with equal biases, with biases, and with one bias the least bit larger."""
    for E, k, groups in ((256, 8, dict(groups=8, top=4, group_top=2)), (256, 20, dict()), (64, 6, dict()), (40, 6, dict(groups=5, top=2, group_top=2)),
                         (512, 10, dict(groups=64, top=9, group_top=2)), (1024, 32, dict())):
        l = torch.zeros(64, E, device="cuda")
        l[8:16] = 3.0
        l[16:24, ::3] = -INF
        l[24:40].scatter_(1, torch.randint(0, E, (16, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(E)), 2.0 ** -20)
        l[40:48] = rand((8, E), E)
        l = l.to(TYPES[dtype])
        b = torch.full((E,), 0.5, device="cuda")
        for bias in (None, torch.zeros(E, device="cuda"), b, b + rand((E,), 1, 0.1)):
            check(moe, l, bias, k, score, renorm=1, **groups)
        b[E - 1] += 2.0 ** -24
        check(moe, l, b, k, score, renorm=1, **groups)


def test_large_biases(moe):
    l, b = rand((300, 64), 1), rand((64,), 2, 300.0)
    b[::2] = b[1::2]   # pairs with one bias: the scores decide
    for score in ("softmax", "sigmoid"):
        check(moe, l, b, 8, score, renorm=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases(moe, score):
    """Experts that a bias puts first or last, fewer and more than the slots."""
    for E, groups in ((64, dict()), (256, dict(groups=8, top=4, group_top=2)), (40, dict(groups=5, top=3, group_top=2))):
        for n in (1, 3, 8, 20):
            l, b = rand((60, E), n), rand((E,), n + 1, 0.1)
            b[torch.randperm(E, device="cuda", generator=torch.Generator("cuda").manual_seed(n))[:n]] = INF
            b[:3] = -INF
            check(moe, l, b, 6, score, renorm=1, **groups)


def test_far_logits(moe):
    """Scores that underflow in 32 bits: renormalised weights stay those of the scores' ratios."""
    for shift in (-60.0, -200.0, -3000.0, 100.0, 3000.0):
        l = rand((50, 32), 9) + shift
        _, idx, w = run(moe, l, None, 5, "sigmoid", renorm=1)
        assert bool(((w.sum(1) - 1).abs() < 1e-6).all())
        for score in ("softmax", "sigmoid"):
            check(moe, l, None, 5, score, renorm=1, scale=16.0)
            check(moe, l, None, 5, score)


def test_wide_logits(moe):
    """Scores of one token that lie many powers of ten apart, some of them below the smallest number of 32 bits."""
    for shift in (-60.0, -20.0, 0.0, 40.0):
        l = rand((300, 24), 11, 40.0) + shift
        for renorm in (0, 1):
            for k in (3, 12):
                check(moe, l, None, k, "sigmoid", renorm=renorm, scale=1.5)
                check(moe, l, None, k, "softmax", renorm=renorm, scale=1.5)


def test_nan_and_infinite_logits(moe):
    l = rand((4, 64), 2)
    l[0, 10] = float("nan")
    l[1, 20] = INF
    l[2] = float("nan")
    for score in ("softmax", "sigmoid"):
        for renorm in (0, 1):
            for b in (None, rand((64,), 3, 0.1)):
                _, idx, w = run(moe, l, b, 6, score, groups=4, top=3, group_top=2, renorm=renorm)
                for t in range(4):
                    assert len(set(idx[t].tolist())) == 6 and int(idx[t].min()) >= 0 and int(idx[t].max()) < 64
                assert 10 not in idx[0].tolist() and bool(torch.isfinite(w[3]).all())
                nan = w.isnan().all(1).tolist()
                assert nan[2] and (nan[0] == (score == "softmax" and not renorm))
                if score == "softmax":
                    assert w[1].isnan().any()
                elif b is None:   # a sigmoid of 1, as the largest
                    assert int(idx[1, 0]) == 20 and bool(torch.isfinite(w[1]).all())


def test_gradient_of_slots_given_by_hand(moe):
    """Indices out of range, the same expert twice, weights that are nothing with gradients that are no numbers."""
    T, E, k = 6, 40, 4
    l = rand((T, E), 8)
    c = rand((T, k), 9, 1.0)
    idx = torch.tensor([[3, 3, 5, 7], [0, -1, 40, 2], [-1, -1, -1, -1], [39, 1 << 30, 0, 1], [1, 2, 3, 4], [9, 8, 7, 6]],
                       dtype=torch.int32, device="cuda")
    l[4, 2] = -INF
    c[4, 1] = float("nan")
    for score in ("softmax", "sigmoid"):
        for renorm in (0, 1):
            cfg = moe.select_config(T, E, k, score, renorm=renorm, scale=1.5)
            dl = torch.empty(T, E, device="cuda")
            moe.moe_select_bwd(cfg, l, idx, c, dl)
            for t in range(T):
                use = [j for j in range(k) if 0 <= int(idx[t, j]) < E and not (t == 4 and j == 1)]
                leaf = l[t:t + 1].double().requires_grad_()
                if use:
                    at = idx[t:t + 1, use].long()
                    weights64(leaf, at, score, renorm, 1.5).backward(c[t:t + 1, use].double())
                    ref = torch.nan_to_num(leaf.grad[0])
                else:
                    ref = torch.zeros(E, dtype=torch.float64, device="cuda")
                assert bool(((dl[t].double() - ref).abs() <= 2e-5).all()), (score, renorm, t)


def test_differences_of_the_forward(moe):
    """The gradient against central differences of the kernel's own weights: with a step of 2^-6 these are off by
    step^2 / 6 of third derivatives below 1 and by two roundings of weights (2^-18) over twice the step."""
    T, E, k, step = 8, 24, 3, 2.0 ** -6
    l = rand((T, E), 12)
    c = rand((T, k), 13, 1.0)
    for score in ("softmax", "sigmoid"):
        for renorm in (0, 1):
            cfg, idx, _ = run(moe, l, None, k, score, renorm=renorm)
            dl = torch.empty(T, E, device="cuda")
            moe.moe_select_bwd(cfg, l, idx, c, dl)
            # a bias holds the selection and its order while a logit moves
            b = torch.zeros(T, E, device="cuda").scatter_(1, idx.long(), torch.arange(30.0, 0.0, -10.0, device="cuda").expand(T, k))
            for e in range(0, E, 5):
                for t in range(T):
                    w = []
                    for sign in (1, -1):
                        m = l[t:t + 1].clone()
                        m[0, e] += sign * step
                        _, at, v = run(moe, m, b[t], k, score, renorm=renorm)
                        assert torch.equal(at[0], idx[t])
                        w.append((v[0] * c[t]).sum().item())
                    diff = (w[0] - w[1]) / (2 * step)
                    size = c[t].abs().sum().item()
                    assert abs(diff - dl[t, e].item()) <= size * (step ** 2 / 6 + 2.0 ** -18 / step) + 1e-6


def test_no_tokens(moe):
    cfg = moe.select_config(0, 8, 2)
    e = torch.empty(0, 8, device="cuda")
    moe.moe_select(cfg, e, None, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    moe.moe_select_bwd(cfg, e, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"), e)


def test_outputs_that_start_anywhere(moe):
    """idx, weights and bias that are parts of larger arrays."""
    T, E, k = 50, 33, 3
    l = rand((T, E), 3)
    b = rand((E + 1,), 4, 0.1)[1:]
    idx = torch.zeros(T * k + 1, dtype=torch.int32, device="cuda")[1:].view(T, k)
    w = torch.zeros(T * k + 1, device="cuda")[1:].view(T, k)
    moe.moe_select(moe.select_config(T, E, k, "sigmoid"), l, b, idx, w)
    assert torch.equal(idx.long(), select64(l, b, k, "sigmoid", 1, 1, 1))


def test_captured_and_on_streams(moe):
    """Two selections at once on two streams, and a captured pair of calls replayed on new logits."""
    T, E, k = 3000, 256, 8
    kw = dict(score="sigmoid", groups=8, top_groups=4, group_top=2, renorm=1, scale=2.5)
    cfg = moe.select_config(T, E, k, **kw)
    b = rand((E,), 1, 0.05)
    l = [rand((T, E), i) for i in (2, 3)]
    idx = [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in l]
    w = [torch.empty(T, k, device="cuda") for _ in l]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in l]
    for _ in range(4):
        for s, a, i, v in zip(streams, l, idx, w):
            moe.moe_select(cfg, a, b, i, v, stream=s)
    torch.cuda.synchronize()
    want = [select64(a, b, k, "sigmoid", 8, 4, 2) for a in l]
    assert all(torch.equal(i.long(), r) for i, r in zip(idx, want))
    c, dl = rand((T, k), 5, 1.0), torch.empty(T, E, device="cuda")
    buf = l[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_select(cfg, buf, b, idx[0], w[0])
        moe.moe_select_bwd(cfg, buf, idx[0], c, dl)
    buf.copy_(l[1])
    graph.replay()
    torch.cuda.synchronize()
    eager = torch.empty_like(dl)
    moe.moe_select_bwd(cfg, l[1], idx[1], c, eager)
    assert torch.equal(idx[0], idx[1]) and torch.equal(w[0], w[1]) and torch.equal(dl, eager)


@pytest.mark.parametrize("dtype,E", [("fp16", 300), ("fp32", 256)])
def test_offsets_past_32_bits(moe, dtype, E):
    """Tokens behind the 2^32nd byte of the logits: the same bits as of those tokens by themselves."""
    T, n, k = (1 << 32) // (E * (2 if dtype == "fp16" else 4)) + 1000, 500, 5
    l = torch.zeros(T, E, dtype=TYPES[dtype], device="cuda")
    l[-n:] = rand((n, E), 1).to(l.dtype)
    b, c = rand((E,), 2, 0.1), torch.zeros(T, k, device="cuda")
    c[-n:] = rand((n, k), 3, 1.0)
    for renorm in (0, 1):
        out = []
        for a, d in ((l, c), (l[-n:].clone(), c[-n:].clone())):
            cfg = moe.select_config(len(a), E, k, renorm=renorm, dtype=l.dtype)
            idx, w = torch.empty(len(a), k, dtype=torch.int32, device="cuda"), torch.empty(len(a), k, device="cuda")
            dl = torch.empty_like(a)
            moe.moe_select(cfg, a, b, idx, w)
            moe.moe_select_bwd(cfg, a, idx, d, dl)
            out.append([t[-n:] for t in (idx, w, dl)])
        assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("T,E,d", [(1, 8, 64), (33, 8, 128), (1000, 40, 192), (513, 64, 64), (2049, 128, 256), (300, 200, 64),
                                   (70, 256, 128)])
def test_router_wgrad(moe, T, E, d):
    """dlogits enter the product in bf16: against the exact product of those, every product and partial sum
    losing at most 2^-23 of the sum of magnitudes; db sums them as they are."""
    cfg = moe.config(T, d, 64, E, 1)
    ws = moe.Buffers.allocate(cfg).ws
    x, dl = rand((T, d), 1).bfloat16(), rand((T, E), 2)
    dW, db = torch.empty(d, E, device="cuda"), torch.empty(E, device="cuda")
    moe.moe_router_wgrad(cfg, x, dl, dW, db, ws)
    assert moe.moe_check_error(ws) == 0
    r = dl.bfloat16().double()
    ref, S = x.double().T @ r, x.double().abs().T @ r.abs()
    assert bool(((dW.double() - ref).abs() <= (T + T // 16 + 16) * 2.0 ** -23 * S + 1e-30).all())
    assert bool(((db.double() - dl.double().sum(0)).abs() <= (T + 8) * 2.0 ** -24 * dl.double().abs().sum(0)).all())
    moe.moe_router_wgrad(cfg, x, dl, dW, None, ws)
    assert bool(((dW.double() - ref).abs() <= (T + T // 16 + 16) * 2.0 ** -23 * S + 1e-30).all())


def test_training_chain(moe):
    """Logits of moe_route, a selection of one's own, dispatch, experts, combine, and back: against the same layer
    in 64 bits (the tolerance of the layer's own parity tests: 2e-2 of the largest value and 1e-2 of each)."""
    T, d, f, E, k = 300, 128, 192, 16, 4
    cfg = moe.config(T, d, f, E, k)
    buf = moe.Buffers.allocate(cfg)
    x, dy = rand((T, d), 1, 1.0).bfloat16(), rand((T, d), 2, 1.0).bfloat16()
    W_r, b = rand((d, E), 3, d ** -0.5), rand((E,), 4, 0.02)
    Wg, Wu, Wd = (rand(s, i, s[-1] ** -0.5).bfloat16() for i, s in ((5, (E, f, d)), (6, (E, f, d)), (7, (E, d, f))))
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, gates, logits = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    row_of_slot, token_of_row = torch.empty(T, k, **i32), torch.empty(T * k, **i32)
    x_perm, o_perm, dx_perm = (torch.empty(buf.rows, d, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    sel = moe.select_config(T, E, k, "sigmoid", groups=4, top_groups=2, group_top=2, renorm=1, scale=2.0)
    moe.moe_route(cfg, x, W_r, None, idx, gates, logits, buf.ws)
    moe.moe_select(sel, logits, b, idx, gates)
    moe.moe_dispatch(cfg, idx, x, counts, offsets, row_of_slot, token_of_row, x_perm, buf.ws)
    moe.moe_expert_ffn_fwd(cfg, x_perm, Wg, Wu, Wd, o_perm, buf.ws)
    moe.moe_combine(cfg, o_perm, gates, y, buf.ws)
    dgates, dlogits = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    dWg, dWu, dWd = torch.empty_like(Wg), torch.empty_like(Wu), torch.empty_like(Wd)
    dW_r, db_r = torch.empty(d, E, device="cuda"), torch.empty(E, device="cuda")
    moe.moe_expert_ffn_bwd(cfg, x_perm, dy, gates, Wg, Wu, Wd, dx_perm, dgates, dWg, dWu, dWd, buf.ws)
    moe.moe_select_bwd(sel, logits, idx, dgates, dlogits)
    moe.moe_router_wgrad(cfg, x, dlogits, dW_r, db_r, buf.ws)
    moe.moe_combine_bwd(cfg, dx_perm, dlogits, W_r, dx, buf.ws)
    assert moe.moe_check_error(buf.ws) == 0
    assert torch.equal(idx.long(), select64(logits, b, k, "sigmoid", 4, 2, 2))

    leaves = [t.double().requires_grad_() for t in (x, W_r, Wg, Wu, Wd)]
    X, R, G, U, D = leaves
    w = weights64(X @ R, idx.long(), "sigmoid", 1, 2.0)
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(X[t] @ G[e].T) * (X[t] @ U[e].T)
        ref = ref.index_add(0, t, (h @ D[e].T) * w[t, j, None])
    ref.backward(dy.double())
    for name, got, want in (("y", y, ref.detach()), ("dx", dx, X.grad), ("dW_r", dW_r, R.grad), ("dW_gate", dWg, G.grad),
                            ("dW_up", dWu, U.grad), ("dW_down", dWd, D.grad)):
        err = (got.double() - want).abs()
        assert bool((err <= 2e-2 * want.abs().max() + 1e-2 * want.abs()).all()), name
