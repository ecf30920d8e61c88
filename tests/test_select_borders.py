"""Expert selection (GPU) where 32 bits are not enough to tell who wins: biases of the type's lowest value, groups whose
two largest keys cancel, sums past the largest number, tokens of one logit.  Experts have to be those of keys in 64 bits,
weights and gradients within the tolerances of test_select."""
import pytest
import torch

from test_select import INF, TYPES, check, rand

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(6, 4, {}), (5, 2, {}), (8, 6, {}), (11, 7, {}), (20, 7, {}), (24, 12, {}), (32, 6, {}), (29, 20, {}),
                                        (200, 9, {}), (32, 5, dict(groups=4, top=2)), (30, 5, dict(groups=5, top=2)),
                                        (64, 6, dict(groups=8, top=3))])
def test_biases_of_the_lowest_value(moe, E, k, groups, score):
    """Experts switched off by the lowest bias there is, until fewer than the slots are left: what is switched off comes
    after all others and before the masked, and no expert of a dropped group or past the last one is chosen.
    (The bound on candidates, less what keys may be off, would be -inf.)"""
    for left in (0, 1, k - 1, k, k + 1):
        l, b = rand((70, E), left), rand((E,), left + 1, 0.1)
        b[torch.randperm(E, device="cuda", generator=torch.Generator("cuda").manual_seed(left))[left:]] = LOWEST
        l[3:20, ::3] = -INF
        l[-1, : E // 2] = -INF
        for renorm in (0, 1):
            check(moe, l, b, k, score, renorm=renorm, **groups)


# groups that fall on lanes, and groups that do not
LAYOUTS = [(256, dict(groups=8, top=4, group_top=2)), (120, dict(groups=5, top=2, group_top=2))]


@pytest.mark.parametrize("per", [4, 5])
def test_two_keys_that_cancel(moe, per):
    """Biases of 1000 and -1000 are in a group's two largest keys, whose sum is about 1: in 32 bits each key has lost 2^-15,
    and the sums of 1.000040 and 1.000031 are 1.0 and 1.000061."""
    b = torch.full((2 * per,), -3000.0, device="cuda")
    b[0::per], b[1::per] = 1000.0, -1000.0
    l = torch.zeros(3, 2 * per, device="cuda")
    s = torch.tensor([0.50002, 0.50002, 0.500031, 0.4999999], dtype=torch.float64)
    l[1, [0, 1, per, per + 1]] = torch.logit(s).float().cuda()
    check(moe, l, b, 2, "sigmoid", groups=2, top=1, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", LAYOUTS)
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e9])
def test_groups_with_large_biases_of_both_signs(moe, size, E, groups, score):
    T, per = 3000, E // groups["groups"]
    l = rand((T, E), int(size) % 1000 + E)
    g = torch.Generator("cuda").manual_seed(E)
    one = torch.full((E,), -size, device="cuda")
    one[::per] = size                                             # one of every group above, the rest below
    some = torch.where(torch.rand(E, device="cuda", generator=g) < 0.5, size, -size)
    some[: 2 * per] = -size
    some[per] = size                                              # (a group of one sign, one with a single large key)
    few = torch.zeros(E, device="cuda")
    few[per + 1 : 2 * per] = -size                                # a group of one expert and others switched off
    few[2 * per : 3 * per] = -size                                # and of none else
    for b in (one, some, few, one + rand((E,), 1, 0.1)):
        check(moe, l, b, 6, score, renorm=1, **groups)
    check(moe, l.bfloat16(), one, 6, score, renorm=1, **groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("per", [8, 5])
def test_sums_past_the_largest_number(moe, per, score):
    """Groups whose two largest biases add up beyond fp32: by their sums all the same, before an infinite one and the masked
    last."""
    n = 8
    l = rand((90, n * per), per)
    l[5:9, :: 2] = -INF
    b = torch.zeros(n * per, device="cuda")
    top = b.view(n, per)
    top[:] = -3.3e38
    for sign in (1.0, -1.0):
        for g, (x, y) in enumerate([(3.0, 0.5), (3.0, 1.0), (3.0, 3.0), (3.2, 3.1), (2.0, 1.0), (3.0, 3.0)]):
            top[g, 0], top[g, 1] = sign * x * 1e38, sign * y * 1e38
        for last in (LOWEST, -INF, INF, 0.0):
            top[6] = last
            top[7, 1:] = LOWEST     # a group of one and others switched off: its sum is below the lowest number, too
            top[7, 0] = 0.0
            for keep in (1, 2, 3, 5, 7):
                check(moe, l, b, min(6, keep * per), score, renorm=1, groups=n, top=keep, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", LAYOUTS)
def test_groups_switched_off_by_the_lowest_value(moe, E, groups, score):
    """Two, one or no expert of a group left by biases of the lowest value, beside masked groups."""
    n, per = groups["groups"], E // groups["groups"]
    l, b = rand((200, E), E), rand((E,), 1, 0.1)
    l[10:60, :per] = -INF
    l[40:90, (n - 1) * per :] = -INF
    l[100:, ::3] = -INF
    b[2:per] = LOWEST
    b[per + 1 : 2 * per] = LOWEST
    b[2 * per : 4 * per] = LOWEST
    for top in range(1, n):
        check(moe, l, b, 6, score, renorm=1, **{**groups, "top": top})


@pytest.mark.parametrize("E,n", [(64, 8), (256, 8), (40, 5), (120, 5), (1024, 64)])
def test_flat_tokens_of_uneven_groups(moe, E, n):
    """Tokens of one logit whose masks leave some groups a single expert: the score of those is one key, that of the others
    two, also where 32 bits hold the key as 0, or as near to it as its error, of either sign."""
    per = E // n
    at = torch.arange(E, device="cuda")
    for top in (1, 2, n - 1):
        for x, b in ((-100.0, None), (-600.0, None), (0.0, None), (0.0, -0.5), (-100.0, 0.0), (1.0, -0.7310586), (1.0, -0.73105854),
                     (-3.0, -0.04742587), (-3.0, -0.047425874), (12.0, -1.0), (3.0, 5.0)):
            l = torch.full((8, E), x, device="cuda")
            l[1, 1:per] = -INF                           # the first group has one expert
            l[2, (at >= per) & (at % per != per - 1)] = -INF   # all but the first
            l[3, at % (2 * per) >= 1] = -INF             # every other one, the rest none
            l[4, at % per != 0] = -INF                   # all
            l[5, (n - 1) * per + 1 :] = -INF             # the last
            l[6, (at % (2 * per) >= 1) & (at % (2 * per) < per)] = -INF
            bias = None if b is None else torch.full((E,), b, device="cuda")
            check(moe, l, bias, min(4, top), "sigmoid", renorm=1, groups=n, top=top, group_top=2)
            if b is not None:
                check(moe, l, bias, min(4, top), "softmax", renorm=1, groups=n, top=top, group_top=2)


@pytest.mark.parametrize("per", [8, 5])
def test_groups_of_subnormal_logits(moe, per):
    """Without biases groups go by their largest logits as they are, to the last bit of the smallest numbers."""
    n, T = 8, 60
    step = torch.finfo(torch.float32).smallest_normal * 2.0 ** -23
    g = torch.Generator("cuda").manual_seed(per)
    l = torch.randint(-5, 6, (T, n * per), device="cuda", generator=g).float() * step
    assert bool((l != 0).any())
    for score in ("softmax", "sigmoid"):
        for top in (1, 4, 7):
            check(moe, l, None, min(6, top * per), score, renorm=1, groups=n, top=top, group_top=1)
