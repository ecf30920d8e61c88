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
