"""The expert MLP of examples/expert_mlp.py (GPU): a training step and 8-bit serving on the layer's routing
against the same MLP in plain torch.

Tolerances: the training path rounds a, h, o and their gradients to bf16, each by up to 2^-8 of a value
(about half that in the mean square), at most six such roundings on the way of an output.  8-bit codes
are off by up to half a step, 1/254 of a row's largest value; against normal values of unit size and rows
of a few hundred (largest near 3.5) that is 0.004 of unit size in the mean square, for each of the four
quantised operands.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("tokens", [1, 37, 512])
def test_expert_mlp(moe, tokens):
    import expert_mlp
    off = expert_mlp.main(["--tokens", str(tokens)])
    for what, v in off.items():
        assert v < (4 * 2 * 0.008 if "8-bit" in what else 6 * 2.0 ** -8), (what, v)
