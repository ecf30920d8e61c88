"""The router's weight gradient from given dlogits (GPU) at widths of 129 to 192 experts, whose rows are padded to 192 columns,
three quarters of a block's threads, and at those next to the other paddings."""
import pytest

import test_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,d", [(1, 160, 64), (31, 160, 128), (1000, 160, 192), (2049, 160, 256), (300, 129, 64), (513, 192, 128),
                                   (77, 193, 64), (100, 65, 128), (64, 1, 64), (97, 63, 64)])
def test_widths(moe, T, E, d):
    test_select.test_router_wgrad(moe, T, E, d)
