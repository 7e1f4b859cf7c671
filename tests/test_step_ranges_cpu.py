"""The ends of the documented ranges of the calls between the layers: what is inside is not refused, what is outside is, also from Python,
where sizes have more than 32 bits.  Nothing here touches a GPU: calls that pass the check of sizes are refused for a missing
array, and the library is a stand-in where a call would go through."""
import pytest
import torch

import bit_grouped_expert_top_gb300 as lm
from bit_grouped_expert_top_gb300 import _abi

FAKE = 0x10000000  # an aligned address that is never dereferenced


@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 256, 272, 496, 512])
def test_rope_takes_all_of_its_documented_range(D):
    """N * (H_q + H_k) * D < 2^34, with D that divides it and D that does not."""
    def call(N, H_q, H_k):
        return lm.load().lily_rope(_abi.lily_rope_shape(N, H_q, H_k, D, 16, 0), None, H_q * D, FAKE, H_k * D, FAKE, FAKE, 1.0, FAKE,
                                   H_q * D, FAKE, H_k * D, None)

    for heads in (1, 3, 16, 1000):
        most = (2 ** 34 - 1) // (D * heads)   # the largest N inside
        H_q, H_k = (heads + 1) // 2, heads // 2
        if most < 2 ** 31:
            assert call(most, H_q, H_k) == -1, (D, heads)       # goes on to q, which is missing
            assert call(most + 1, H_q, H_k) == -2, (D, heads)
    assert call(1, 2 ** 20 - 1, 0) == (-1 if (2 ** 20 - 1) * D < 2 ** 34 else -2)
