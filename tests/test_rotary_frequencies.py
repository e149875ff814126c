"""What rotary_frequencies states of its scalings, over lengths from one token on (CPU)."""
import math

import numpy as np
import pytest

from chunkwise_linear_rnn_02_b200 import binding as gla


@pytest.mark.parametrize("R", [2, 4, 64, 128, 512])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("slow,fast", [(1.0, 32.0), (0.5, 0.75), (4.0, 1e6)])
def test_yarn_leaves_fast_pairs_and_interpolates_slow_ones(R, base, slow, fast):
    plain = gla.rotary_frequencies(R, base=base, device="cpu")[0].numpy()
    for trained in (1, 2, 5, 6, 7, 12, 13, 100, 4096, 1 << 20):
        freq, scale = gla.rotary_frequencies(R, base=base, scaling="yarn", factor=8.0, trained=trained, slow=slow, fast=fast,
                                             device="cpu")
        freq, turns = freq.numpy(), plain * trained / (2 * math.pi)
        np.testing.assert_allclose(freq[turns > fast], plain[turns > fast], rtol=1e-12)
        np.testing.assert_allclose(freq[turns < slow], plain[turns < slow] / 8, rtol=1e-12)
        assert np.all(freq <= plain * (1 + 1e-12)) and np.all(freq >= plain / 8 * (1 - 1e-12))
        assert scale == pytest.approx(0.1 * math.log(8) + 1)
