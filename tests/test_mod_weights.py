"""Softmax weights of attention with modified scores: their rounding to bf16, once."""

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Extend


@pytest.mark.gpu
@pytest.mark.parametrize("window", [3, 4, 9, 16])
def test_rows_of_few_keys_in_two_tiles(window):
    """Windows over the border of two key tiles (a row tile of one head is 128 tokens, and its
    keys are taken 64 at a time from the multiple of 16 before its first one on), where only
    keys behind the border have values: an error of such a weight is the output's, and a
    weight must not be rounded twice."""
    import torch
    e = Extend([(0, 1100)] * 6, 8, 8, 128, seed=window, mag=1.5)
    for r in range(6):
        p = np.arange(1100)
        e.v[:, :, e.up(e.table[e.rows[r], :1100][(p % 64 != 48) & (p % 64 != 0)]).long()] = 0
    for slopes in (None, torch.full((8,), 0.05, device="cuda")):
        out, lse = e.run(window=window, slopes=slopes)
        assert rx.device_check() == 0
        e.check(out, lse, window=window, slopes=slopes)
