"""Raw scores under a cap whose square leaves fp32."""

import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Extend


@pytest.mark.gpu
@pytest.mark.parametrize("slope", [0.0, 1.0])
def test_raw_scores_whose_square_leaves_fp32(slope):
    """Raw scores are 0 and 2^66, 2^26 apart when scaled: only the largest one's keys
    count.  (fp32 does not tell scores of 2^26 apart that differ by 2, so how these keys
    share the weight is open: an output lies between their values.)"""
    import torch
    e = Extend([(300, 70), (0, 200)], 8, 2, 128, seed=4, scale=2.0 ** -40)
    e.q.zero_()
    e.k.zero_()
    e.q[..., 3] = 2.0 ** 33
    e.k[..., 3] = 2.0 ** 33 * (torch.arange(e.k.shape[2], device="cuda") % 2)
    slopes = torch.full((8,), slope, device="cuda") if slope else None
    out, lse = e.run(softcap=2.0 ** 39, slopes=slopes)
    assert rx.device_check() == 0
    assert torch.isfinite(out[:e.total]).all() and torch.isfinite(lse[:e.total]).all()
    for r, (p, s) in enumerate(e.reqs):
        slot = e.up(e.table[e.rows[r], :p + s]).long()
        raw = e.k[1, 0, slot, 3].float()
        for i in (0, 1, s // 2, s - 1):
            top = slot[:p + i + 1][raw[:p + i + 1] == raw[:p + i + 1].max()]
            for h in range(8):
                v = e.v[1, h // 4, top].float()
                o, room = out[int(e.qo[r]) + i, h], 2.0 ** -8 * v.abs().amax(0)
                assert (o >= v.amin(0) - room).all() and (o <= v.amax(0) + room).all()
