"""Attention with modified scores gives the same bits every time, whichever row tiles a
CTA comes to take over."""

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Decode, Extend


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["none", "cap", "slopes", "window"])
def test_extend_repeats_itself(d, kind):
    import torch
    rng = np.random.default_rng(1)
    reqs = [(int(rng.integers(0, 900)), int(rng.integers(1, 400))) for _ in range(40)]
    e = Extend(reqs, 16, 4, d, seed=2)
    kw = {"none": dict(), "cap": dict(softcap=50.0), "window": dict(window=300),
          "slopes": dict(slopes=torch.full((16,), 0.01, device="cuda"))}[kind]
    e.run(**kw)
    want, wlse = (t.clone() for t in e.args[13:15])
    for _ in range(12):
        out, lse = e.args[13].fill_(7.0), e.args[14].fill_(7.0)
        rx.extend_attention_mod(*e.args)
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
def test_decode_repeats_itself(d):
    import torch
    c = Decode([40 + 13 * i for i in range(90)], 1111, 8, 2, d, seed=1)
    c.run(softcap=30.0)
    out, lse = (t.clone() for t in c.args[10:12])
    for _ in range(12):
        c.args[10].fill_(7.0)
        rx.decode_attention_mod(*c.args)
        assert torch.equal(c.args[10], out) and torch.equal(c.args[11], lse)
    assert rx.device_check() == 0
