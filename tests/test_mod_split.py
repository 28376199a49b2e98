"""Row tiles whose keys the CTAs of a cluster share, where the shares' references differ
and several of them count; and large scores whose products are exact."""

import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Extend, _check, _reference


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("shape", ["steps", "climb", "fall", "swing", "spikes"])
@pytest.mark.parametrize("reqs", [[(4500, 5)], [(4000, 33), (5300, 2)], [(8000, 120)]],
                         ids=["one_tile", "two_requests", "many_tiles"])
def test_shares_under_different_references(d, shape, reqs):
    import torch
    e = Extend(reqs, 8, 2, d, seed=11, mag=0.2)
    N = max(p + s for p, s in reqs)
    n = torch.arange(N, device="cuda").float()
    share = torch.div(n, 512, rounding_mode="floor")
    # (natural units: 50 to 76 are 72 to 110 in log2 units; a share has 512 keys and more)
    amp = {"steps": 55 + 3.5 * (share * 5 % 7), "climb": 48 + n * (28.0 / N),
           "fall": 76 - n * (28.0 / N),
           "swing": 62 * torch.sign(torch.sin(n * (math.pi / 640))),
           "spikes": torch.where(n % 701 == 11, 60 + 4 * (share % 4), torch.zeros_like(n))}[shape]
    look = torch.tensor([1.0, 1.0, -1.0, 0.01], device="cuda").repeat(e.q.shape[0], 2)
    q = e.q.float()
    q[..., :16] = look[..., None] * 0.25 / e.scale
    e.q = q.to(torch.bfloat16)
    for r, (p, s) in enumerate(e.reqs):
        slot = e.up(e.table[e.rows[r], :p + s]).long()
        k = e.k[:, :, slot].float() * 0.1
        k[..., :16] = 0.25 * amp[:p + s, None]
        e.k[:, :, slot] = k.to(torch.bfloat16)
    for mod in (dict(), dict(window=3100), dict(softcap=500.0),
                dict(slopes=torch.full((8,), 0.002, device="cuda"))):
        for dt in (torch.float32, torch.bfloat16):
            out, lse = e.run(dt, **mod)
            assert rx.device_check() == 0
            e.check(out, lse, **mod)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("reqs", [[(4500, 5)], [(300, 200), (0, 90)]], ids=["shared", "alone"])
def test_large_scores_of_exact_products(d, reqs):
    """Queries and keys of small integers times powers of two: raw scores are exact, up to
    2^13 when scaled, and no two keys of a row that count are nearer than their errors."""
    import torch
    e = Extend(reqs, 8, 2, d, seed=5, scale=0.125)
    g = torch.Generator(device="cuda").manual_seed(1)
    e.q = torch.randint(-8, 9, e.q.shape, generator=g, device="cuda").to(torch.bfloat16) * 8
    e.k = torch.randint(-8, 9, e.k.shape, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = e.run()
    assert rx.device_check() == 0
    for r, (p, s) in enumerate(reqs):
        slot = e.up(e.table[e.rows[r], :p + s]).long()
        a, pos = slice(int(e.qo[r]), int(e.qo[r + 1])), torch.arange(p, p + s, device="cuda")
        for h in range(2):
            hs = slice(4 * h, 4 * h + 4)
            o, l, A, off = _reference(e.q[a, hs], e.k[1, h, slot], e.v[1, h, slot], pos, e.scale)
            # (without the share of inexact products; moving to log2 units and to the
            # reference is left)
            x = torch.einsum("sgd,nd->sgn", e.q[a, hs].double(), e.k[1, h, slot].double())
            seen = (torch.arange(p + s, device="cuda")[None] <= pos[:, None])[:, None]
            most = torch.where(seen, x.abs() * e.scale, torch.zeros_like(x)).amax(2)
            assert most.max() > 512
            _check(out[a, hs], lse[a, hs], (o, l, A, 2.0 ** -21 * most))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("tiles", [16, 17, 19, 20, 38])
def test_as_many_row_tiles_as_clusters_may_have(d, tiles):
    """One KV head's row tiles at the ends of the cluster sizes' ranges."""
    import torch
    e = Extend([(4200, 32 * tiles - 5)], 4, 1, d, seed=7)
    out, lse = e.run(softcap=30.0)
    assert rx.device_check() == 0
    e.check(out, lse, softcap=30.0)


@pytest.mark.gpu
def test_a_first_call_may_be_captured():
    """What a cluster's size is asked of the device, also while a stream is captured (no other
    test shares keys under a high cap with slopes)."""
    import torch
    e = Extend([(4500, 5)], 8, 2, 256, seed=3)
    e.run()
    slopes = torch.full((8,), 0.01, device="cuda")
    a = list(e.args)
    a[12] = rx.score_mod(softcap=150.0, slopes=slopes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rx.extend_attention_mod(*a)
    for t in a[13:15]:
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert rx.device_check() == 0
    e.check(*a[13:15], softcap=150.0, slopes=slopes)
