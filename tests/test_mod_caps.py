"""Capped scores next to scores (of other rows, or of other keys of the row) that reach
the cap, and raw scores whose square leaves fp32.

Tolerance: as in test_score_mod.py, with the cap's own error 2^-20 of the capped score, or
2^-15 under a softcap of at most 88, whatever the neighbours.
"""

import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Decode, Extend, _reference


def _check(o, lse, want, softcap):
    wo, wl, A, off = want
    cap = 2.0 ** -20 * wl.abs()  # (the scores that count are below lse)
    off = off - 2.0 ** -21 * softcap + (cap.clamp(min=2.0 ** -15) if softcap <= 88 else cap)
    tol = (2.0 ** -8 + 4 * off + 2.0 ** -16)[..., None] * A
    assert ((o.double() - wo).abs() <= tol).all(), float(((o.double() - wo).abs() / tol).max())
    err = (lse.double() - wl).abs()
    assert (err <= 2 * off + 2.0 ** -20 * (1 + wl.abs())).all(), float(err.max())


def _rows(e, out, lse, rows, softcap, slopes=None, zero=()):
    """Checks the rows at the numbers `rows` of each request; keys at slots `zero` as 0."""
    import torch
    G = e.hq // e.hkv
    for r, (p, s) in enumerate(e.reqs):
        slot = e.up(e.table[e.rows[r], :p + s]).long()
        i = torch.tensor([x for x in rows if x < s], device="cuda")
        for h in range(e.hkv):
            hs = slice(h * G, (h + 1) * G)
            a = int(e.qo[r]) + i
            k = e.k[1, h].clone()
            k[list(zero)] = 0
            kb = None if not len(zero) else torch.full_like(i, 40)
            _check(out[a][:, hs], lse[a][:, hs],
                   _reference(e.q[a][:, hs], k[slot], e.v[1, h, slot], p + i, e.scale,
                              softcap=softcap, key_begin=kb,
                              slopes=None if slopes is None else slopes[hs]), softcap)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("softcap", [50.0, 4096.0, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("slope", [0.0, 0.01])
def test_extend_rows_beside_rows_at_the_cap(d, softcap, slope):
    """Every fourth token's queries reach the cap; the rows between score a few units."""
    import torch
    e = Extend([(400, 70), (0, 200), (5, 130)], 8, 2, d, seed=3)
    e.q[::4] *= 4 * softcap
    slopes = torch.full((8,), slope, device="cuda") if slope else None
    out, lse = e.run(softcap=softcap, slopes=slopes)
    assert rx.device_check() == 0
    _rows(e, out, lse, [i for i in range(200) if all((int(q) + i) % 4 for q in e.qo[:-1])],
          softcap, slopes)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("softcap", [50.0, 2.0 ** 20])
def test_extend_keys_far_below_beside_keys_that_count(d, softcap):
    """In every row some scores lie near -softcap and weigh nothing; the rest are small."""
    import torch
    e = Extend([(400, 70), (0, 200), (5, 130)], 8, 2, d, seed=4)
    e.q[..., 0] = 4.0
    e.k[..., 0] = 0.0
    for r, (p, s) in enumerate(e.reqs):
        low = e.up(e.table[e.rows[r], 5:p + s:9]).long()
        e.k[:, :, low, 0] = -softcap * math.sqrt(d) / 4
    out, lse = e.run(softcap=softcap)
    assert rx.device_check() == 0
    # (S of such a row is that of the low keys, whose raw scores need not be exact: their
    # weights are below 2^-50.  What counts is the others'.)
    G = e.hq // e.hkv
    for r, (p, s) in enumerate(e.reqs):
        pos = torch.arange(p, p + s, device="cuda")
        keep = torch.ones(p + s, dtype=torch.bool, device="cuda")
        keep[5::9] = False
        slot = e.up(e.table[e.rows[r], :p + s]).long()[keep]
        n = torch.cumsum(keep, 0)[pos] - 1  # the newest of the keys that count
        a = slice(int(e.qo[r]), int(e.qo[r + 1]))
        for h in range(e.hkv):
            hs = slice(h * G, (h + 1) * G)
            _check(out[a, hs], lse[a, hs],
                   _reference(e.q[a, hs], e.k[1, h, slot], e.v[1, h, slot], n, e.scale,
                              softcap=softcap), softcap)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [50.0, 2.0 ** 30])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_extend_rows_that_do_not_see_a_key_that_is_not_finite(softcap, bad):
    import torch
    e = Extend([(0, 150)], 4, 4, 128, seed=6)
    kb = [np.full(150, 40)]
    kb[0][:40] = np.arange(40)
    kb[0][39] = 0
    at = e.up(e.table[e.rows[0], 36:38]).long()
    e.k[:, :, at] = bad
    out, lse = e.run(key_begin=kb, softcap=softcap)
    assert rx.device_check() == 0
    _rows(e, out, lse, range(41, 150), softcap, zero=at.tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 2, 256), (16, 1, 128)])
@pytest.mark.parametrize("softcap", [50.0, 4096.0, 2.0 ** 30])
def test_decode_rows_beside_rows_at_the_cap(hq, hkv, d, softcap):
    """Some heads reach the cap, in tiles of shared segments and in streams."""
    import torch
    c = Decode([40 + 3 * i for i in range(37)], 700, hq, hkv, d, seed=1)
    c.q[:, 1::4] *= 4 * softcap
    heads = [h for h in range(hq) if h % 4 != 1]
    out, lse = c.run(softcap=softcap)
    assert rx.device_check() == 0
    G = hq // hkv
    for b in range(c.B):
        n = int(c.ctx[b])
        slot = c.up(c.table[b, :n]).long()
        for h in heads:
            _check(out[b:b + 1, h:h + 1], lse[b:b + 1, h:h + 1],
                   _reference(c.q[b:b + 1, h:h + 1], c.k[1, h // G, slot], c.v[1, h // G, slot],
                              torch.tensor([n - 1], device="cuda"), c.scale, softcap=softcap),
                   softcap)


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
