"""Rows in which one key weighs nearly all, in attention with modified scores:
the rounding of its weight to bf16 must not be the output's.

Tolerance.  The product with V takes the weights w'_j = w_j (1 + e_j), |e_j| <= 2^-8, and
the output is divided by a sum of weights of which the heaviest at least counts as it was
rounded, so that with p_j = w_j / sum w its error of o is p_m e_m (v_m - o), and another
key's p_j e_j (v_j - o) or p_j e_j v_j.  With 1 - p_m = r and |v_j| <= V both p_m |v_m - o|
and the sum of p_j |v_j - o| over the others are at most 2 r V, in all at most 2^-8 (1 +
2^-7) 4 r V.  An error delta of a score (as in test_score_mod.py) is an e_j of 2 delta.  The
sums in fp32 and the division add 2^-16 A, A = sum_j p_j |v_j|; a bf16 output its own 2^-8
|o|.  The logarithm of the sum is that of the weights before their rounding:
2 delta + 2^-20 (1 + |lse|).  Extend's rows of 16 keys and fewer are divided by the sum before
the rounding, and err by 2^-8 A.
"""

import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import Decode, Extend, _docs

INF = math.inf


def _check(o, lse, q, k, v, pos, scale, softcap=0.0, window=0, slopes=None, key_begin=None,
           few=0):
    """One KV head's outputs [s, G, d] of queries at positions pos over keys [n, d]."""
    import torch
    q, k, v = q.double(), k.double(), v.double()
    d, n = q.shape[2], k.shape[0]
    x = torch.einsum("sgd,nd->sgn", q, k) * scale
    S = torch.einsum("sgd,nd->sgn", q.abs(), k.abs()) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    j, p = torch.arange(n, device=q.device)[None, :], pos[:, None]
    bias = torch.zeros((1, 1, 1), dtype=torch.float64, device=q.device)
    if slopes is not None:
        bias = slopes.double()[None, :, None] * (p - j).abs()[:, None, :]
        x = x - bias
    seen = j <= p
    if window:
        seen &= p - j < window
    if key_begin is not None:
        seen &= j >= key_begin[:, None]
    seen = seen[:, None, :].expand_as(x)
    x = torch.where(seen, x, torch.full_like(x, -INF))
    zero = torch.zeros_like(x)
    want = torch.logsumexp(x, dim=2)
    w = torch.exp(x - want[..., None])
    wo, A = w @ v, w @ v.abs()
    V = torch.where(seen[..., None].any(1).any(0), v.abs(), torch.zeros_like(v)).amax(0)
    r = 1 - w.amax(dim=2)
    delta = (d + 8) * 2.0 ** -24 * torch.where(seen, S, zero).amax(dim=2) + \
        2.0 ** -21 * softcap + 2.0 ** -22 * bias.abs().amax(dim=2) + \
        2.0 ** -21 * torch.where(seen, x, zero).abs().amax(dim=2)
    e = 2.0 ** -8 * (1 + 2.0 ** -7) + 2 * delta
    tol = (4 * e * r)[..., None] * V + 2.0 ** -16 * A + 1e-30
    tol = torch.where((seen.sum(dim=2) <= few)[..., None], (2.0 ** -8 + 2 * delta[..., None]) * A +
                      2.0 ** -16 * A + 1e-30, tol)
    if o.dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * wo.abs()
    err = (o.double() - wo).abs()
    assert (err <= tol).all(), float((err / tol).max())
    lerr = (lse.double() - want).abs()
    assert (lerr <= 2 * delta + 2.0 ** -20 * (1 + want.abs())).all(), float(lerr.max())


def _peak(q, k, scale, at, amp):
    """Gives the keys at slots `at` scores of about amp, and every other key none of the
    direction that they lie in; rows look along it more or less."""
    import torch
    look = 1 + 0.01 * (torch.arange(q[..., 0].numel(), device="cuda") % 17)
    q[..., :16] = (0.25 / scale * look.view(q.shape[:-1]))[..., None].to(q.dtype)
    k[..., :16] = 0
    k[:, :, at, :16] = 0.25 * amp


KINDS = {"none": dict(), "cap": dict(softcap=50.0), "high_cap": dict(softcap=90.0),
         "slopes": dict(slope=2e-4), "window": dict(window=901), "short": dict(window=41),
         "all": dict(softcap=60.0, window=1500, slope=1e-3)}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["plain"] + list(KINDS) + ["docs"])
@pytest.mark.parametrize("many", [False, True], ids=["few_tiles", "many_tiles"])
def test_extend_rows_of_one_heavy_key(d, kind, many):
    """(short: rows of 41 keys, most of them over two tiles; few_tiles: the keys of a row
    tile are shared among CTAs; plain: rx_extend_attention, which the bound holds for too)"""
    import torch
    reqs = [(2300, 40), (2100, 33)] if not many else [(0, 700), (700, 300), (100, 200), (90, 77)] * 2
    hq, hkv = (8, 2) if not many else (16, 4)
    e = Extend(reqs, hq, hkv, d, seed=len(kind))
    lengths = [p + s for p, s in reqs]
    for amp, every in ((13.0, 600), (9.0, 30)):
        at = torch.cat([e.up(e.table[e.rows[r], :n][(np.arange(n) - 11 * r) % every == 17])
                        for r, n in enumerate(lengths)]).long()
        _peak(e.q, e.k, e.scale, at, amp)
        kw = dict(KINDS.get(kind, {}))
        slope = kw.pop("slope", 0.0)
        slopes = torch.full((hq,), slope, device="cuda") if slope else None
        kb = None
        if kind == "docs":
            rng = np.random.default_rng(2)
            kb = [_docs(rng, p + s, 400)[p:] for p, s in reqs]
        for dt in (torch.float32, torch.bfloat16):
            out, lse = e.run(dt, key_begin=kb, slopes=slopes, **kw)
            if kind == "plain":
                if dt is torch.bfloat16:
                    continue
                rx.extend_attention(*e.args[:12], out, lse)
            assert rx.device_check() == 0
            for r, (p, s) in enumerate(reqs):
                slot = e.up(e.table[e.rows[r], :p + s]).long()
                a = slice(int(e.qo[r]), int(e.qo[r + 1]))
                for h in range(hkv):
                    hs = slice(h * hq // hkv, (h + 1) * hq // hkv)
                    got = lse[a, hs]
                    args = (e.q[a, hs], e.k[1, h, slot], e.v[1, h, slot],
                            torch.arange(p, p + s, device="cuda"), e.scale)
                    more = dict(kw, slopes=None if slopes is None else slopes[hs],
                                key_begin=None if kb is None else e.up(kb[r]).long())
                    if kind == "plain":  # (its lse is the rounded weights')
                        q, k = (t.double() for t in args[:2])
                        x = torch.einsum("sgd,nd->sgn", q, k) * e.scale
                        far = torch.arange(p + s, device="cuda")[None] > args[3][:, None]
                        got = torch.logsumexp(x.masked_fill(far[:, None], -INF), 2).float()
                    _check(out[a, hs], got, *args, few=0 if kind == "plain" else 16, **more)


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


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 2, 256), (40, 1, 128), (16, 2, 128)])
@pytest.mark.parametrize("kind", list(KINDS))
def test_decode_rows_of_one_heavy_key(hq, hkv, d, kind):
    """Heavy keys in a shared segment (tiles) and in private tails (streams of one or two
    row groups)."""
    import torch
    c = Decode([300 + 7 * i for i in range(21)] + [1, 2], 900, hq, hkv, d, seed=len(kind))
    for amp, every in ((13.0, 500), (9.0, 30)):
        at = torch.cat([c.up(c.table[b, :n][(np.arange(n) - (n > 900) * b) % every == 17])
                        for b, n in enumerate(c.ctx)]).long()
        _peak(c.q, c.k, c.scale, at, amp)
        kw = dict(KINDS[kind])
        slope = kw.pop("slope", 0.0)
        slopes = torch.full((hq,), slope, device="cuda") if slope else None
        for dt in (torch.float32, torch.bfloat16):
            out, lse = c.run(dt, slopes=slopes, **kw)
            assert rx.device_check() == 0
            for b in range(c.B):
                n = int(c.ctx[b])
                slot = c.up(c.table[b, :n]).long()
                for h in range(hkv):
                    hs = slice(h * hq // hkv, (h + 1) * hq // hkv)
                    _check(out[b:b + 1, hs], lse[b:b + 1, hs], c.q[b:b + 1, hs], c.k[1, h, slot],
                           c.v[1, h, slot], torch.tensor([n - 1], device="cuda"), c.scale,
                           slopes=None if slopes is None else slopes[hs], **kw)
