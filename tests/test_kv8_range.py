"""Attention over the 8-bit pool at the limits of what a pool may hold: K scales
of 2^-126 to 2^120, V scales far apart.
"""

import numpy as np
import pytest

from test_kv8 import Case, _decode, _extend


def _scaled(c, ks=None, vs=None):
    """Sets the K scales (one value) or the V scales (one value a block) of a
    case's pool."""
    torch = c.torch
    blocks = np.nonzero(c.index >= 0)[0] // c.block
    for which, new in ((0, ks), (1, vs)):
        if new is None:
            continue
        new = np.full(c.N // c.block, new, dtype=np.float64)
        sc = c.sc[1][..., which]
        old = sc.double().cpu().numpy()[:, blocks]
        sc.copy_(torch.where(torch.isnan(sc), sc, torch.from_numpy(new).float().cuda()))
        if which == 0:
            c.k = c.k / old[..., None] * new[blocks][None, :, None]
        else:
            c.v = c.v / old[..., None] * new[blocks][None, :, None]
            c.vs = np.broadcast_to(new[blocks], old.shape)


def _aimed(c, b, js, mag):
    """Queries that point at the keys js of request b: the signs of the key's
    codes.  Returns them with the rows of V that they select and their scores."""
    G = c.Hq // c.H
    idx = c.index[c.table[b, :c.ctx[b]]]
    q = np.zeros((len(js), c.Hq, c.d))
    want, score = np.zeros(q.shape), np.zeros(q.shape[:2])
    for h in range(c.Hq):
        k, v = c.k[h // G][idx], c.v[h // G][idx]
        for i, (j, lim) in enumerate(js):
            q[i, h] = np.where(k[j] < 0, -mag, mag)
            s = k[:lim] @ q[i, h] * c.scale
            others = np.delete(s, j)
            # nothing is left for the others, whatever the scores' rounding
            assert s[j] - (others.max() if lim > 1 else 0) > 60 + 2.0 ** -10 * s[j]
            want[i, h], score[i, h] = v[j], s[j]
    return q, want, score


SHAPES = [(32, 8, 128, 1, [300 + i for i in range(12)], 256),       # tiles and streams
          (16, 4, 256, 16, [700, 33, 16, 1], 0),                    # streams
          (64, 1, 128, 4, [513, 40], 0),                            # tiles
          (128, 1, 256, 1, [1700], 0)]                              # clusters of tiles
# K scale and query magnitude: the largest of each, and of both together
RANGES = [(2.0 ** 120, 2.0 ** -14), (2.0 ** 103, 2.0 ** 4), (2.0 ** 22, 2.0 ** 83),
          (1.0, 2.0 ** 16), (2.0 ** 20, 1.0)]


def _check(got_o, got_l, want, score, c, value=2.0 ** -23):
    go, gl = got_o.double().cpu().numpy(), got_l.double().cpu().numpy()
    # one weight of 1, exact; V to `value` of the largest V scale (times it and
    # its inverse in fp32)
    assert (np.abs(go - want) <= np.abs(want) * 2.0 ** -20 + c.vs.max() * value).all()
    # fp32 sums of d products, the row's scale, the logarithm's base
    assert (np.abs(gl - score) <= np.abs(score) * 2.0 ** -17 + 2.0 ** -20).all()


@pytest.mark.gpu
@pytest.mark.parametrize("ks,mag", RANGES)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_k_scales_up_to_the_limit(i, ks, mag):
    """Scores of 2^25 to 2^115: each query takes the row of V it points at."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 500 + i, shared=shared, pow2=True)
    _scaled(c, ks=ks)
    rng = np.random.default_rng(i)
    parts = [_aimed(c, b, [(int(rng.integers(x)), x)], mag) for b, x in enumerate(ctx)]
    q, want, score = (np.concatenate([p[k] for p in parts]) for k in range(3))
    o, lse = _decode(c, torch.from_numpy(q).to(torch.bfloat16).cuda(), bf16=False)
    _check(o, lse, want, score, c)
    sfx = [min(x, 5) for x in ctx]
    prefix = [x - s for x, s in zip(ctx, sfx)]
    parts = [_aimed(c, b, [(int(rng.integers(p + 1 + t)), p + 1 + t) for t in range(s)], mag)
             for b, (p, s) in enumerate(zip(prefix, sfx))]
    q, want, score = (np.concatenate([p[k] for p in parts]) for k in range(3))
    o, lse, _ = _extend(c, prefix, torch.from_numpy(q).to(torch.bfloat16).cuda(), False)
    _check(o, lse, want, score, c)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_the_smallest_k_scale(i):
    """Scales of 2^-126 and queries near their limit."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 600 + i, shared=shared, pow2=True)
    _scaled(c, ks=2.0 ** -126)
    q = c.queries(len(ctx), 2.0 ** 80)
    qn = q.double().cpu().numpy()
    o, lse = _decode(c, q, bf16=False)
    o2, lse2, _ = _extend(c, [x - 1 for x in ctx], q, False)
    for b in range(len(ctx)):
        ref = c.reference(qn[b:b + 1], b, [ctx[b]])
        c.compare(o[b:b + 1], lse[b:b + 1], ref, False)
        c.compare(o2[b:b + 1], lse2[b:b + 1], ref, False)


@pytest.mark.gpu
@pytest.mark.parametrize("exp", range(7, 16))
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_scores_whose_neighbours_are_whole_steps_apart(i, exp):
    """Scores of 2^22 to 2^31 (in powers of two of a weight), a few fp32 steps
    of theirs, 2^-2 to 2^7, apart: whatever the sums' rounding, the outputs are
    means of V, and lse is right to fp32."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 700 + i, shared=shared, pow2=True)
    used = torch.from_numpy(np.nonzero(c.index >= 0)[0]).cuda()
    codes = torch.full((H, len(used), d), 0x78, dtype=torch.uint8, device="cuda")     # 256
    codes[..., -1] = torch.randint(0, 8, codes.shape[:2], generator=c.gen, device="cuda",
                                   dtype=torch.uint8)       # 0 .. 7 times 2^-9
    c.kc[1][:, used] = codes
    _scaled(c, ks=1.0)
    c.scale = float(np.log(2.0))
    q = torch.full((len(ctx), Hq, d), 2.0 ** exp, device="cuda").to(torch.bfloat16)
    score = (d - 1) * 256.0 * 2.0 ** exp * c.scale
    for o, lse in (_decode(c, q, bf16=False), _extend(c, [x - 1 for x in ctx], q, False)[:2]):
        go, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.isfinite(go).all()
        assert (np.abs(gl - score) <= score * 2.0 ** -20 + 10).all()
        for b in range(len(ctx)):
            v = c.v[:, c.index[c.table[b, :ctx[b]]]]
            lo, hi = (np.repeat(f(v, axis=1), Hq // H, axis=0) for f in (np.min, np.max))
            room = 2.0 ** -10 * np.abs(v).max()
            assert (go[b] >= lo - room).all() and (go[b] <= hi + room).all()


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [10, 13, 20, 22])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_the_key_that_counts_has_a_small_v_scale(i, apart):
    """V scales 2^-10 to 2^-22 of the largest: exact to 2^-13, then off by at
    most 2^-23 of the largest scale."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 800 + i, shared=shared, pow2=True)
    rng = np.random.default_rng(i)
    js = [int(rng.integers(x)) for x in ctx]
    vs = np.full(c.N // block, 2.0 ** -5)
    vs[[c.table[b, j] // block for b, j in enumerate(js)]] *= 2.0 ** -apart
    _scaled(c, ks=2.0 ** -7, vs=vs)
    parts = [_aimed(c, b, [(js[b], x)], 32.0) for b, x in enumerate(ctx)]
    q, want, score = (np.concatenate([p[k] for p in parts]) for k in range(3))
    q = torch.from_numpy(q).to(torch.bfloat16).cuda()
    for o, lse in (_decode(c, q, bf16=False), _extend(c, [x - 1 for x in ctx], q, False)[:2]):
        _check(o, lse, want, score, c, 0.0 if apart <= 13 else 2.0 ** -23)
