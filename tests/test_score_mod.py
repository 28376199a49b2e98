"""Attention with modified scores (a tanh cap, distance slopes, a window,
documents, a part seen both ways) over the bf16 pool, against the formula in
64 bits.

Tolerances.  A raw score is a sum of d products held in fp32: off by at most
(d + 8) 2^-24 of S, the sum of the products' magnitudes times the scale.  The cap
adds 2^-21 of the softcap at most, the bias 2^-22 of itself, and moving to log2
units and to the row's maximum 2^-21 of the largest score: delta in all.  A
weight is then off by 2 delta of itself, and by 2^-8 from its rounding to bf16
(which the row sum does not share), so with A = sum_j p_j |v_j|
  |o - o64| <= (2^-8 + 4 delta + 2^-16) A  (+ 2^-8 |o| for bf16 outputs),
  |lse - lse64| <= 2 delta + 2^-20 (1 + |lse|),
2^-16 and 2^-20 for the sums and exponentials in fp32.
"""

import ctypes as C
import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx

INF = math.inf


# ------------------------------------------------------------------ refusals
def test_calls_refuse_before_any_cuda_call():
    X = 1 << 24
    pool = rx.rx_pool_desc(X, X, 64, 2, 2, 128, 0)
    info = rx.rx_decode_plan_info()
    info.n_work, info.n_parts, info.workspace_bytes = 1, 1, 4096

    def mod(**kw):
        m = rx.rx_score_mod(0.0, 0, None, None, None, X)
        for k, v in kw.items():
            setattr(m, k, v)
        return m

    def ext(pool=pool, layer=0, q=X, hq=4, table=X, rows=X, pre=X, qo=X, tiles=X, R=1, nt=1,
            m=mod(), out=X, ot=0, lse=X, scale=0.1):
        return rx._lib.rx_extend_attention_mod(C.byref(pool), layer, q, hq, table, 64, rows, pre,
                                               qo, tiles, R, nt, scale, C.byref(m), out, ot, lse,
                                               None)

    def dec(pool=pool, layer=0, q=X, hq=4, table=X, plan=X, info=info, B=1, step=0, m=mod(), out=X,
            ot=0, lse=X, ws=X, nb=4096, scale=0.1):
        return rx._lib.rx_decode_attention_mod(
            C.byref(pool), layer, q, hq, table, 64, plan, None if info is None else C.byref(info),
            B, step, scale, C.byref(m), out, ot, lse, ws, nb, None)
    assert ext(R=0) == rx.RX_OK and ext(nt=0) == rx.RX_OK and dec(B=0) == rx.RX_OK
    for fn in (ext, dec):
        for kw in (dict(layer=2), dict(layer=-1), dict(q=None), dict(q=X + 8), dict(hq=3),
                   dict(hq=0), dict(table=None), dict(out=None), dict(out=X + 8), dict(ot=2),
                   dict(ot=-1), dict(lse=None), dict(m=mod(softcap=-1.0)),
                   dict(m=mod(softcap=2.0 ** -41)), dict(m=mod(softcap=2.0 ** 41)),
                   dict(scale=2.0 ** -41), dict(scale=2.0 ** 41),
                   dict(m=mod(softcap=math.nan)), dict(m=mod(softcap=INF)),
                   dict(m=mod(window=-1)), dict(scale=0.0), dict(scale=-1.0),
                   dict(scale=math.nan), dict(scale=INF), dict(pool=rx.rx_pool_desc(X, X, 64, 2, 2, 96, 0))):
            assert fn(**kw) == rx.RX_ERR_INVALID, (fn, kw)
    for kw in (dict(rows=None), dict(pre=None), dict(qo=None), dict(tiles=None), dict(R=-1),
               dict(nt=-1), dict(nt=1 << 31)):
        assert ext(**kw) == rx.RX_ERR_INVALID, kw
    bad = rx.rx_decode_plan_info()
    bad.n_work, bad.n_work_tc = 1, 2
    for kw in (dict(plan=None), dict(info=None), dict(B=-1), dict(step=-1), dict(ws=None),
               dict(ws=X + 8), dict(nb=4095), dict(info=bad),
               dict(m=mod(window=3, d_ctx_len=None)), dict(m=mod(d_slopes=X, d_ctx_len=None))):
        assert dec(**kw) == rx.RX_ERR_INVALID, kw


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    for kw in (dict(slopes=torch.ones(4, dtype=torch.float64)),
               dict(key_begin=torch.zeros((2, 2), dtype=torch.int32)),
               dict(ctx_len=torch.zeros(8, dtype=torch.int32)[::2]),
               dict(bidir_end=torch.zeros(4, dtype=torch.int64))):
        with pytest.raises(ValueError):
            rx.score_mod(**kw)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rx.extend_attention_mod(None and 0 or rx.rx_pool_desc(1, 1, 8, 1, 1, 128, 0), 0, q, 4,
                                i.view(1, 4), i, i, i, i, 1, 1, 1.0, rx.score_mod(), q, q)


# --------------------------------------------------------------- window plans
def _tree(priv, shared, page=1, steps=0, seed=0, second=0):
    """A cache where every request shares `shared` tokens (and the requests of
    odd index `second` more), then has priv[b] of its own, `steps` of which
    were decoded outside the tree.  (cache, nodes, ctx, table)"""
    B = len(priv)
    need = shared + second + sum(priv) + 64 + (page + shared % page) * (B + 4)
    cache = rx.RadixCache(-(-need // page) * page, page)
    ctx = np.array([shared + (second if b % 2 else 0) + priv[b] for b in range(B)], np.int32)
    table = np.zeros((B, int(ctx.max()) + steps + 4), np.int32)
    slots = np.arange(page, cache.num_slots, dtype=np.int32)
    rng = np.random.default_rng(seed)
    if page == 1:
        rng.shuffle(slots)
    at, nodes = 0, []

    def take(n):
        nonlocal at
        out = slots[at:at + n]
        at += -(-n // page) * page
        return out
    cut = shared // page * page
    com, com2 = take(cut), take(second // page * page)
    for b in range(B):
        c2 = com2 if b % 2 else com2[:0]
        own = take(int(ctx[b]) - cut - len(c2))
        table[b, :ctx[b]] = np.concatenate([com, c2, own])
        keep = max(0, int(ctx[b]) - min(steps, priv[b]))
        ids = np.arange(keep, dtype=np.int32)
        ids[cut:cut + len(c2)] += 5000000
        ids[cut + len(c2):] += 100000 * (b + 1)
        nodes.append(cache.insert(ids, table[b, :keep])[1])
    return cache, nodes, ctx, table


def _covered(plan, info, B, step=0):
    """For each request the key positions its parts cover, from the plan."""
    out = [[] for _ in range(B)]
    parts = 0
    owner = {}
    for w in range(info.n_work):
        row, kb, ke, moff, nm, pb, nr, grow = plan[w * 8:w * 8 + 8]
        ke = min(ke, grow + step) if grow > 0 else ke
        assert pb == parts
        for i in range(nm):
            b = int(plan[info.off_members + moff + i])
            out[b].append((int(row), int(kb), max(int(kb), int(ke))))
            owner[pb + i] = b
        parts += nm
    assert parts == info.n_parts
    ip = plan[info.off_req_part_indptr:info.off_req_part_indptr + B + 1]
    rp = plan[info.off_req_parts:info.off_req_parts + parts]
    for b in range(B):
        got = rp[ip[b]:ip[b + 1]]
        assert len(got) == len(out[b]) and all(owner[int(p)] == b for p in got)
    return out


@pytest.mark.parametrize("window", [1, 7, 100, 500, 10 ** 6])
@pytest.mark.parametrize("n_steps", [1, 5])
def test_window_plan_covers_the_windows(window, n_steps):
    priv = [3, 40, 1, 300, 77, 9, 250, 1]
    cache, nodes, ctx, table = _tree(priv, shared=400, second=64)
    B = len(priv)
    plan, info = cache.plan_decode(nodes, ctx, np.arange(B), 8, 2, 128, n_steps=n_steps,
                                   window=window)
    full, finfo = cache.plan_decode(nodes, ctx, np.arange(B), 8, 2, 128, n_steps=n_steps)
    for step in range(n_steps):
        for b, ranges in enumerate(_covered(plan, info, B, step)):
            keys = []
            for row, kb, ke in ranges:
                # a segment's row holds the member's own slots there
                assert np.array_equal(table[row, kb:min(ke, ctx[b])],
                                      table[b, kb:min(ke, ctx[b])])
                keys += range(kb, ke)
            assert len(set(keys)) == len(keys)
            need = range(max(0, int(ctx[b]) + step - window), int(ctx[b]) + step)
            assert set(need) <= set(keys) and (not keys or max(keys) < ctx[b] + step)
    assert info.distinct_kv_tokens <= finfo.distinct_kv_tokens
    if window >= ctx.max() + n_steps:
        assert np.array_equal(plan[:info.plan_words], full[:finfo.plan_words])
    if window == 1:
        assert info.n_work <= B * n_steps and info.distinct_kv_tokens == B
    assert info.tails_private == finfo.tails_private


def test_window_plan_refuses():
    cache, nodes, ctx, _ = _tree([5], shared=8)
    with pytest.raises(rx.RxError):
        cache.plan_decode(nodes, ctx, np.arange(1), 4, 2, 128, window=-1)


# ------------------------------------------------------------------ on the GPU
def _bf(shape, g, mag=1.0):
    import torch
    return (mag * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def _reference(q, k, v, pos, scale, softcap=0.0, window=0, slopes=None, key_begin=None, bidir=0):
    """One KV head's queries [s, G, d] at positions pos over keys [n, d] in 64
    bits: (o, lse, A, delta)."""
    import torch
    q, k, v = q.double(), k.double(), v.double()
    d, n = q.shape[2], k.shape[0]
    x = torch.einsum("sgd,nd->sgn", q, k) * scale
    S = torch.einsum("sgd,nd->sgn", q.abs(), k.abs()) * abs(scale)
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    j = torch.arange(n, device=q.device)[None, :]
    p = pos[:, None]
    bias = torch.zeros((1, 1, 1), dtype=torch.float64, device=q.device)
    if slopes is not None:
        bias = slopes.double()[None, :, None] * (p - j).abs()[:, None, :]
        x = x - bias
    seen = (j <= p) | (j < bidir)
    if window:
        seen &= p - j < window
    if key_begin is not None:
        seen &= j >= key_begin[:, None]
    seen = seen[:, None, :].expand_as(x)
    x = torch.where(seen, x, torch.full_like(x, -INF))
    zero = torch.zeros_like(x)
    lse = torch.logsumexp(x, dim=2)
    some = torch.isfinite(lse)[..., None]
    w = torch.where(some, torch.exp(x - torch.where(some, lse[..., None], zero[..., :1])), zero)
    most = torch.where(seen, x, zero).abs().amax(dim=2)
    off = (d + 8) * 2.0 ** -24 * torch.where(seen, S, zero).amax(dim=2) + 2.0 ** -21 * softcap + \
        2.0 ** -22 * bias.abs().amax(dim=2) + 2.0 ** -21 * most
    return w @ v, lse, w @ v.abs(), off


def _check(o, lse, want):
    import torch
    wo, wl, A, off = want
    assert o.shape == wo.shape
    tol = (2.0 ** -8 + 4 * off + 2.0 ** -16)[..., None] * A
    if o.dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * wo.abs()
    assert ((o.double() - wo).abs() <= tol + 1e-30).all(), \
        float(((o.double() - wo).abs() / (tol + 1e-30)).max())
    dead = ~torch.isfinite(wl)
    assert (lse[dead] == -INF).all() and not o[dead].any()
    live = ~dead
    err = (lse.double() - wl)[live].abs()
    assert (err <= (2 * off + 2.0 ** -20 * (1 + wl.abs()))[live]).all(), float(err.max())


class Extend:
    """Requests of (prefix, suffix) tokens over shuffled runs of slots (pages:
    each request's runs start at a multiple of `page` of its positions)."""

    def __init__(self, reqs, hq, hkv, d, seed=0, mag=1.0, scale=None, runs=37, pad=3, page=0):
        import torch
        self.reqs, self.hq, self.hkv, self.d = reqs, hq, hkv, d
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        rng = np.random.default_rng(seed)
        n = [p + s for p, s in reqs]
        if page:
            room = [-(-x // page) * page for x in n]
            N = sum(room) + 2 * page
            pages = 1 + rng.permutation(sum(room) // page)
            order = (pages[:, None] * page + np.arange(page)).reshape(-1)
        else:
            room = n
            N = sum(n) + 8
            cuts = np.arange(1, N - 7, runs)
            order = np.concatenate([np.arange(c, min(c + runs, N - 7)) for c in
                                    rng.permutation(cuts)])
        self.N = N
        self.table = np.zeros((len(reqs) + 1, max(n) + 2), np.int32)
        self.rows = rng.permutation(len(reqs) + 1)[:len(reqs)].astype(np.int32)
        at = 0
        for r, x in enumerate(n):
            self.table[self.rows[r], :x] = order[at:at + x]
            at += room[r]
        self.qo = np.concatenate([[0], np.cumsum([s for _, s in reqs])]).astype(np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = _bf((2, hkv, N, d), g), _bf((2, hkv, N, d), g)
        self.total = int(self.qo[-1])
        self.q = _bf((self.total + pad, hq, d), g, mag)
        self.pad = pad

    def up(self, a):
        import torch
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def run(self, out_dtype=None, layer=1, key_begin=None, bidir=None, slopes=None, stream=None,
            **mod):
        """(out, lse) with the rows behind the last query filled with 7."""
        import torch
        tiles, nt = rx.extend_plan(self.qo, self.hq, self.hkv, self.d)
        # (an entry for every row of q, those behind the last query among them)
        self.mod = rx.score_mod(slopes=slopes, key_begin=None if key_begin is None else
                                self.up(np.concatenate(key_begin + [np.zeros(self.pad)])),
                                bidir_end=None if bidir is None else self.up(bidir), **mod)
        shape = (self.total + self.pad, self.hq)
        out = torch.full(shape + (self.d,), 7.0, dtype=out_dtype or torch.float32, device="cuda")
        lse = torch.full(shape, 7.0, device="cuda")
        self.args = (rx.pool_desc(self.k, self.v), layer, self.q, self.hq, self.up(self.table),
                     self.up(self.rows), self.up([p for p, _ in self.reqs]), self.up(self.qo),
                     self.up(tiles), len(self.reqs), nt, self.scale, self.mod, out, lse)
        rx.extend_attention_mod(*self.args, stream=stream)
        return out, lse

    def spoil(self, lo):
        """NaN in the pool's rows behind no table entry at position lo[r] and
        later."""
        import torch
        keep = torch.zeros(self.N, dtype=torch.bool, device="cuda")
        for r, (p, s) in enumerate(self.reqs):
            keep[self.up(self.table[self.rows[r], lo[r]:p + s]).long()] = True
        for t in (self.k, self.v):
            t[:, :, ~keep] = float("nan")

    def check(self, out, lse, layer=1, key_begin=None, bidir=None, slopes=None, window=0,
              softcap=0.0):
        import torch
        G = self.hq // self.hkv
        assert (out[self.total:] == 7).all() and (lse[self.total:] == 7).all()
        for r, (p, s) in enumerate(self.reqs):
            if s == 0:
                continue
            slot = self.up(self.table[self.rows[r], :p + s]).long()
            a = slice(int(self.qo[r]), int(self.qo[r + 1]))
            pos = torch.arange(p, p + s, device="cuda")
            for h in range(self.hkv):
                hs = slice(h * G, (h + 1) * G)
                k, v = (torch.nan_to_num(t[layer, h, slot].float()) for t in (self.k, self.v))
                _check(out[a, hs], lse[a, hs], _reference(
                    self.q[a, hs], k, v, pos, self.scale, softcap=softcap, window=window,
                    slopes=None if slopes is None else slopes[hs],
                    key_begin=None if key_begin is None else self.up(key_begin[r]).long(),
                    bidir=0 if bidir is None else min(int(bidir[r]), p + s)))


def _docs(rng, n, mean):
    """The first position of each position's document."""
    cut = np.concatenate([[0], np.cumsum(rng.integers(1, 2 * mean, n + 1))])
    return cut[np.searchsorted(cut, np.arange(n), side="right") - 1]


SHAPES = [
    # requests, hq, hkv, d
    ([(0, 1)], 4, 4, 128),
    ([(0, 1), (5, 3), (0, 0), (300, 1)], 8, 2, 256),
    ([(0, 130), (77, 45), (1000, 33)], 16, 2, 128),
    ([(513, 200), (0, 64), (2, 2)], 4, 1, 256),
    ([(900, 7), (0, 300)], 5, 1, 128),
    ([(0, 1100)], 3, 3, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{s[1]}/{s[2]}-{s[3]}")
@pytest.mark.parametrize("kind", ["none", "cap", "tight_cap", "slopes", "window1", "window",
                                  "docs", "bidir", "empty", "all"])
def test_extend_parity(shape, kind):
    import torch
    reqs, hq, hkv, d = shape
    e = Extend(reqs, hq, hkv, d, seed=len(kind) + d, mag=6.0 if kind in ("cap", "tight_cap")
               else 1.5)
    rng = np.random.default_rng(5)
    mod, kb, bidir, slopes = {}, None, None, None
    if kind in ("cap", "all"):
        mod["softcap"] = 50.0
    if kind == "tight_cap":
        mod["softcap"] = 2.0
    if kind in ("slopes", "all"):
        slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    if kind == "window1":
        mod["window"] = 1
    if kind in ("window", "all"):
        mod["window"] = 100
    if kind in ("docs", "all"):
        kb = [_docs(rng, p + s, 40)[p:] for p, s in reqs]
    if kind == "empty":  # some rows see nothing, whole tiles among them
        kb = [np.where(np.arange(s) % 3 == 1, p + np.arange(s) + 1, -5) for p, s in reqs]
        kb[-1] = np.full(reqs[-1][1], 2 ** 31 - 1)
    if kind in ("bidir", "all"):
        bidir = [(0, 60, 10 ** 9)[r % 3] for r in range(len(reqs))]
    for dt in (torch.float32, torch.bfloat16):
        out, lse = e.run(dt, key_begin=kb, bidir=bidir, slopes=slopes, **mod)
        assert rx.device_check() == 0
        e.check(out, lse, key_begin=kb, bidir=bidir, slopes=slopes, **mod)


@pytest.mark.gpu
def test_extend_without_modification_is_extend_attention():
    """mod NULL, and every field left out, against rx_extend_attention."""
    import torch
    e = Extend([(100, 150), (0, 20)], 8, 2, 128, seed=3)
    out, lse = e.run()
    a = list(e.args)
    plain, plse = torch.empty_like(out), torch.empty_like(lse)
    rx.extend_attention(*a[:12], plain, plse)
    again, alse = torch.empty_like(out), torch.empty_like(lse)
    rx.extend_attention_mod(*a[:12], None, again, alse)
    n = e.total
    assert torch.equal(again[:n], out[:n]) and torch.equal(alse[:n], lse[:n])
    # each is off by 2^-8 of sum p |v| for its weights' roundings, and the plain
    # call's row sums by 2^-8 again
    assert (plain[:n] - out[:n]).abs().max() <= 2.0 ** -6 * e.v.abs().max().item()
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [1, 8, 16, 32, 64, 128, 192])
def test_extend_over_pages(d, page):
    """Pages that groups and boxes of keys fall on, and that end inside them;
    windows that begin inside a page."""
    import torch
    e = Extend([(70, 130), (0, 333), (1000, 1), (47, 17)], 8, 2, d, seed=page, page=page)
    slopes = torch.exp2(-1.0 * torch.arange(1, 9, device="cuda"))
    for mod in (dict(), dict(window=77), dict(softcap=20.0), dict(window=201, softcap=20.0,
                                                                 slopes=slopes)):
        out, lse = e.run(torch.bfloat16, **mod)
        assert rx.device_check() == 0
        e.check(out, lse, **mod)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_outputs_that_start_on_16_bytes(dtype):
    """Outputs and workspaces need 16-byte alignment, not more."""
    import torch
    dt = getattr(torch, dtype)
    e = Extend([(90, 70), (0, 9)], 8, 2, 128, seed=12)
    want, _ = e.run(dt, softcap=20.0)
    room = torch.full((want.numel() + 64,), 7.0, dtype=dt, device="cuda")
    off = (16 - room.data_ptr() % 32) % 32 // room.element_size()
    out = room[off:off + want.numel()].view_as(want)
    assert out.data_ptr() % 32 == 16
    rx.extend_attention_mod(*e.args[:13], out, e.args[14])
    assert torch.equal(out, want)
    c = Decode([40 + 3 * i for i in range(37)], 300, 8, 2, 128, seed=1)
    want, _ = c.run(dt, softcap=20.0)
    ws = torch.zeros(c.args[12].numel() + 64, dtype=torch.uint8, device="cuda")
    ws = ws[(16 - ws.data_ptr() % 32) % 32:]
    out = room.new_full((want.numel() + 64,), 7.0)
    out = out[off:off + want.numel()].view_as(want)
    rx.decode_attention_mod(*c.args[:10], out, c.args[11], ws)
    assert torch.equal(out, want) and rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
def test_extend_reads_no_key_before_its_windows(d):
    e = Extend([(700, 90), (0, 400), (64, 1)], 8, 2, d, seed=9)
    w = 64
    e.spoil([max(0, p - w + 1) for p, s in e.reqs])
    out, lse = e.run(window=w)
    assert rx.device_check() == 0
    e.check(out, lse, window=w)


@pytest.mark.gpu
@pytest.mark.parametrize("mag,softcap,slope", [(1e-3, 1e-3, 0.0), (1e3, 30.0, 0.0),
                                               (1.0, 0.0, 1e4), (30.0, 1e5, -0.5),
                                               (1e4, 0.0, 0.0), (1.0, 2.0 ** 40, 0.0),
                                               (1.0, 2.0 ** -40, 0.0), (10.0, 1e4, 0.1)])
def test_extend_extreme_scores(mag, softcap, slope):
    import torch
    e = Extend([(50, 70), (0, 200)], 4, 2, 128, seed=4, mag=mag)
    slopes = torch.full((4,), slope, device="cuda") if slope else None
    out, lse = e.run(softcap=softcap, slopes=slopes)
    assert rx.device_check() == 0
    e.check(out, lse, softcap=softcap, slopes=slopes)


@pytest.mark.gpu
def test_extend_key_that_is_not_finite_under_a_mask():
    """An infinite or NaN key whose value is finite weighs nothing where it
    is masked."""
    e = Extend([(0, 150)], 4, 4, 128, seed=6)
    kb = [np.full(150, 40)]
    kb[0][:40] = np.arange(40)   # each of the first 40 sees itself alone
    kb[0][39] = 0                # ... and the keys before 40 all at once
    bad = e.up(e.table[e.rows[0], 20:22]).long()
    e.k[:, :, bad[0]] = float("inf")
    e.k[:, :, bad[1]] = float("nan")
    out, lse = e.run(key_begin=kb)
    rows = [i for i in range(150) if i not in (20, 21, 39)]
    e.k[:, :, bad] = 0
    want, wlse = e.run(key_begin=kb)
    import torch
    assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wlse[rows])
    assert rx.device_check() == 0


# --------------------------------------------------------------------- decode
class Decode:
    def __init__(self, priv, shared, hq, hkv, d, page=1, steps=0, second=0, seed=0, mag=1.5):
        import torch
        self.hq, self.hkv, self.d, self.B = hq, hkv, d, len(priv)
        self.cache, self.nodes, self.ctx, self.table = _tree(priv, shared, page, steps, seed,
                                                             second)
        N = self.cache.num_slots
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = _bf((2, hkv, N, d), g), _bf((2, hkv, N, d), g)
        self.q = _bf((self.B, hq, d), g, mag)
        self.scale = 1 / math.sqrt(d)
        self.pad = 2

    def up(self, a):
        import torch
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def run(self, out_dtype=None, layer=1, window=0, key_begin=None, slopes=None, softcap=0.0,
            plan_window=None, n_steps=None, step=0, stream=None):
        import torch
        plan, info = self.cache.plan_decode(self.nodes, self.ctx, np.arange(self.B), self.hq,
                                            self.hkv, self.d, n_steps=n_steps,
                                            window=window if plan_window is None else plan_window)
        self.info = info
        out = torch.full((self.B + self.pad, self.hq, self.d), 7.0,
                         dtype=out_dtype or torch.float32, device="cuda")
        lse = torch.full((self.B + self.pad, self.hq), 7.0, device="cuda")
        # (a workspace is not cleared by its owner)
        ws = torch.full((int(info.workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
        self.mod = rx.score_mod(softcap=softcap, window=window, slopes=slopes,
                                key_begin=None if key_begin is None else self.up(key_begin),
                                ctx_len=self.up(self.ctx))
        self.args = (rx.pool_desc(self.k, self.v), layer, self.q, self.hq, self.up(self.table),
                     self.up(plan[:info.plan_words]), info, self.B, self.scale, self.mod, out, lse,
                     ws)
        rx.decode_attention_mod(*self.args, step=step, stream=stream)
        return out, lse

    def check(self, out, lse, layer=1, window=0, key_begin=None, slopes=None, softcap=0.0,
              step=0):
        import torch
        G = self.hq // self.hkv
        assert (out[self.B:] == 7).all() and (lse[self.B:] == 7).all()
        for b in range(self.B):
            n = int(self.ctx[b]) + step
            slot = self.up(self.table[b, :n]).long()
            pos = torch.tensor([n - 1], device="cuda")
            for h in range(self.hkv):
                hs = slice(h * G, (h + 1) * G)
                _check(out[b:b + 1, hs], lse[b:b + 1, hs], _reference(
                    self.q[b:b + 1, hs], torch.nan_to_num(self.k[layer, h, slot].float()),
                    torch.nan_to_num(self.v[layer, h, slot].float()), pos, self.scale,
                    softcap=softcap, window=window, slopes=None if slopes is None else slopes[hs],
                    key_begin=None if key_begin is None else self.up(key_begin[b:b + 1]).long()))


DECODES = [
    # own tokens, shared, hq, hkv, d, page, second
    ([1], 0, 4, 4, 128, 1, 0),
    ([3201], 0, 32, 8, 128, 1, 0),
    ([5, 700, 33], 130, 8, 2, 256, 16, 0),
    ([3, 90, 1, 210, 17, 260, 64, 8, 2], 600, 16, 4, 128, 1, 77),
    ([40 + 3 * i for i in range(37)], 1111, 8, 2, 128, 1, 200),
    ([20 + 5 * i for i in range(24)], 500, 16, 2, 256, 64, 0),
    ([2 + i for i in range(70)], 300, 2, 2, 256, 1, 0),
    ([9, 30], 250, 40, 1, 128, 1, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{len(c[0])}x{c[2]}/{c[3]}-{c[4]}-{c[1]}")
@pytest.mark.parametrize("kind", ["none", "cap", "slopes", "window1", "window", "wide_plan",
                                  "docs", "empty", "all"])
def test_decode_parity(case, kind):
    import torch
    priv, shared, hq, hkv, d, page, second = case
    if kind == "cap":
        mag, cap = 6.0, 20.0
    else:
        mag, cap = 1.5, 50.0 if kind == "all" else 0.0
    c = Decode(priv, shared, hq, hkv, d, page, second=second, seed=len(kind), mag=mag)
    kw = dict(softcap=cap)
    if kind in ("slopes", "all"):
        kw["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    if kind in ("window", "all", "wide_plan"):
        kw["window"] = 150
    if kind == "window1":
        kw["window"] = 1
    if kind in ("docs", "all"):
        kw["key_begin"] = np.maximum(0, c.ctx - 1 - np.arange(c.B) * 61 % 400)
    if kind == "empty":
        kw["key_begin"] = np.where(np.arange(c.B) % 2 == 0, c.ctx, c.ctx // 2)
    for dt in (torch.float32, torch.bfloat16):
        out, lse = c.run(dt, plan_window=400 if kind == "wide_plan" else None, **kw)
        assert rx.device_check() == 0
        c.check(out, lse, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [DECODES[3], DECODES[4], DECODES[5]],
                         ids=lambda c: f"{len(c[0])}-{c[4]}")
def test_decode_steps_of_one_plan(case):
    """Steps of a multi-step plan: contexts, positions and windows move on."""
    import torch
    priv, shared, hq, hkv, d, page, second = case
    steps = 4
    c = Decode(priv, shared, hq, hkv, d, page, steps=min(steps, 2), second=second, seed=2)
    # the slots of the steps to come lie behind the context
    free = np.setdiff1d(np.arange(1, c.cache.num_slots), c.table[c.table > 0])[:steps]
    for b in range(c.B):
        c.table[b, c.ctx[b]:c.ctx[b] + steps] = free
    slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    kw = dict(window=90, softcap=30.0, slopes=slopes)
    for step in range(steps):
        out, lse = c.run(n_steps=steps, step=step, **kw)
        assert rx.device_check() == 0
        c.check(out, lse, step=step, **kw)


@pytest.mark.gpu
def test_decode_reads_no_key_before_its_windows():
    import torch
    w = 50
    for case in (DECODES[1], DECODES[3], DECODES[4]):
        priv, shared, hq, hkv, d, page, second = case
        c = Decode(priv, shared, hq, hkv, d, page, second=second, seed=8)
        keep = torch.zeros(c.cache.num_slots, dtype=torch.bool, device="cuda")
        for b in range(c.B):
            keep[c.up(c.table[b, max(0, c.ctx[b] - w):c.ctx[b]]).long()] = True
        for t in (c.k, c.v):
            t[:, :, ~keep] = float("nan")
        out, lse = c.run(window=w)
        assert rx.device_check() == 0
        c.check(out, lse, window=w)


@pytest.mark.gpu
def test_drafts_see_their_root_path_and_windows():
    """Drafts of two requests: positions and windows from the root path."""
    import torch
    hq, hkv, d, w = 8, 2, 128, 40
    pre = [100, 33]
    parents = [-1, 0, 0, 1, -1, 0, 1]
    indptr = np.array([0, 4, 7], np.int64)
    N = 256
    cache = rx.RadixCache(N)
    rows = np.zeros((2, 128), np.int32)
    nodes = []
    for r, n in enumerate(pre):
        rows[r, :n] = np.arange(1 + 120 * r, 1 + 120 * r + n)
        nodes.append(cache.insert(np.arange(n) + 1000 * r, rows[r, :n])[1])
    slots = np.arange(240, 247, dtype=np.int32)
    table, ctx, pos = rx.verify_rows(pre, rows, indptr, parents, slots, 128)
    c = Decode.__new__(Decode)
    c.hq, c.hkv, c.d, c.B, c.pad = hq, hkv, d, 7, 2
    c.cache, c.nodes, c.ctx, c.table = cache, [nodes[0]] * 4 + [nodes[1]] * 3, ctx, table
    g = torch.Generator(device="cuda").manual_seed(1)
    c.k, c.v, c.q = _bf((2, hkv, N, d), g), _bf((2, hkv, N, d), g), _bf((7, hq, d), g)
    c.scale = 0.1
    slopes = torch.linspace(0.01, 1, hq, device="cuda")
    kw = dict(window=w, slopes=slopes, softcap=10.0)
    out, lse = c.run(**kw)
    assert rx.device_check() == 0
    c.check(out, lse, **kw)


@pytest.mark.gpu
def test_captured_streams_and_two_at_once():
    """Calls captured and replayed with new inputs, and two of them at once on
    two streams with their own workspaces."""
    import torch
    c = Decode([40 + 3 * i for i in range(37)], 1111, 8, 2, 128, seed=1)
    e = Extend([(513, 200), (0, 64)], 4, 1, 256, seed=2)
    kw = dict(softcap=30.0, window=300)
    want = [t.clone() for t in c.run(**kw) + e.run(**kw)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    for t in c.args[10:12] + e.args[13:15]:
        t.fill_(7.0)
    with torch.cuda.graph(graph):
        rx.decode_attention_mod(*c.args)
        rx.extend_attention_mod(*e.args)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    got = list(c.args[10:12] + e.args[13:15])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    c.check(*c.args[10:12], **kw)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    d2 = Decode([40 + 3 * i for i in range(37)], 1111, 8, 2, 128, seed=1)
    torch.cuda.synchronize()
    a = c.run(stream=one, **kw)
    b = d2.run(stream=two, **kw)
    f = e.run(stream=two, **kw)
    torch.cuda.synchronize()
    c.check(*a, **kw)
    d2.check(*b, **kw)
    e.check(*f, **kw)
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("bad", [-1, -7, "num_slots", 2 ** 31 - 1])
def test_slots_outside_the_pool_are_flagged_and_read_as_slot_0(d, bad):
    """A table entry of -1 too, which is no mark for the end of a request."""
    import torch
    e = Extend([(70, 130), (0, 333)], 8, 2, d, seed=21)
    c = Decode([40 + 3 * i for i in range(37)], 300, 8, 2, d, seed=1)
    for x, rows in ((e, e.rows), (c, range(c.B))):
        x.table = x.table.copy()
        at = [(r, p) for r in rows for p in (0, 17, 39, 40)]
        slots = {}
        for slopes in (None, torch.full((8,), 0.01, device="cuda")):
            for value in (0, x.k.shape[2] if bad == "num_slots" else bad):
                for r, p in at:
                    x.table[r, p] = value
                got = x.run(softcap=30.0, slopes=slopes)
                if value:
                    with pytest.raises(rx.RxError, match="flags 2"):
                        rx.device_check()
                slots[value == 0] = got
                assert rx.device_check() == 0
            assert all(torch.equal(a, b) for a, b in zip(slots[True], slots[False]))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("shape", ["climb", "fall", "swing", "spikes", "low"])
def test_scores_that_move_by_hundreds_from_tile_to_tile(d, shape):
    """Every row's largest score so far is overtaken (or left far behind) again and
    again, within tiles of 64 keys and from one to the next, in some rows only."""
    import torch
    e = Extend([(900, 70), (0, 400)], 8, 2, d, seed=31, mag=0.2)
    g = torch.Generator(device="cuda").manual_seed(7)
    n = torch.arange(970, device="cuda").float()
    amp = {"climb": n * 0.9 - 400, "fall": 400 - n * 0.9,
           "swing": 300 * torch.sign(torch.sin(n * (math.pi / 64))),
           "spikes": torch.where(n % 97 == 11, n * 0.5, torch.zeros_like(n)) - 90,
           "low": -600 + torch.randn(970, generator=g, device="cuda")}[shape]
    # one direction of unit length carries the amplitudes; half of the rows look along
    # it, one in four the other way, the rest hardly at all
    u = torch.zeros(d, device="cuda")
    u[:16] = 0.25
    look = torch.tensor([1.0, 1.0, -1.0, 0.01], device="cuda").repeat(e.q.shape[0], 2)
    q = e.q.float()
    q[..., :16] = look[..., None] * 0.25 / e.scale
    e.q = q.to(torch.bfloat16)
    for r, (p, s) in enumerate(e.reqs):
        slot = e.up(e.table[e.rows[r], :p + s]).long()
        k = e.k[:, :, slot].float() * 0.1
        k[..., :16] = (u[:16] * amp[:p + s, None])
        e.k[:, :, slot] = k.to(torch.bfloat16)
    slopes = torch.full((8,), 0.03, device="cuda")
    for mod in (dict(), dict(window=300), dict(slopes=slopes), dict(softcap=500.0),
                dict(softcap=200.0, slopes=slopes)):
        out, lse = e.run(**mod)
        assert rx.device_check() == 0
        e.check(out, lse, **mod)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1.0, 44.0, 52.6, 52.8, 90.0])
@pytest.mark.parametrize("d", [128, 256])
def test_caps_that_scores_reach(d, softcap):
    """Scores at both ends of the cap, in extend and in decode's tiles and streams, at caps
    around 76 ln 2, up to which every row's weights stand under one reference."""
    import torch
    e = Extend([(300, 70), (0, 200)], 8, 2, d, seed=5, mag=2.0 * softcap)
    for sign in (1, -1):
        # (the first request's rows see nothing but one end)
        e.k[:, :, :, 0] = sign * e.k[:, :, :, 0].abs().clamp(min=0.5)
        e.q[:70, :, 0] = 8 * softcap
        for kw in (dict(softcap=softcap), dict(softcap=softcap, window=90)):
            out, lse = e.run(**kw)
            assert rx.device_check() == 0
            e.check(out, lse, **kw)
    c = Decode([40 + 3 * i for i in range(37)], 700, 8, 2, d, seed=1, mag=2.0 * softcap)
    out, lse = c.run(softcap=softcap)
    assert rx.device_check() == 0
    c.check(out, lse, softcap=softcap)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["none", "cap", "high_cap", "slopes"])
def test_a_row_of_one_key_is_its_value(d, kind):
    """Windows of one key, documents of one token, and a prompt's first token: the weight
    is 1 and rounds to nothing, whatever the score."""
    import torch
    e = Extend([(300, 70), (0, 200), (64, 130)], 8, 2, d, seed=6, mag=3.0)
    kw = {"none": dict(), "cap": dict(softcap=30.0), "high_cap": dict(softcap=60.0),
          "slopes": dict(slopes=torch.full((8,), 0.3, device="cuda"))}[kind]
    value = torch.cat([e.v[1][:, e.up(e.table[e.rows[r], p:p + s]).long()]
                       for r, (p, s) in enumerate(e.reqs)], 1).repeat_interleave(4, 0)
    value = value.transpose(0, 1).float()
    alone = [np.arange(p, p + s) // 3 * 3 for p, s in e.reqs]  # every third token
    for mod in (dict(window=1), dict(key_begin=alone)):
        out, _ = e.run(**mod, **kw)
        assert rx.device_check() == 0
        rows = torch.ones(e.total, dtype=torch.bool, device="cuda") if "window" in mod else \
            torch.from_numpy(np.concatenate([np.arange(p, p + s) % 3 == 0
                                             for p, s in e.reqs])).cuda()
        assert torch.equal(out[:e.total][rows], value[rows])
    out, _ = e.run(**kw)
    assert torch.equal(out[70], value[70])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["none", "cap", "high_cap", "slopes", "window", "docs", "both_ways",
                                  "empty", "all"])
def test_few_row_tiles_over_long_contexts(d, kind):
    """Calls whose row tiles share their keys among CTAs: contexts of shares of 512 keys and
    of less than one, rows that see keys of one share only, or none."""
    import torch
    reqs = [(9000, 5), (4000, 40), (30, 3), (0, 1), (1500, 33)]
    e = Extend(reqs, 8, 2, d, seed=len(kind), mag=2.0)
    rng = np.random.default_rng(3)
    kw = {"none": dict(), "cap": dict(softcap=20.0), "high_cap": dict(softcap=60.0),
          "slopes": dict(slopes=torch.exp2(-1.0 * torch.arange(1, 9, device="cuda"))),
          "window": dict(window=3001), "docs": dict(), "both_ways": dict(bidir=[9003, 10, 33, 0, 9]),
          "empty": dict(), "all": dict(softcap=30.0, window=2500)}[kind]
    if kind in ("docs", "all"):
        kw["key_begin"] = [_docs(rng, p + s, 700)[p:] for p, s in reqs]
    if kind == "empty":
        kw["key_begin"] = [np.where(np.arange(s) % 2, p + s + 5, p // 2) for p, s in reqs]
    if kind == "all":
        kw["slopes"] = torch.full((8,), 0.01, device="cuda")
        kw["bidir"] = [100, 4040, 5, 1, 1533]
    for dt in (torch.float32, torch.bfloat16):
        out, lse = e.run(dt, **kw)
        assert rx.device_check() == 0
        e.check(out, lse, **kw)
        again, _ = e.run(dt, **kw)
        assert torch.equal(out, again)
