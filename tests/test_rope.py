"""Norm and position rotation of queries and keys, and their append to the
pool, against the formulas in 64 bits.

Tolerances: a result y has one rounding to bf16 (2^-8 of |y|) over fp32
arithmetic on the pair (a, b) that it comes from.  Sine and cosine are off by
2^-20.5 from the special-function unit, by 2^-22 from the angle's fp32 value
and by 2^-21 from the fraction of a turn at position 2^31; the norm's factor by
some 2^-21 of itself, products and the sum by 2^-23: together below 2^-18 of
(|a| + |b|) times the magnitude.  2^-17 of it is allowed.
"""

import ctypes as C
import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx

TWO_PI = 2 * math.pi


def freqs(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, low=0, high=0, **_):
    """Radians a position of each pair, and the magnitude, in 64 bits."""
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":
        c = [rot * math.log(original_len / (n * TWO_PI)) / (2 * math.log(base))
             for n in (high, low)]
        a, b = max(0, math.floor(c[0])), min(rot - 1, math.ceil(c[1]))
        w = np.clip((np.arange(rot // 2) - a) / max(b - a, 0.001), 0, 1)
        return f / factor * w + f * (1 - w), 0.1 * math.log(factor) + 1
    if scaling == "wavelength":
        w = 1 - np.clip((original_len * f / TWO_PI - low) / (high - low), 0, 1)
        return f / factor * w + f * (1 - w), 1.0
    return f, 1.0


SCALED = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
          dict(scaling="parts", factor=8.0, original_len=4096, low=1.0, high=32.0),
          dict(scaling="wavelength", factor=8.0, original_len=8192, low=1.0, high=4.0,
               base=500000.0)]


@pytest.mark.parametrize("kw", SCALED)
@pytest.mark.parametrize("rot", [2, 34, 128, 256])
def test_rope_init_is_the_formula(kw, rot):
    r = rx.rope(rot, **kw)
    f, m = freqs(rot, **kw)
    got = np.array([t / 2.0 ** 64 for t in r.turns])
    # pow and its few products: some 2^-51 of the value; the fraction 2^-65
    assert np.all(np.abs(got[:rot // 2] - f / TWO_PI) <= 2.0 ** -50 * f + 2.0 ** -64)
    assert not got[rot // 2:].any()
    assert (r.rot_dim, r.layout, r.reserved) == (rot, 0, 0)
    assert abs(r.magnitude - m) <= 2 ** -23
    assert rx.rope(rot, magnitude=0.5, layout="interleaved", **kw).magnitude == 0.5


def test_rope_init_refuses():
    ok = dict(base=10000.0, factor=2.0, original_len=4096.0, low=1.0, high=4.0, magnitude=0.0,
              rot_dim=64, layout=0, scaling=3, reserved=0)
    out = rx.rx_rope()

    def call(**kw):
        d = dict(ok, **kw)
        cfg = rx.rx_rope_config(*[d[n] for n, _ in rx.rx_rope_config._fields_])
        return rx._lib.rx_rope_init(C.byref(cfg), C.byref(out))
    assert call() == rx.RX_OK
    assert call(rot_dim=0) == rx.RX_OK
    for kw in (dict(base=1.0), dict(base=-3.0), dict(base=math.inf), dict(base=math.nan),
               dict(factor=0.5), dict(factor=math.nan), dict(factor=math.inf),
               dict(original_len=0.0), dict(low=0.0), dict(high=1.0), dict(high=math.nan),
               dict(magnitude=-1.0), dict(magnitude=math.nan), dict(rot_dim=-2), dict(rot_dim=63),
               dict(rot_dim=258), dict(layout=2), dict(scaling=5), dict(scaling=-1),
               dict(reserved=1)):
        assert call(**kw) == rx.RX_ERR_INVALID, kw
    assert call(scaling=0, factor=0.0, original_len=0.0, low=0.0) == rx.RX_OK
    assert rx._lib.rx_rope_init(None, C.byref(out)) == rx.RX_ERR_INVALID
    cfg = rx.rx_rope_config(10000.0, 1.0, 0, 0, 0, 0, 64, 0, 0, 0)
    assert rx._lib.rx_rope_init(C.byref(cfg), None) == rx.RX_ERR_INVALID


def test_calls_refuse_before_any_cuda_call():
    X, T, r = 1 << 24, 3, rx.rope(128)
    pool = rx.rx_pool_desc(X, X, 64, 2, 2, 128, 0)

    def rot(rope=r, norm=None, d=128, pos=X, T=T, q=X, qs=512, hq=4, k=X, ks=256, hkv=2, qo=X,
            qos=512, ko=X, kos=256):
        return rx._lib.rx_qk_rope(None if rope is None else C.byref(rope),
                                  None if norm is None else C.byref(norm), d, pos, T, q, qs, hq,
                                  k, ks, hkv, qo, qos, ko, kos, None)

    def sto(pool=pool, layer=0, rope=r, norm=None, pos=X, slots=X, T=T, q=X, qs=512, hq=4, k=X,
            ks=256, v=X, vs=256, qo=X, qos=512):
        return rx._lib.rx_qkv_store(C.byref(pool), layer, None if rope is None else C.byref(rope),
                                    None if norm is None else C.byref(norm), pos, slots, T, q, qs,
                                    hq, k, ks, v, vs, qo, qos, None)
    wide = rx.rope(256)
    odd = rx.rx_rope()
    odd.rot_dim, odd.magnitude = 3, 1.0
    lay = rx.rope(64)
    lay.layout = 7
    nan = rx.rope(64)
    nan.magnitude = math.nan
    for fn in (rot, sto):
        assert fn(T=0) == rx.RX_OK
        for kw in (dict(T=-1), dict(T=1 << 31), dict(pos=None), dict(q=None), dict(q=X + 8),
                   dict(qo=None), dict(qo=X + 2), dict(qs=504), dict(qs=516), dict(qos=8),
                   dict(k=None), dict(k=X + 4), dict(ks=255), dict(ks=260), dict(hq=-1),
                   dict(rope=wide), dict(rope=odd), dict(rope=lay), dict(rope=nan),
                   dict(norm=rx.rx_head_norm(None, None, -1.0, 0)),
                   dict(norm=rx.rx_head_norm(None, None, math.nan, 0)),
                   dict(norm=rx.rx_head_norm(X + 2, None, 1e-6, 0))):
            assert fn(**kw) == rx.RX_ERR_INVALID, (fn, kw)
    for kw in (dict(d=64), dict(hkv=-1), dict(ko=None), dict(ko=X + 8), dict(kos=248),
               dict(kos=257)):
        assert rot(**kw) == rx.RX_ERR_INVALID, kw
    for kw in (dict(layer=2), dict(slots=None), dict(v=None), dict(v=X + 8), dict(vs=128),
               dict(vs=257), dict(pool=rx.rx_pool_desc(X, X, 64, 2, 2, 64, 0))):
        assert sto(**kw) == rx.RX_ERR_INVALID, kw
    assert rot(hq=0, hkv=0, q=None, k=None) == rx.RX_OK


def test_binding_refuses_cpu_and_wrong_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rx.qk_rope(rx.rope(128), pos, q, q, q, q)
    with pytest.raises(ValueError):
        rx.head_norm(torch.ones(128), None, 1e-6)
    with pytest.raises(KeyError):
        rx.rope(128, layout="pairs")


# ------------------------------------------------------------------ on the GPU
def reference(x, pos, d, rot, layout, kw, norm, w, eps):
    """fp64 rows [T, H, d] and the tolerance of each element."""
    y = x.astype(np.float64)
    if norm and w is not None:
        y = y / np.sqrt((y * y).mean(axis=2, keepdims=True) + eps)
        y = y * (w.astype(np.float64) + (1 if norm == "plus_one" else 0))
    z, size = y.copy(), np.abs(y)
    m = 1.0
    if rot:
        f, m = freqs(rot, **kw)
        t = np.asarray(pos, dtype=np.float64)[:, None] * f[None, :]
        c, s = np.cos(t)[:, None, :] * m, np.sin(t)[:, None, :] * m
        ia = np.arange(rot // 2) if layout == "half" else 2 * np.arange(rot // 2)
        ib = ia + (rot // 2 if layout == "half" else 1)
        a, b = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia] = size[..., ib] = m * (np.abs(a) + np.abs(b))
    return z, 2.0 ** -8 * np.abs(z) + 2.0 ** -17 * size + 1e-30


class Rows:
    """bf16 queries, keys and values of T tokens, apart or side by side."""

    def __init__(self, T, hq, hkv, d, fused, seed, spread=0.0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = hq + 2 * hkv
        x = torch.randn((T, n + (3 if fused else 0), d), generator=g, device="cuda")
        if spread:
            x = x * torch.exp(spread * torch.randn((T, x.shape[1], 1), generator=g, device="cuda"))
        x = x.to(torch.bfloat16)
        cut = (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:n])
        self.all = x
        self.q, self.k, self.v = cut if fused else tuple(c.contiguous() for c in cut)
        self.w = tuple((torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
                       for _ in range(2))


def _np(t):
    return t.detach().float().cpu().numpy()


def _norm(kind, w, eps=1e-6):
    if not kind:
        return None
    return rx.head_norm(w[0], None if kind == "q_only" else w[1], eps,
                        plus_one=kind == "plus_one")


CASES = [
    # T, hq, hkv, d, rot, layout, scaling, norm, fused
    (1, 32, 8, 128, 128, "half", 0, "weight", False),
    (1, 1, 1, 128, 128, "interleaved", 0, "", False),
    (3, 5, 1, 128, 64, "half", 1, "plus_one", True),
    (33, 8, 2, 256, 256, "half", 2, "weight", True),
    (33, 3, 3, 256, 64, "interleaved", 3, "q_only", False),
    (700, 7, 1, 128, 34, "half", 4, "weight", True),
    (700, 2, 2, 128, 2, "half", 0, "plus_one", False),
    (129, 16, 4, 256, 250, "half", 3, "", True),
    (129, 16, 4, 256, 250, "interleaved", 3, "weight", True),
    (64, 8, 2, 128, 32, "half", 0, "", False),
    (64, 8, 2, 128, 0, "half", 0, "weight", True),
    (5000, 4, 1, 128, 128, "half", 0, "weight", False),
    (20011, 3, 1, 256, 128, "interleaved", 4, "plus_one", True),
]


def _positions(T, seed):
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 1 << 20, T)
    ends = [0, (1 << 31) - 1, -(1 << 31), -1, 1 << 30, 1][:T]
    pos[:len(ends)] = ends
    return pos.astype(np.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("in_place", [False, True])
def test_qk_rope_parity(case, in_place):
    import torch
    T, hq, hkv, d, rot, layout, sc, norm, fused = case
    r = Rows(T, hq, hkv, d, fused, seed=T + d, spread=1.0)
    before = r.all.clone()
    q0, k0 = _np(r.q), _np(r.k)
    pos = _positions(T, 7)
    dpos = torch.from_numpy(pos).cuda()
    qo, ko = (r.q, r.k) if in_place else (torch.empty_like(r.q.contiguous()),
                                          torch.empty_like(r.k.contiguous()))
    rope = rx.rope(rot, layout=layout, **SCALED[sc]) if rot else None
    rx.qk_rope(rope, dpos, r.q, r.k, qo, ko, _norm(norm, r.w))
    assert rx.device_check() == 0
    for x, got, w in ((q0, qo, r.w[0]), (k0, ko, None if norm == "q_only" else r.w[1])):
        want, tol = reference(x, pos, d, rot, layout, SCALED[sc], norm, _np(w) if w is not None
                              else None, 1e-6)
        assert np.all(np.abs(_np(got) - want) <= tol)
    if in_place and fused:  # what lies beside the queries and keys
        assert torch.equal(r.all[:, hq + hkv:], before[:, hq + hkv:])


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_qkv_store_equals_rotation_and_store(case):
    """The pool and the queries bit for bit as rx_qk_rope then rx_kv_store
    leave them, and the pool's other rows as they were."""
    import torch
    T, hq, hkv, d, rot, layout, sc, norm, fused = case
    r = Rows(T, hq, hkv, d, fused, seed=T + 1)
    L, N = 2, T + 9
    g = torch.Generator(device="cuda").manual_seed(3)
    pools = [torch.randn((L, hkv, N, d), generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2)]
    mine = [p.clone() for p in pools]
    slots = torch.randperm(N - 1, generator=g, device="cuda")[:T].to(torch.int32) + 1
    dpos = torch.from_numpy(_positions(T, 8)).cuda()
    rope = rx.rope(rot, layout=layout, **SCALED[sc]) if rot else None
    hn = _norm(norm, r.w)
    qo = [torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ko = torch.empty((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    rx.qk_rope(rope, dpos, r.q, r.k, qo[0], ko, hn)
    rx.kv_store(rx.pool_desc(*pools), 1, slots, ko, r.v.contiguous())
    rx.qkv_store(rx.pool_desc(*mine), 1, rope, dpos, slots, r.q, r.k, r.v, qo[1], hn)
    assert rx.device_check() == 0
    assert torch.equal(qo[0], qo[1])
    assert torch.equal(pools[0], mine[0]) and torch.equal(pools[1], mine[1])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_store_with_queries_in_place(layout):
    """Queries turned where they lie in the projection's rows, whose tokens are
    no multiple of 32 bytes apart."""
    import torch
    T, hq, hkv, d = 50, 4, 2, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    room = torch.randn((T, (hq + 2 * hkv) * d + 8), generator=g, device="cuda").to(torch.bfloat16)
    x = room[:, 8:].unflatten(1, (hq + 2 * hkv, d))
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    before = room.clone()
    pool = [torch.zeros((1, hkv, T + 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want, tol = reference(_np(q), pos.cpu().numpy(), d, d, layout, {}, "", None, 0)
    rx.qkv_store(rx.pool_desc(*pool), 0, rx.rope(d, layout=layout), pos, pos + 1, q, k, v, q)
    assert rx.device_check() == 0
    assert np.all(np.abs(_np(q) - want) <= tol)
    rest = torch.ones_like(room, dtype=torch.bool)
    rest[:, 8:8 + hq * d] = False
    assert torch.equal(room[rest], before[rest])
    assert torch.equal(pool[1][0, :, 1:].transpose(0, 1), v)


@pytest.mark.gpu
def test_norm_of_extreme_rows():
    """Rows of zeros (eps alone), of the smallest and of large magnitudes, and
    rows that are not finite, which stay within themselves."""
    import torch
    T, d = 6, 128
    x = torch.randn((T, 2, d), device="cuda")
    x[0] = 0
    x[1] *= 1e-18
    x[2] *= 1e15
    x[3, 0, 5] = float("inf")
    x[4, 1, 9] = float("nan")
    x = x.to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out, ko = torch.empty_like(x), torch.empty_like(x)
    rx.qk_rope(rx.rope(d), pos, x, x.clone(), out, ko, rx.head_norm(w, w, 1e-5))
    fine = torch.ones((T, 2), dtype=torch.bool)
    fine[3, 0] = fine[4, 1] = False
    want, tol = reference(_np(x), pos.cpu().numpy(), d, d, "half", {}, "weight", _np(w), 1e-5)
    ok = np.abs(_np(out) - want) <= tol
    assert ok[fine.numpy()].all()
    assert torch.isnan(out[4, 1].float()).all()
    assert torch.isfinite(out.float())[fine.cuda()].all()


@pytest.mark.gpu
def test_keys_alone_bad_slots_and_rows_behind():
    import torch
    T, hkv, d, N = 9, 2, 128, 32
    r = Rows(T + 2, 4, hkv, d, True, seed=5)
    pool = [torch.zeros((1, hkv, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([3, 0, -1, N, 5, 2 ** 31 - 1, 6, -2 ** 31, 7], dtype=torch.int32,
                         device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    desc = rx.pool_desc(*pool)
    rx.qkv_store(desc, 0, None, pos, slots, None, r.k[:T], r.v[:T], None)
    with pytest.raises(rx.RxError) as e:
        rx.device_check()
    assert "flags 1" in str(e.value)
    good = [0, 4, 6, 8]
    for p, x in zip(pool, (r.k, r.v)):
        want = torch.zeros_like(p)
        for t in good:
            want[0, :, int(slots[t])] = x[t]
        assert torch.equal(p, want)
    # queries of a token without a slot are written, rows behind T are not
    qo = torch.full((T + 2, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    rx.qkv_store(desc, 0, None, pos, slots, r.q[:T], r.k[:T], r.v[:T], qo[:T])
    with pytest.raises(rx.RxError):
        rx.device_check()
    assert torch.equal(qo[:T], r.q[:T]) and (qo[T:] == 7.0).all()
    rx.qkv_store(desc, 0, None, pos[:0], slots[:0], r.q[:0], r.k[:0], r.v[:0], qo[:0])
    assert rx.device_check() == 0


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    import torch
    T, hq, hkv, d, N = 40, 8, 2, 256, 64
    r = Rows(T, hq, hkv, d, True, seed=11)
    pool = [torch.zeros((1, hkv, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    desc = rx.pool_desc(*pool)
    slots = torch.arange(1, T + 1, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope, hn = rx.rope(d, layout="interleaved"), rx.head_norm(r.w[0], r.w[1], 1e-6)
    want = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
    rx.qkv_store(desc, 0, rope, pos, slots, r.q, r.k, r.v, want, hn)
    keep = [p.clone() for p in pool]
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rx.qkv_store(desc, 0, rope, pos, slots, r.q, r.k, r.v, out, hn)
    for p in pool:
        p.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(pool, keep))
    pos.add_(3)   # a replay reads its inputs anew
    graph.replay()
    torch.cuda.synchronize()
    other = torch.empty_like(want)
    with torch.cuda.stream(side):
        rx.qkv_store(desc, 0, rope, pos, slots, r.q, r.k, r.v, other, hn)
    side.synchronize()
    assert torch.equal(out, other) and not torch.equal(out, want)
    assert rx.device_check() == 0


@pytest.mark.gpu
def test_norm_alone_needs_no_positions():
    import torch
    r = Rows(9, 4, 2, 128, True, seed=3)
    norm = _norm("weight", r.w)
    q, k = r.q.clone(), r.k.clone()
    rx.qk_rope(None, None, r.q, r.k, q, k, norm)
    for got, x, w in ((q, r.q, r.w[0]), (k, r.k, r.w[1])):
        want, tol = reference(_np(x), None, 128, 0, "half", {}, "weight", _np(w), 1e-6)
        assert (np.abs(_np(got) - want) <= tol).all()
    pool = [torch.zeros((1, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.arange(1, 10, dtype=torch.int32, device="cuda")
    q2 = torch.empty_like(q)
    rx.qkv_store(rx.pool_desc(*pool), 0, None, None, slots, r.q, r.k, r.v, q2, norm)
    assert torch.equal(q2, q) and torch.equal(pool[0][0, :, 1:10], k.transpose(0, 1))
    assert torch.equal(pool[1][0, :, 1:10], r.v.transpose(0, 1)) and rx.device_check() == 0
