"""The 8-bit KV pool: store and load bit for bit, decode and extend attention
against softmax attention in 64 bits, and every refusal.

Tolerances of the attention follow from its roundings.  A softmax weight is
rounded to f16 (half a step: 2^-11 of it; below f16's normal range, where the
weight is under 2^-20 of the largest, 2^-25 of 2^-6 of the largest V scale);
a score carries fp32 rounding of its d products, and of a query elements under
2^-27 of the row's largest or so, in all at most 2^-18 of the row's largest
magnitude per element; an fp32 output nothing else of size, a bf16 output half
a step more (2^-8).  The tiles apply a V scale as the f16 product of a code and
the quotient of the scale and a reference: exact for powers of two, for any
other scale two more roundings of 2^-11 each.  Then a term p v is off by at
most (1 + 2^-11)^3 - 1 < 3.01 2^-11 of itself.  K scales multiply scores in
fp32.
"""

import ctypes as C

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx

E4M3 = np.zeros(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    E4M3[_c] = (-1.0 if _c & 128 else 1.0) * (
        np.nan if (_c & 127) == 127 else _m * 2.0 ** -9 if _e == 0 else
        (8 + _m) * 2.0 ** (_e - 10))
_POS = E4M3[:127]


def to_e4m3(x):
    """float64 -> e4m3 codes: nearest, ties to the even code, 448 at most."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | (np.signbit(x) * 128)).astype(np.uint8)


def scale_exp(amax):
    """The least e >= -126 with amax <= 448 * 2^e."""
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return e


def store_reference(codes, scales, block, slots, x):
    """rx_kv8_store of one of K and V, in place: codes uint8 [H, N, d],
    scales float64 [H, N / block], x float64 [T, H, d]."""
    N = codes.shape[1]
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 1 or s >= N:
            t += 1
            continue
        n = 1
        while (t + n < len(slots) and slots[t + n] == s + n and (s + n) // block == s // block
               and s + n < N):
            n += 1
        first, b = s % block, s // block
        for h in range(x.shape[1]):
            rows = x[t:t + n, h].copy()
            rows[np.isnan(rows)] = 0
            fin = np.abs(rows[np.isfinite(rows)])
            new = 2.0 ** scale_exp(fin.max() if fin.size else 0.0)
            old = scales[h, b] if first else 0.0
            if not 0 < old < np.inf:
                old = 0.0
            now = max(new, old)
            if first and now > old:
                codes[h, b * block:s] = to_e4m3(E4M3[codes[h, b * block:s]] * (old / now))
            scales[h, b] = now
            codes[h, s:s + n] = to_e4m3(rows / now)
        t += n


# ------------------------------------------------------------------ refusals
def _desc(**kw):
    f = dict(k_codes=1 << 20, v_codes=1 << 21, scales=1 << 22, num_slots=64, num_layers=2,
             num_kv_heads=2, head_dim=128, block=1)
    f.update(kw)
    return rx.rx_kv8_pool_desc(*(f[n] for n, _ in rx.rx_kv8_pool_desc._fields_))


BAD_POOLS = [dict(k_codes=0), dict(v_codes=None), dict(scales=None), dict(k_codes=(1 << 20) + 8),
             dict(v_codes=(1 << 20) + 1), dict(scales=(1 << 20) + 4), dict(head_dim=64),
             dict(head_dim=192), dict(num_slots=1), dict(num_layers=0), dict(num_kv_heads=0),
             dict(num_kv_heads=-1), dict(block=0), dict(block=3), dict(block=128),
             dict(block=-2), dict(block=32, num_slots=48), dict(num_slots=1 << 30),
             dict(num_slots=1 << 31, num_layers=1, num_kv_heads=1),
             dict(num_layers=1 << 20, num_kv_heads=1 << 20)]


def _calls():
    """Every device call with valid arguments, as (name, function of the pool
    and keyword changes)."""
    lib, X = rx._lib, 1 << 24
    info = rx.rx_decode_plan_info()
    info.plan_words, info.n_work, info.n_parts, info.workspace_bytes = 64, 1, 1, 4096

    def io(fn):
        def call(pool, layer=0, slots=X, k=X, v=X, T=4, **kw):
            return fn(C.byref(pool) if pool else None, layer, slots, k, v, T, None)
        return call

    def ext(pool, layer=0, q=X, hq=4, table=X, stride=64, rows=X, prefix=X, qo=X, tiles=X, R=1,
            nt=1, scale=0.1, out=X, ot=1, lse=X, **kw):
        return lib.rx_kv8_extend_attention(C.byref(pool) if pool else None, layer, q, hq, table,
                                           stride, rows, prefix, qo, tiles, R, nt, scale, out, ot,
                                           lse, None)

    def dec(pool, layer=0, q=X, hq=4, table=X, stride=64, plan=X, inf=info, B=1, step=0,
            scale=0.1, out=X, ot=0, lse=X, ws=X, wsb=4096, **kw):
        return lib.rx_kv8_decode_attention(C.byref(pool) if pool else None, layer, q, hq, table,
                                           stride, plan, C.byref(inf) if inf else None, B, step,
                                           scale, out, ot, lse, ws, wsb, None)
    return {"store": io(lib.rx_kv8_store), "load": io(lib.rx_kv8_load), "extend": ext,
            "decode": dec}


@pytest.mark.parametrize("call", ["store", "load", "extend", "decode"])
def test_bad_pools_are_refused_before_any_cuda_call(call):
    fn = _calls()[call]
    assert fn(None) == rx.RX_ERR_INVALID
    for bad in BAD_POOLS:
        assert fn(_desc(**bad)) == rx.RX_ERR_INVALID, bad
        assert rx.last_error()
    for layer in (-1, 2):
        assert fn(_desc(), layer=layer) == rx.RX_ERR_INVALID


X8 = (1 << 24) + 8


@pytest.mark.parametrize("call,bad", [
    (c, b) for c in ("store", "load") for b in (
        dict(T=-1), dict(T=1 << 30), dict(slots=None), dict(k=None), dict(v=None), dict(k=X8),
        dict(v=X8))] + [
    ("extend", b) for b in (
        dict(hq=3), dict(hq=0), dict(hq=-2), dict(R=-1), dict(nt=-1), dict(nt=1 << 40),
        dict(q=None), dict(table=None), dict(rows=None), dict(prefix=None), dict(qo=None),
        dict(tiles=None), dict(out=None), dict(lse=None), dict(q=X8), dict(out=X8),
        dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan")), dict(scale=float("inf")),
        dict(scale=2.0 ** -41), dict(scale=2.0 ** 41), dict(ot=2), dict(ot=-1),
        dict(stride=-1))] + [
    ("decode", b) for b in (
        dict(hq=3), dict(hq=0), dict(B=-1), dict(step=-1), dict(inf=None), dict(q=None),
        dict(table=None), dict(plan=None), dict(out=None), dict(lse=None), dict(ws=None),
        dict(ws=X8), dict(wsb=4095), dict(q=X8), dict(out=X8), dict(scale=0.0),
        dict(scale=float("nan")), dict(ot=7), dict(stride=-1))])
def test_bad_arguments_are_refused_before_any_cuda_call(call, bad):
    assert _calls()[call](_desc(), **bad) == rx.RX_ERR_INVALID
    assert rx.last_error()


def test_bad_plan_infos_are_refused():
    dec = _calls()["decode"]
    for f, v in (("n_work", -1), ("n_parts", -1), ("n_work_tc", 2), ("n_work_tc", -1),
                 ("n_work", 1 << 40)):
        info = rx.rx_decode_plan_info()
        info.n_work, info.n_parts, info.workspace_bytes = 1, 1, 0
        setattr(info, f, v)
        assert dec(_desc(), inf=info) == rx.RX_ERR_INVALID, f


def test_empty_calls_launch_nothing():
    c = _calls()
    assert c["store"](_desc(), T=0, slots=None, k=None, v=None) == rx.RX_OK
    assert c["load"](_desc(), T=0, slots=None, k=None, v=None) == rx.RX_OK
    assert c["extend"](_desc(), R=0) == rx.RX_OK
    assert c["extend"](_desc(), nt=0) == rx.RX_OK
    assert c["decode"](_desc(), B=0) == rx.RX_OK


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    kc = torch.zeros((1, 2, 64, 128), dtype=torch.uint8)
    sc = torch.ones((1, 2, 16, 2))
    p = rx.kv8_pool_desc(kc, kc.clone(), sc)
    assert p.block == 4 and p.num_slots == 64
    for args in ((kc, kc[:, :1], sc), (kc.float(), kc, sc), (kc, kc, sc.double()),
                 (kc, kc, sc[:, :, :7]), (kc, kc, sc[..., :1]), (kc, kc, sc[:, :1]),
                 (kc.transpose(1, 2), kc.transpose(1, 2), sc), (kc, kc, sc[0])):
        with pytest.raises(ValueError):
            rx.kv8_pool_desc(*args)
    s = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):        # not on a GPU
        rx.kv8_store(p, 0, s, x, x)


def test_reference_quantiser():
    """The reference itself: every code is its own rounding, midpoints go to
    the even code, and the scale rule at its borders."""
    keep = [c for c in range(256) if c & 127 != 127 and c != 128]
    assert (to_e4m3(E4M3[keep]) == keep).all()
    for c in range(126):
        mid = (E4M3[c] + E4M3[c + 1]) / 2
        assert to_e4m3(np.array([mid]))[0] == (c if c % 2 == 0 else c + 1)
    assert scale_exp(0.0) == -126 and scale_exp(448.0) == 0 and scale_exp(449.0) == 1
    assert scale_exp(1.0) == -8 and scale_exp(1.75) == -8 and scale_exp(1.7578125) == -7


# ------------------------------------------------------------- store and load
def _pool(torch, L, H, N, d, block, seed, fill=True):
    """A pool with random codes and scales everywhere (finite ones)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kc, vc = (torch.randint(0, 256, (L, H, N, d), generator=g, device="cuda",
                            dtype=torch.uint8) for _ in range(2))
    for c in (kc, vc):
        c[(c & 127) == 127] = 5
    e = torch.randint(-10, 3, (L, H, N // block, 2), generator=g, device="cuda")
    return kc, vc, torch.ldexp(torch.ones((), device="cuda"), e).float().contiguous()


def _check_store(torch, H, d, block, slots, N, x, layer=1, L=2, seed=3):
    kc, vc, sc = _pool(torch, L, H, N, d, block, seed)
    want_k, want_v = kc[layer].cpu().numpy().copy(), vc[layer].cpu().numpy().copy()
    want_s = sc[layer].double().cpu().numpy()
    rest = (kc.clone(), vc.clone(), sc.clone())
    pool = rx.kv8_pool_desc(kc, vc, sc)
    d_slots = torch.tensor(np.asarray(slots), dtype=torch.int32, device="cuda")
    rx.kv8_store(pool, layer, d_slots, x[0], x[1])
    torch.cuda.synchronize()
    ks, vs = want_s[..., 0].copy(), want_s[..., 1].copy()
    store_reference(want_k, ks, block, slots, x[0].double().cpu().numpy())
    store_reference(want_v, vs, block, slots, x[1].double().cpu().numpy())
    # a code of a negative value that rounds to zero keeps its sign on the
    # device as in the reference
    assert (kc[layer].cpu().numpy() == want_k).all()
    assert (vc[layer].cpu().numpy() == want_v).all()
    assert (sc[layer].double().cpu().numpy() == np.stack([ks, vs], axis=2)).all()
    other = 1 - layer
    assert torch.equal(kc[other], rest[0][other]) and torch.equal(sc[other], rest[2][other])
    return pool


def _rows(torch, T, H, d, seed, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn((T, H, d), generator=g, device="cuda") *
             torch.exp(spread * torch.randn((T, H, 1), generator=g, device="cuda"))
             ).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (77, 2), (1031, 3)])
def test_store_is_exact(d, block, T, H):
    """Runs of random lengths at random places of their blocks, blocks in a
    random order: codes and scales equal the definition's, and nothing else
    of the pool changes."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(T * 1000 + block + d)
    slots, left = [], T
    n_blocks = T + 3
    for b in rng.permutation(np.arange(1, n_blocks)):
        if left == 0:
            break
        n = int(rng.integers(1, min(block, left) + 1))
        first = int(rng.integers(0, block - n + 1))
        slots += list(range(b * block + first, b * block + first + n))
        left -= n
    assert left == 0
    _check_store(torch, H, d, block, slots, n_blocks * block, _rows(torch, T, H, d, T + d))
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 16, 64])
def test_store_of_contiguous_blocks_and_the_last_slot(block):
    """A run over many blocks (as a prefill hands out) up to the pool's last
    slot; the first block of a run starts late."""
    torch = pytest.importorskip("torch")
    N = 640
    slots = list(range(block // 2 + 1, N))
    _check_store(torch, 2, 128, block, slots, N, _rows(torch, len(slots), 2, 128, 9))
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
def test_store_token_by_token_grows_the_block_scale(d):
    """Appending a block's tokens one call at a time, each larger than the
    last: the scale follows, and the earlier rows are rounded again."""
    torch = pytest.importorskip("torch")
    H, block, N = 2, 16, 48
    kc, vc, sc = _pool(torch, 1, H, N, d, block, 1)
    pool = rx.kv8_pool_desc(kc, vc, sc)
    wk, wv = kc[0].cpu().numpy().copy(), vc[0].cpu().numpy().copy()
    ws = sc[0].double().cpu().numpy()
    ks, vs = ws[..., 0].copy(), ws[..., 1].copy()
    x = _rows(torch, 40, H, d, 4, spread=2.0)
    for i, s in enumerate(list(range(16, 48)) + list(range(16, 24))):
        st = torch.tensor([s], dtype=torch.int32, device="cuda")
        rx.kv8_store(pool, 0, st, x[0][i:i + 1].contiguous(), x[1][i:i + 1].contiguous())
        store_reference(wk, ks, block, [s], x[0][i:i + 1].double().cpu().numpy())
        store_reference(wv, vs, block, [s], x[1][i:i + 1].double().cpu().numpy())
    assert (kc[0].cpu().numpy() == wk).all() and (vc[0].cpu().numpy() == wv).all()
    assert (sc[0].double().cpu().numpy() == np.stack([ks, vs], axis=2)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 8])
def test_store_of_extreme_values(block):
    """Zeros, the smallest subnormals, the largest finite values and values at
    the scale rule's borders."""
    torch = pytest.importorskip("torch")
    vals = [0.0, 2.0 ** -133, 2.0 ** -126, 3.3895313892515355e38, 448.0, 450.0, 1.75, 1.7578125,
            -448.0, -0.0, 2.0 ** -120, 1e-30, 2.0 ** 120]
    T, H, d = len(vals) * 2, 2, 128
    x = torch.zeros((T, H, d))
    for i, v in enumerate(vals):
        x[i, 0, 5] = v
        x[i, 1] = v
        x[len(vals) + i, 0, 127] = v
        x[len(vals) + i, 0, 0] = v * 2.0 ** -9
    x = x.to(torch.bfloat16).cuda()
    N = 64 if block == 1 else (T + 1) * 8
    slots = list(range(1, T + 1)) if block == 1 else [8 * (i + 1) for i in range(T)]
    _check_store(torch, H, d, block, slots, N, [x, x.neg().contiguous()])
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 16])
def test_store_reports_values_that_are_not_finite(block):
    torch = pytest.importorskip("torch")
    x = _rows(torch, 32, 2, 128, 12)
    x[0][3, 1, 7] = float("nan")
    x[0][3, 0, 9] = float("inf")
    x[1][20, 0, 100] = float("-inf")
    x[1][21, 1] = float("nan")
    _check_store(torch, 2, 128, block, list(range(16, 48)), 64, x)
    with pytest.raises(rx.RxError) as e:
        rx.device_check()
    assert "flags 64" in str(e.value)
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("block", [1, 4])
def test_bad_slots_are_skipped_and_reported(block):
    torch = pytest.importorskip("torch")
    slots = [0, 5, 64, -1, 12, 13, 2 ** 31 - 1, -2 ** 31, 63]
    x = _rows(torch, len(slots), 2, 128, 2)
    pool = _check_store(torch, 2, 128, block, slots, 64, x)
    with pytest.raises(rx.RxError) as e:
        rx.device_check()
    assert "flags 1" in str(e.value)
    out = [torch.full_like(t, 7.0) for t in x]
    rx.kv8_load(pool, 1, torch.tensor(slots, dtype=torch.int32, device="cuda"), *out)
    for i, s in enumerate(slots):
        if s < 1 or s > 63:
            assert not out[0][i].any() and not out[1][i].any()
        else:
            assert out[0][i].any()
    with pytest.raises(rx.RxError):
        rx.device_check()


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 13, 250])
def test_tokens_of_a_block_out_of_slot_order_are_skipped_and_reported(shift):
    """A repeated slot, one before its neighbour's and one that leaves a gap:
    the first run of the block is stored, the later one is not.  (shift: at
    other places of the kernel's window of tokens.)"""
    torch = pytest.importorskip("torch")
    lead = list(range(512, 512 + shift))
    slots = lead + [5, 4, 9, 9, 10, 16, 17, 19, 20, 24]
    kept = [i for i in range(len(slots)) if i - shift not in (1, 3, 4, 7, 8)]
    x = _rows(torch, len(slots), 2, 128, 9)
    kc, vc, sc = _pool(torch, 1, 2, 1024, 128, 8, 4)
    two = [t.clone() for t in (kc, vc, sc)]
    rx.kv8_store(rx.kv8_pool_desc(kc, vc, sc), 0,
                 torch.tensor(slots, dtype=torch.int32, device="cuda"), *x)
    with pytest.raises(rx.RxError) as e:
        rx.device_check()
    assert "flags 128" in str(e.value) and "out of slot order" in str(e.value)
    # what remains, without a repeat: 24's neighbour is 17, of another block
    rx.kv8_store(rx.kv8_pool_desc(*two), 0,
                 torch.tensor([slots[i] for i in kept], dtype=torch.int32, device="cuda"),
                 *[t[kept].contiguous() for t in x])
    assert rx.device_check() == 0
    for u, v in zip((kc, vc, sc), two):
        assert torch.equal(u, v)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("block,T,H", [(1, 1, 1), (1, 333, 3), (16, 517, 2), (64, 5, 7)])
def test_load_is_exact(d, block, T, H):
    """Every finite code comes back as bf16(code * scale), for powers of two
    and for other scales, repeated slots included."""
    torch = pytest.importorskip("torch")
    N = 640
    kc, vc, sc = _pool(torch, 2, H, N, d, block, 5)
    sc[0, :, ::3] *= 1.2345
    pool = rx.kv8_pool_desc(kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), sc)
    rng = np.random.default_rng(T)
    slots = rng.integers(1, N, T)
    out = [torch.full((T + 1, H, d), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for layer in (0, 1):
        rx.kv8_load(pool, layer, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                    out[0][:T], out[1][:T])
        for o, c, w in ((out[0], kc, 0), (out[1], vc, 1)):
            val = E4M3[c[layer].cpu().numpy()[:, slots]].astype(np.float32)
            val *= sc[layer].cpu().numpy()[:, slots // block, w][..., None]   # one fp32 product
            want = torch.from_numpy(val).to(torch.bfloat16).permute(1, 0, 2)
            assert torch.equal(o[:T].cpu(), want)
            assert (o[T] == 3.0).all()
    assert rx.device_check() == 0


# ------------------------------------------------------------------ attention
class Case:
    """A pool in which only the slots the tables name hold anything finite,
    requests over it, and attention in 64 bits with its error bound."""

    def __init__(self, torch, Hq, H, d, block, ctx, seed, shared=0, page=None, spread=0.5,
                 unit_scale=False, pow2=False):
        self.torch, self.Hq, self.H, self.d, self.block = torch, Hq, H, d, block
        self.page = page = page or block
        rng = np.random.default_rng(seed)
        cut = shared // page * page
        lens = [cut] + [c - cut for c in ctx]
        n_pages = [-(-x // page) for x in lens]
        total = sum(n_pages) + 4
        order = 1 + rng.permutation(total - 1)
        self.N = -(-total * page // block) * block
        rows, at = [], 0
        for x, p in zip(lens, n_pages):
            ids = order[at:at + p]
            if p > 3:          # long runs of pages in order, as an allocator gives
                ids = np.sort(ids)
            at += p
            rows.append((ids[:, None] * page + np.arange(page)).reshape(-1)[:x])
        self.ctx, self.cut = list(ctx), cut
        self.table = np.zeros((len(ctx), max(ctx) + 3), dtype=np.int32)
        for b, c in enumerate(ctx):
            self.table[b, :c] = np.concatenate([rows[0], rows[1 + b]])
            self.table[b, c:] = 2 ** 30          # never read
        used = np.unique(np.concatenate(rows).astype(np.int64))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        L = 2
        self.layer = 1
        self.kc, self.vc = (torch.full((L, H, self.N, d), 127, dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.sc = torch.full((L, H, self.N // block, 2), float("nan"), device="cuda")
        for c in (self.kc, self.vc):
            r = torch.randn((H, len(used), d), generator=g, device="cuda") * 100
            r = r.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c[1][:, torch.from_numpy(used).cuda()] = r
        e = torch.randn((H, self.N // block, 2), generator=g, device="cuda") * spread
        s = (torch.exp(e) * 0.01)
        if pow2:
            s = torch.exp2(torch.floor(torch.log2(s)))
        self.term = 2.0 ** -11 if pow2 else 3.01 * 2.0 ** -11
        self.score = 2.0 ** -20
        ub = torch.from_numpy(np.unique(used // block)).cuda()
        self.sc[1][:, ub] = s[:, ub]
        self.scale = 1.0 / np.sqrt(d) if not unit_scale else 1.0
        self.pool = rx.kv8_pool_desc(self.kc, self.vc, self.sc)
        self.k = E4M3[self.kc[1].cpu().numpy()[:, used]]
        self.v = E4M3[self.vc[1].cpu().numpy()[:, used]]
        sc = self.sc[1].double().cpu().numpy()[:, used // block]
        self.k, self.v, self.vs = self.k * sc[..., :1], self.v * sc[..., 1:], sc[..., 1]
        self.index = np.full(self.N, -1)
        self.index[used] = np.arange(len(used))
        self.gen = g

    def up(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def queries(self, n, mag=1.0):
        t = self.torch
        q = t.randn((n, self.Hq, self.d), generator=self.gen, device="cuda") * mag
        return q.to(t.bfloat16)

    def reference(self, q, b, lim):
        """o, lse and their bounds of queries q [s, Hq, d] of request b seeing
        lim[i] keys."""
        G = self.Hq // self.H
        idx = self.index[self.table[b, :self.ctx[b]]]
        o = np.zeros(q.shape)
        lse = np.zeros(q.shape[:2])
        bo, bl = np.zeros(q.shape), np.zeros(q.shape[:2])
        for h in range(self.Hq):
            k, v, vs = (x[h // G][idx] for x in (self.k, self.v, self.vs))
            qh = q[:, h]
            s = qh @ k.T * self.scale
            a = np.abs(qh) @ np.abs(k).T * self.scale          # fp32 rounding of the products
            split = np.abs(qh).max(axis=1)[:, None] * np.abs(k).sum(axis=1)[None] * self.scale
            hide = np.arange(len(idx))[None] >= np.asarray(lim)[:, None]
            s[hide] = -np.inf
            a[hide] = split[hide] = 0
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(axis=1, keepdims=True)
            o[:, h] = p @ v / l
            lse[:, h] = (m + np.log(l))[:, 0]
            ds = (a * self.score + split * 2.0 ** -18).max(axis=1) + 2.0 ** -20
            w = p @ np.abs(v) / l
            tiny = 448 * vs.max() * 2.0 ** -31 * p.astype(bool).sum(axis=1) / l[:, 0]
            bo[:, h] = (self.term + ds)[:, None] * w + ds[:, None] * np.abs(o[:, h]) + \
                tiny[:, None]
            bl[:, h] = ds + np.abs(lse[:, h]) * 2.0 ** -22
        return o, lse, bo, bl

    def compare(self, got_o, got_l, ref, bf16):
        o, lse, bo, bl = ref
        go, gl = got_o.double().cpu().numpy(), got_l.double().cpu().numpy()
        if bf16:
            bo = bo * (1 + 2.0 ** -8) + np.abs(o) * 2.0 ** -8
        assert np.isfinite(go).all() and np.isfinite(gl).all()
        bad = np.abs(go - o) > bo
        assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst " \
                              f"{(np.abs(go - o) / bo).max():.3f} of the bound"
        assert (np.abs(gl - lse) <= bl).all(), np.abs(gl - lse).max()


def _decode(c, q, nodes=None, depth=None, bf16=True, n_steps=None, step=0, ctx=None, q_rows=None):
    """rx_kv8_decode_attention of the case's requests (table rows 0 ..)."""
    torch = c.torch
    B = len(c.ctx) if ctx is None else len(ctx)
    ctx = c.ctx if ctx is None else ctx
    cache = rx.RadixCache(c.N // c.page * c.page, c.page)
    nodes = []
    for b in range(B):
        keep = c.ctx[b] if depth is None else depth[b]
        ids = np.arange(keep, dtype=np.int32)
        ids[c.cut:] += 1000000 * (b + 1)
        nodes.append(cache.insert(ids, c.table[b, :keep])[1])
    plan, info = cache.plan_decode(nodes, ctx, np.arange(B), c.Hq, c.H, c.d, n_steps=n_steps)
    out = torch.full((B + 1, c.Hq, c.d), 9.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                     device="cuda")
    lse = torch.full((B + 1, c.Hq), 9.0, device="cuda")
    ws = torch.full((int(info.workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
    d_plan, d_table = c.up(plan[:int(info.plan_words)]), c.up(c.table)
    rx.kv8_decode_attention(c.pool, c.layer, q, c.Hq, d_table, d_plan, info, B, c.scale, out[:B],
                            lse[:B], ws, step=step)
    torch.cuda.synchronize()
    assert (out[B] == 9.0).all() and (lse[B] == 9.0).all()
    assert rx.device_check() == 0
    return out[:B], lse[:B]


DECODE = [
    # Hq, Hkv, d, block, page, contexts, shared
    (1, 1, 128, 1, 1, [1], 0),
    (4, 1, 256, 1, 1, [1, 2, 31, 32, 33], 0),
    (8, 2, 128, 1, 1, [5, 700, 129, 64], 0),
    (32, 8, 128, 16, 16, [300, 17, 1025], 0),
    (8, 8, 128, 64, 64, [63, 64, 65, 200], 0),
    (24, 2, 128, 2, 4, [100, 3], 0),                 # 12 heads a group
    (16, 1, 128, 1, 1, [257, 1100], 0),              # 16 rows a request
    (64, 1, 128, 1, 1, [513, 40], 0),                # 64 rows a request: tiles alone
    (16, 4, 256, 16, 16, [900, 450, 1, 16], 0),
    (32, 1, 256, 4, 16, [333], 0),
    (32, 8, 128, 1, 1, [1200 + i for i in range(12)], 1100),
    (16, 4, 256, 16, 16, [700 + 7 * i for i in range(40)], 640),
    (8, 1, 128, 1, 1, [800 + i for i in range(3)], 800),
    (16, 2, 256, 1, 1, [600 + (i % 3) for i in range(70)], 599),
    (64, 8, 128, 8, 16, [2600 + 3 * i for i in range(24)], 2592),
    # few tiles over many common keys: clusters share a tile's keys
    (16, 2, 128, 1, 1, [3000 + i for i in range(30)], 2999),
    (8, 1, 256, 16, 16, [4100 + (i % 5) for i in range(20)], 4096),
    (64, 1, 256, 1, 1, [1500], 0),
    (128, 1, 128, 64, 64, [2500, 1], 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_matches_64_bits(i, bf16):
    torch = pytest.importorskip("torch")
    Hq, H, d, block, page, ctx, shared = DECODE[i]
    c = Case(torch, Hq, H, d, block, ctx, 100 + i, shared=shared, page=page)
    q = c.queries(len(ctx))
    o, lse = _decode(c, q, bf16=bf16)
    qn = q.double().cpu().numpy()
    for b in range(len(ctx)):
        c.compare(o[b:b + 1], lse[b:b + 1], c.reference(qn[b:b + 1], b, [ctx[b]]), bf16)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode_with_power_of_two_scales(i):
    """Scales as rx_kv8_store writes them: one rounding of a weight is all."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, page, ctx, shared = DECODE[i]
    c = Case(torch, Hq, H, d, block, ctx, 300 + i, shared=shared, page=page, spread=1.5, pow2=True)
    q = c.queries(len(ctx))
    o, lse = _decode(c, q, bf16=False)
    qn = q.double().cpu().numpy()
    for b in range(len(ctx)):
        c.compare(o[b:b + 1], lse[b:b + 1], c.reference(qn[b:b + 1], b, [ctx[b]]), False)


def _extend(c, prefix, q, bf16=True, R=None):
    torch = c.torch
    sfx = np.array(c.ctx) - np.array(prefix)
    R = len(sfx)
    qo = np.concatenate([[0], np.cumsum(sfx)])
    tiles, n = rx.extend_plan(qo, c.Hq, c.H, c.d)
    T = int(qo[-1])
    out = torch.full((T + 1, c.Hq, c.d), 9.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                     device="cuda")
    lse = torch.full((T + 1, c.Hq), 9.0, device="cuda")
    rx.kv8_extend_attention(c.pool, c.layer, q, c.Hq, c.up(c.table), c.up(np.arange(R)),
                            c.up(prefix), c.up(qo), c.up(tiles), R, n, c.scale, out[:T], lse[:T])
    torch.cuda.synchronize()
    assert (out[T] == 9.0).all() and (lse[T] == 9.0).all()
    assert rx.device_check() == 0
    return out[:T], lse[:T], qo


EXTEND = [
    # Hq, Hkv, d, block, page, prefixes, suffixes
    (1, 1, 128, 1, 1, [0], [1]),
    (4, 4, 256, 1, 1, [0, 3], [1, 2]),
    (8, 2, 128, 1, 1, [0, 129, 1], [64, 31, 200]),
    (32, 8, 128, 16, 16, [256, 0, 1000], [33, 0, 7]),
    (16, 4, 256, 16, 16, [640, 16, 0], [50, 129, 65]),
    (24, 2, 128, 2, 4, [100, 0], [11, 40]),
    (8, 1, 256, 64, 64, [64, 0], [70, 3]),
    (3, 1, 128, 1, 1, [77], [300]),
    (64, 1, 128, 8, 8, [15], [5]),
    (16, 2, 256, 1, 16, [1500], [20]),
    (8, 8, 128, 32, 32, [0], [700]),
    # few tiles over many keys: clusters share a tile's keys, rows see some parts only
    (1, 1, 128, 1, 1, [0], [2000]),
    (8, 2, 128, 16, 16, [4992], [3]),
    (2, 1, 256, 16, 16, [1488, 0, 4000], [100, 900, 1]),
    (4, 4, 256, 1, 1, [700, 0], [30, 5]),
    (32, 8, 128, 8, 8, [600], [400]),                # 104 CTAs: none
    (16, 4, 256, 64, 64, [576], [390]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("i", range(len(EXTEND)))
def test_extend_matches_64_bits(i, bf16):
    torch = pytest.importorskip("torch")
    Hq, H, d, block, page, prefix, sfx = EXTEND[i]
    ctx = [max(1, p + s) for p, s in zip(prefix, sfx)]
    prefix = [x - s for x, s in zip(ctx, sfx)]
    c = Case(torch, Hq, H, d, block, ctx, 200 + i, page=page)
    q = c.queries(int(sum(sfx)))
    o, lse, qo = _extend(c, prefix, q, bf16)
    qn = q.double().cpu().numpy()
    for b in range(len(ctx)):
        a, e = int(qo[b]), int(qo[b + 1])
        if e > a:
            lim = prefix[b] + 1 + np.arange(e - a)
            c.compare(o[a:e], lse[a:e], c.reference(qn[a:e], b, lim), bf16)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(EXTEND)))
def test_extend_with_power_of_two_scales(i):
    torch = pytest.importorskip("torch")
    Hq, H, d, block, page, prefix, sfx = EXTEND[i]
    ctx = [max(1, p + s) for p, s in zip(prefix, sfx)]
    prefix = [x - s for x, s in zip(ctx, sfx)]
    c = Case(torch, Hq, H, d, block, ctx, 400 + i, page=page, spread=1.5, pow2=True)
    q = c.queries(int(sum(sfx)))
    o, lse, qo = _extend(c, prefix, q, False)
    qn = q.double().cpu().numpy()
    for b in range(len(ctx)):
        a, e = int(qo[b]), int(qo[b + 1])
        if e > a:
            lim = prefix[b] + 1 + np.arange(e - a)
            c.compare(o[a:e], lse[a:e], c.reference(qn[a:e], b, lim), False)
