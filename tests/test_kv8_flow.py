"""The 8-bit KV pool as it is used: the request flow over it (store, extend,
decode, read back), and the calls around one another: captured and replayed,
on other streams, two at once, planned steps, drafts, empty contexts, queries
that are not finite, pools beyond 2^31 bytes.

In the flows every K and V value is an e4m3 number of magnitude 2^-6 .. 4, or
zero, which a block's scale (its largest 4 at most, so 2^-7 at most) holds
exactly: the pool then has exactly the oracle's K and V, and the flow's
tolerance is the one of the bf16 pool, of which the roundings here (a weight
2^-11, a score 2^-18 of its row's largest query times the key's sum) take
less than half.
"""

import ctypes as C
import functools

import numpy as np
import pytest

from radix_tree_prefix_gb300 import engine as engine_mod
from radix_tree_prefix_gb300 import rx, workloads
from radix_tree_prefix_gb300.engine import Engine

from test_kv8 import Case, _calls, _decode, _desc, _extend


# ------------------------------------------------------------------ refusals
def test_engine_refuses_blocks_that_pages_do_not_hold():
    wl = workloads.agent_loop(calls=3, preamble=100, lo=10, hi=20, decode_steps=2)
    for block in (2, 3, 128, -1):
        with pytest.raises(ValueError):
            Engine(wl, kv8_block=block)
    paged = workloads.with_pages(wl, 8)
    with pytest.raises(ValueError):
        Engine(paged, kv8_block=16)
    with pytest.raises(ValueError):
        Engine(paged, kv8_block=8, host_slots=64)
    assert Engine(paged, kv8_block=8).run().as_tuple() == Engine(paged).run().as_tuple()


def test_waves_refuse_bad_lists_before_any_cuda_call():
    lib, X = rx._lib, 1 << 24
    ok = _desc()
    rec = np.zeros(1, dtype=rx.EXTEND_BATCH_DTYPE)
    st = np.zeros(1, dtype=rx.DECODE_STEP_DTYPE)

    def ext(pool=ok, layer=0, p=rec.ctypes.data, n=1):
        return lib.rx_kv8_extend_batches(C.byref(pool), layer, 4, p, n, 0.1, None, None)

    def dec(pool=ok, layer=0, hq=4, p=st.ctypes.data, n=1, B=1):
        return lib.rx_kv8_decode_steps(C.byref(pool), layer, hq, X, 64, p, n, B, 0.1, X, 4096,
                                       None)
    for fn in (ext, dec):
        assert fn(n=-1) == rx.RX_ERR_INVALID
        assert fn(p=None) == rx.RX_ERR_INVALID
        assert fn(pool=_desc(block=3)) == rx.RX_ERR_INVALID
        assert fn(layer=2) == rx.RX_ERR_INVALID
        assert fn(n=0) == rx.RX_OK
    assert dec(hq=3) == rx.RX_ERR_INVALID
    assert dec() == rx.RX_ERR_INVALID           # the record: NULL inputs
    assert dec(B=-1) == rx.RX_ERR_INVALID
    rec["n_new"] = 1
    assert ext() == rx.RX_ERR_INVALID
    rec["n_new"] = 0
    assert ext() == rx.RX_OK                    # no tokens, no tiles: nothing to launch
    assert _calls()["store"](ok, T=-1) == rx.RX_ERR_INVALID


def test_calls_refuse_the_other_kind_of_pool():
    """A bf16 call never reads an 8-bit pool's descriptor, nor the reverse."""
    torch = pytest.importorskip("torch")
    kc = torch.zeros((1, 2, 64, 128), dtype=torch.uint8)
    p8 = rx.kv8_pool_desc(kc, kc.clone(), torch.ones((1, 2, 16, 2)))
    kp = torch.zeros((1, 2, 64, 128), dtype=torch.bfloat16)
    p16 = rx.pool_desc(kp, kp)
    lib = rx._lib
    for name, types in rx._SIGS.items():
        if types and types[0] in (rx.POOL, rx.POOL8):
            other = p16 if types[0] is rx.POOL8 else p8
            args = [C.byref(other) if t in (rx.POOL, rx.POOL8) else
                    0 if t in (C.c_int32, C.c_int64, C.c_size_t) else
                    0.0 if t is C.c_float else None for t in types]
            with pytest.raises(C.ArgumentError):
                getattr(lib, name)(*args)
    s = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(AttributeError):
        rx.kv8_store(p16, 0, s, x, x)


# --------------------------------------------------------------------- flows
def _to_e4m3_values(vals):
    import torch
    for kind in ("k", "v"):
        for layer, x in vals[kind].items() if isinstance(vals[kind], dict) else \
                enumerate(vals[kind]):
            if x is None:
                continue
            y = x.float().clamp(-4, 4)
            y = torch.where(y.abs() < 2.0 ** -6, torch.zeros_like(y), y)
            x.copy_(y.to(torch.float8_e4m3fn).to(torch.bfloat16))


FLOWS = [
    # workload, page, block, engine arguments
    ("agent", 1, 1, {}),
    ("agent", 64, 8, dict(chunk_tokens=97)),
    ("chat", 16, 16, {}),
    ("chat", 32, 4, {}),
    ("nested", 8, 2, {}),
    ("fork", 1, 1, dict(policy="lpm")),
    ("shared", 64, 64, {}),
]


def _flow_workload(name, page):
    wl = {
        "agent": lambda: workloads.agent_loop(calls=6, preamble=300, lo=20, hi=60,
                                              decode_steps=4),
        "chat": lambda: workloads.multi_turn_chat(sessions=6, turns=3, system=200, user=30,
                                                  decode_steps=6, layers=1),
        "nested": lambda: workloads.nested_share(instr=150, doc=90, unique=33),
        "fork": lambda: workloads.fork_tree(branching=3, depth=3, level_tokens=40,
                                            decode_steps=3),
        "shared": lambda: workloads.long_shared(batch=6, prefix=700, unique=90, decode_steps=5,
                                                q_heads=16, kv_heads=8),
    }[name]()
    return workloads.with_pages(wl, page) if page > 1 else wl


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(FLOWS)))
def test_flow_matches_the_oracle(i, monkeypatch):
    """A workload through store, extend and decode over an 8-bit pool:
    bookkeeping equal to the oracle's, attention within the flow's tolerance,
    and the last wave's tokens read back exactly."""
    torch = pytest.importorskip("torch")
    from parity_util import DeviceRun
    name, page, block, kw = FLOWS[i]
    wl = _flow_workload(name, page)
    monkeypatch.setattr(engine_mod, "Engine", functools.partial(Engine, kv8_block=block))
    run = DeviceRun(wl, layers=[0], values_fn=_to_e4m3_values, extend_tokens=24, **kw)
    run.assert_close()
    eng = run.engine
    assert eng.kv8_block == block and eng.k_pool.dtype == torch.float8_e4m3fn
    assert eng.gpu_launches > 0
    wave = wl.waves[-1]
    by_rid = {int(r.rid): b for b, r in enumerate(wave)}
    last = eng.trace.decode_steps[-1] if wl.decode_steps else None
    assert len(by_rid) == len(wave)
    order = [int(x) for x in last.rids] if last is not None else [int(r.rid) for r in wave]
    for b, rid in enumerate(order):
        r = wl.requests[rid]
        idx = np.concatenate([wl.prompt_store_index(r),
                              wl.output_store_index(r)[:wl.decode_steps]])
        slots = torch.from_numpy(eng.h_table[b, :len(idx)].copy()).cuda()
        k, v = (torch.empty((len(idx), wl.num_kv_heads, wl.head_dim), dtype=torch.bfloat16,
                            device="cuda") for _ in range(2))
        rx.kv8_load(eng.pool, 0, slots, k, v)
        at = torch.from_numpy(np.asarray(idx, dtype=np.int64)).cuda()
        assert torch.equal(k, run.vals["k"][0].index_select(0, at))
        assert torch.equal(v, run.vals["v"][0].index_select(0, at))
    assert rx.device_check() == 0


@pytest.mark.gpu
def test_timed_flow_records_its_kernels():
    pytest.importorskip("torch")
    import torch
    from radix_tree_prefix_gb300.engine import GatherInputs
    wl = _flow_workload("agent", 16)
    dev = torch.device("cuda:0")
    vals = workloads.make_values(wl, dev, [0])
    for kw in ({}, dict(chunk_tokens=50)):
        eng = Engine(wl, device=dev, inputs=GatherInputs(wl, vals, [0]), layers=[0], timing=True,
                     kv8_block=16, **kw)
        eng.run()
        torch.cuda.synchronize()
        kinds = {k for k, *_ in eng.kernel_events}
        assert kinds == {"kv_store", "extend", "decode"}
        assert all(w > 0 and s.elapsed_time(e) >= 0 for _, s, e, w in eng.kernel_events)
        eng.close()
    assert rx.device_check() == 0


# ------------------------------------------------------- calls around calls
def _step(c):
    """The arguments of a decode call of the case, as a program keeps them."""
    torch = c.torch
    B = len(c.ctx)
    cache = rx.RadixCache(c.N // c.page * c.page, c.page)
    nodes = []
    for b in range(B):
        ids = np.arange(c.ctx[b], dtype=np.int32)
        ids[c.cut:] += 1000000 * (b + 1)
        nodes.append(cache.insert(ids, c.table[b, :c.ctx[b]])[1])
    plan, info = cache.plan_decode(nodes, c.ctx, np.arange(B), c.Hq, c.H, c.d)
    d_plan, table = c.up(plan[:int(info.plan_words)]), c.up(c.table)

    def call(q, out, lse, ws, stream=None):
        rx.kv8_decode_attention(c.pool, c.layer, q, c.Hq, table, d_plan, info, B, c.scale, out,
                                lse, ws, stream=stream)

    def bufs():
        return (torch.empty((B, c.Hq, c.d), device="cuda"), torch.empty((B, c.Hq), device="cuda"),
                torch.empty(int(info.workspace_bytes), dtype=torch.uint8, device="cuda"))
    return call, bufs


SHAPES = [(32, 8, 128, 1, [700 + i for i in range(12)], 600),      # tiles and streams
          (16, 4, 256, 16, [900, 450, 1, 16], 0),                  # streams alone
          (64, 8, 128, 16, [640 + 5 * i for i in range(80)], 624)]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_decode_on_streams_and_in_graphs(i):
    """The same bits eagerly, on another stream, as two calls at once with a
    workspace each, and captured and replayed with other queries."""
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 50 + i, shared=shared)
    qa, qb = c.queries(len(ctx)), c.queries(len(ctx))
    call, bufs = _step(c)
    want = []
    for q in (qa, qb):
        o, l, ws = bufs()
        call(q, o, l, ws)
        want.append((o, l))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    b1, b2 = bufs(), bufs()
    for _ in range(3):
        call(qa, *b1, stream=s1)
        with torch.cuda.stream(s2):
            call(qb, *b2)
    torch.cuda.synchronize()
    for got, w in ((b1, want[0]), (b2, want[1])):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    q, b3 = qa.clone(), bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, *b3)
    for src, w in ((qb, want[1]), (qa, want[0]), (qb, want[1])):
        q.copy_(src)
        b3[0].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b3[0], w[0]) and torch.equal(b3[1], w[1])
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d,block,Hq,T", [(128, 1, 16, 200), (256, 16, 16, 200),
                                          (128, 64, 16, 200), (128, 1, 4, 1000),
                                          (256, 8, 4, 700)])
def test_store_extend_and_load_in_a_graph(d, block, Hq, T):
    """A captured prefill (store, extend over it, load) replayed with other
    rows equals the eager calls (the last two: over clusters)."""
    torch = pytest.importorskip("torch")
    H, N = 4, 1088
    slots = torch.arange(64, 64 + T, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(h):
        return torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16)

    def up(a):
        return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    tiles, n = rx.extend_plan(np.array([0, T]), Hq, H, d)
    table, zero, one, qo, tl = slots.view(1, T), up([0]), up([0]), up([0, T]), up(tiles)

    def run(pool, k, v, q, o, l, kb, vb):
        rx.kv8_store(pool, 0, slots, k, v)
        rx.kv8_extend_attention(pool, 0, q, Hq, table, zero, one, qo, tl, 1, n, d ** -0.5, o, l)
        rx.kv8_load(pool, 0, slots, kb, vb)

    def make():
        kc, vc = (torch.zeros((1, H, N, d), dtype=torch.uint8, device="cuda") for _ in range(2))
        sc = torch.zeros((1, H, N // block, 2), device="cuda")
        return [rx.kv8_pool_desc(kc, vc, sc), rows(H), rows(H), rows(Hq),
                torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda"),
                torch.empty((T, Hq), device="cuda"),
                torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda"),
                torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")]
    a, b = make(), make()
    run(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*b)
    for x, y in zip(b[1:4], a[1:4]):
        x.copy_(y)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a[4:], b[4:]):
        assert torch.equal(x, y)
    for x, y in zip(a[0].tensors, b[0].tensors):
        assert torch.equal(x, y)
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d,block,page", [(16, 4, 256, 16, 16), (32, 8, 128, 1, 1),
                                               (64, 1, 128, 4, 8)])
def test_steps_of_one_plan_match_64_bits(Hq, H, d, block, page):
    """rx_plan_decode_steps: at step t every context is t keys longer."""
    torch = pytest.importorskip("torch")
    steps, base = 40, [300, 331, 1, 129, 640]
    c = Case(torch, Hq, H, d, block, [x + steps - 1 for x in base], 77, page=page)
    q = c.queries(len(base))
    qn = q.double().cpu().numpy()
    depth = [max(0, (x - 1) // page * page) for x in base]
    for t in (0, 1, 17, steps - 1):
        o, lse = _decode(c, q, depth=depth, bf16=False, n_steps=steps, step=t, ctx=base)
        for b, x in enumerate(base):
            c.compare(o[b:b + 1], lse[b:b + 1], c.reference(qn[b:b + 1], b, [x + t]), False)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d,G", [(64, 1, 128, 64), (16, 1, 256, 16), (32, 2, 256, 16),
                                      (8, 2, 128, 4), (4, 1, 256, 4)])
def test_items_whose_keys_come_at_later_steps(Hq, H, d, G):
    """A plan of 700 steps from a short context: chunks of the growing tail
    that no step has reached yet leave empty partial rows (tiles where the
    group is large, streams where it is not)."""
    torch = pytest.importorskip("torch")
    assert Hq == H * G
    steps, base = 700, [1, 100]
    c = Case(torch, Hq, H, d, 1, [x + steps - 1 for x in base], 78)
    q = c.queries(len(base))
    qn = q.double().cpu().numpy()
    for t in (0, 1, 300, steps - 1):
        o, lse = _decode(c, q, depth=[x - 1 for x in base], bf16=False, n_steps=steps, step=t,
                         ctx=base)
        for b, x in enumerate(base):
            c.compare(o[b:b + 1], lse[b:b + 1], c.reference(qn[b:b + 1], b, [x + t]), False)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d,block", [(32, 8, 128, 1), (16, 4, 256, 1)])
def test_drafts_of_a_tree_match_64_bits(Hq, H, d, block):
    """The rows of rx_verify_rows as a decode batch: each draft sees the
    prefix and its path to the root."""
    torch = pytest.importorskip("torch")
    parents = np.array([-1, 0, 0, 1, -1, 4, 3, 2], dtype=np.int32)
    n, prefix = len(parents), 333
    c = Case(torch, Hq, H, d, block, [prefix + n], 91)
    drafts = c.table[0, prefix:prefix + n].copy()
    rows, ctx, _ = rx.verify_rows([prefix], c.table[:1, :prefix].copy(),
                                  np.array([0, n], dtype=np.int64), parents, drafts, prefix + n)
    cache = rx.RadixCache(c.N, 1)
    _, node = cache.insert(np.arange(prefix, dtype=np.int32), c.table[0, :prefix])
    plan, info = cache.plan_decode([node] * n, ctx, np.arange(n), Hq, H, d)
    q = c.queries(n)
    out = torch.empty((n, Hq, d), device="cuda")
    lse = torch.empty((n, Hq), device="cuda")
    ws = torch.empty(int(info.workspace_bytes), dtype=torch.uint8, device="cuda")
    rx.kv8_decode_attention(c.pool, c.layer, q, Hq, c.up(rows), c.up(plan[:int(info.plan_words)]),
                            info, n, c.scale, out, lse, ws)
    assert rx.device_check() == 0
    qn = q.double().cpu().numpy()
    c.table, c.ctx = rows, [int(x) for x in ctx]
    for b in range(n):
        c.compare(out[b:b + 1], lse[b:b + 1], c.reference(qn[b:b + 1], b, [c.ctx[b]]), False)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_queries_that_are_not_finite_stay_in_their_rows(i, bad):
    torch = pytest.importorskip("torch")
    Hq, H, d, block, ctx, shared = SHAPES[i]
    c = Case(torch, Hq, H, d, block, ctx, 60 + i, shared=shared)
    q = c.queries(len(ctx))
    o, l = _decode(c, q, bf16=False)
    p = q.clone()
    p[1, 3, 7] = bad
    p[2 % len(ctx), Hq - 1, d - 1] = bad
    o2, l2 = _decode(c, p, bf16=False)
    hit = torch.zeros((len(ctx), Hq), dtype=torch.bool, device="cuda")
    hit[1, 3] = hit[2 % len(ctx), Hq - 1] = True
    assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(l2[~hit], l[~hit])
    pre = [x - 2 if x > 2 else 0 for x in ctx]
    n = sum(x - y for x, y in zip(ctx, pre))
    qe = c.queries(n)
    o, l, _ = _extend(c, pre, qe, False)
    p = qe.clone()
    p[1, 2, 5] = bad
    o2, l2, _ = _extend(c, pre, p, False)
    hit = torch.zeros((n, Hq), dtype=torch.bool, device="cuda")
    hit[1, 2] = True
    assert torch.isnan(o2[hit]).all() and torch.isnan(l2[hit]).all()
    assert torch.equal(o2[~hit], o[~hit]) and torch.equal(l2[~hit], l[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("B", [2, 700])      # few rows and many: both forms of the merge
def test_a_request_without_keys_gets_zeros(d, B):
    """A plan that gives a request no segment (rx_plan_decode itself asks for
    one key at least)."""
    torch = pytest.importorskip("torch")
    c = Case(torch, 8, 2, d, 1, [40, 50], 5)
    info = rx.rx_decode_plan_info()
    info.plan_words, info.workspace_bytes = B + 1, 1024
    plan = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    q = c.queries(B)
    o, l = torch.full((B, 8, d), 5.0, device="cuda"), torch.full((B, 8), 5.0, device="cuda")
    ws = torch.empty(1024, dtype=torch.uint8, device="cuda")
    rx.kv8_decode_attention(c.pool, 1, q, 8, c.up(c.table), plan, info, B, c.scale, o, l, ws)
    assert not o.any() and (l == -float("inf")).all()
    assert rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mag", [0.0, 1e-30, 100.0])
def test_queries_of_any_size(mag):
    """Zeros and vanishing queries: the mean of V.  Large ones: a hard
    maximum, still within the bound."""
    torch = pytest.importorskip("torch")
    c = Case(torch, 16, 4, 128, 8, [77, 300], 6, pow2=True)
    q = c.queries(2, mag)
    qn = q.double().cpu().numpy()
    o, l = _decode(c, q, bf16=False)
    for b in range(2):
        c.compare(o[b:b + 1], l[b:b + 1], c.reference(qn[b:b + 1], b, [c.ctx[b]]), False)
    o, l, _ = _extend(c, [76, 299], q, False)
    for b in range(2):
        c.compare(o[b:b + 1], l[b:b + 1], c.reference(qn[b:b + 1], b, [c.ctx[b]]), False)


@pytest.mark.gpu
@pytest.mark.parametrize("d,block,page", [(128, 1, 1), (256, 16, 16), (128, 64, 64)])
def test_pools_beyond_32_bit_offsets(d, block, page):
    """The last slots of a pool of 4.8 GB a side hold what a small pool
    holds: the same bits from every call."""
    torch = pytest.importorskip("torch")
    H, Hq, T = 3, 12, 320
    big = (1 << 32) // (H * d) // 64 * 64 + (1 << 20)
    outs = []
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((T, H, d), generator=g, device="cuda").to(torch.bfloat16)
            for _ in range(2))
    qd, qe = (torch.randn((n, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
              for n in (1, 150))

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    for N in (512, big):
        assert N % 64 == 0
        kc, vc = (torch.empty((1, H, N, d), dtype=torch.uint8, device="cuda") for _ in range(2))
        sc = torch.empty((1, H, N // block, 2), device="cuda")
        pool = rx.kv8_pool_desc(kc, vc, sc)
        slots = np.arange(N - T, N)
        rx.kv8_store(pool, 0, up(slots), k, v)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        rx.kv8_load(pool, 0, up(slots), kb, vb)
        cache = rx.RadixCache(N, page)
        row = slots.astype(np.int32)
        _, node = cache.insert(np.arange(T, dtype=np.int32), row)
        plan, info = cache.plan_decode([node], [T], [0], Hq, H, d)
        ws = torch.empty(int(info.workspace_bytes), dtype=torch.uint8, device="cuda")
        od, ld = torch.empty((1, Hq, d), device="cuda"), torch.empty((1, Hq), device="cuda")
        rx.kv8_decode_attention(pool, 0, qd, Hq, up(row[None]), up(plan[:int(info.plan_words)]),
                                info, 1, d ** -0.5, od, ld, ws)
        tiles, n = rx.extend_plan(np.array([0, 150]), Hq, H, d)
        oe = torch.empty((150, Hq, d), device="cuda")
        le = torch.empty((150, Hq), device="cuda")
        rx.kv8_extend_attention(pool, 0, qe, Hq, up(row[None]), up([0]), up([T - 150]),
                                up([0, 150]), up(tiles), 1, n, d ** -0.5, oe, le)
        assert rx.device_check() == 0
        outs.append((kb, vb, od, ld, oe, le))
        del kc, vc, sc, pool
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_binding_refuses_other_types_devices_and_layouts():
    torch = pytest.importorskip("torch")
    kc, vc = (torch.zeros((1, 2, 64, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.ones((1, 2, 16, 2), device="cuda")
    pool = rx.kv8_pool_desc(kc, vc, sc)
    s = torch.arange(1, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros((3, 2, 256), dtype=torch.bfloat16, device="cuda")[..., :128]
    for args in ((s.long(), x, x), (s.cpu(), x, x), (s, x.half(), x), (s, x, x.cpu()),
                 (s, x[:2], x), (s, wide, x), (s, x, x.transpose(0, 1))):
        for fn in (rx.kv8_store, rx.kv8_load):
            with pytest.raises(ValueError):
                fn(pool, 0, *args)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    o, l = torch.zeros((1, 4, 128), device="cuda"), torch.zeros((1, 4), device="cuda")
    t = torch.zeros((1, 64), dtype=torch.int32, device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        rx.kv8_extend_attention(pool, 0, q, 4, t, i, i, i, i, 1, 1, 0.1, o.half(), l)
    with pytest.raises(ValueError):
        rx.kv8_extend_attention(pool, 0, q, 4, t, i, i, i, i, 1, 1, 0.1, o, l[:, :3])
    with pytest.raises(ValueError):
        rx.kv8_extend_attention(pool, 0, q, 4, t.float(), i, i, i, i, 1, 1, 0.1, o, l)
    assert not kc.any() and rx.device_check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name,page,block", [("agent", 1, 1), ("agent", 16, 16), ("chat", 16, 8),
                                             ("wide", 1, 1), ("wide", 16, 4), ("alone", 32, 32)])
def test_chained_steps_equal_steps_one_by_one(name, page, block, monkeypatch):
    """rx_kv8_decode_steps overlaps the kernels of consecutive steps: every
    output of a run of steps has the bits of the steps called one at a time
    with a wait between them (shared segments in tiles beside private tails,
    tails in tiles where the group is large, no tiles at all)."""
    torch = pytest.importorskip("torch")
    from radix_tree_prefix_gb300.engine import GatherInputs
    wl = {
        "agent": lambda: workloads.agent_loop(calls=40, preamble=1500, lo=150, hi=250,
                                              decode_steps=48),
        "chat": lambda: workloads.multi_turn_chat(sessions=48, turns=2, system=600, user=60,
                                                  decode_steps=32, layers=1),
        "wide": lambda: workloads.agent_loop(calls=6, preamble=300, lo=20, hi=900,
                                             decode_steps=40, q_heads=64, kv_heads=2),
        "alone": lambda: workloads.agent_loop(calls=2, preamble=0, lo=30, hi=90,
                                              decode_steps=40, head_dim=256),
    }[name]()
    wl = workloads.with_pages(wl, page) if page > 1 else wl
    dev = torch.device("cuda:0")
    vals = workloads.make_values(wl, dev, [0])
    runs = []
    steps = rx.decode_steps

    def one_by_one(pool, layer, hq, d_table, recs, B, scale, ws, stream=None):
        for i in range(len(recs)):
            steps(pool, layer, hq, d_table, recs[i:i + 1], B, scale, ws, stream)
            torch.cuda.synchronize()
    for fn in (one_by_one, steps, steps, steps):
        monkeypatch.setattr(rx, "decode_steps", fn)
        got = {}
        Engine(wl, device=dev, inputs=GatherInputs(wl, vals, [0]), layers=[0], kv8_block=block,
               on_decode_wave=lambda s, rids, ctx, outs, info: got.__setitem__(
                   s, tuple(x.clone() for x in outs[0]))).run()
        torch.cuda.synchronize()
        assert rx.device_check() == 0
        runs.append(got)
    assert runs[0]
    for got in runs[1:]:
        assert got.keys() == runs[0].keys()
        for k in got:
            assert torch.equal(got[k][0], runs[0][k][0]) and torch.equal(got[k][1], runs[0][k][1])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["agent", "wide", "alone"])
def test_chained_steps_in_a_graph(name, monkeypatch):
    """A captured run of steps, replayed, gives the eager run's bits (blocks of
    one slot: storing a token again changes nothing)."""
    torch = pytest.importorskip("torch")
    from radix_tree_prefix_gb300.engine import GatherInputs
    wl = {
        "agent": lambda: workloads.agent_loop(calls=24, preamble=900, lo=50, hi=150,
                                              decode_steps=12),
        "wide": lambda: workloads.agent_loop(calls=4, preamble=300, lo=20, hi=600,
                                             decode_steps=12, q_heads=64, kv_heads=2),
        "alone": lambda: workloads.agent_loop(calls=2, preamble=0, lo=30, hi=90,
                                              decode_steps=12, head_dim=256),
    }[name]()
    dev = torch.device("cuda:0")
    vals = workloads.make_values(wl, dev, [0])
    steps = rx.decode_steps

    def replayed(*args):
        steps(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps(*args[:-1], torch.cuda.current_stream())
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        kept.append(graph)
    runs, kept = [], []
    for fn in (steps, replayed):
        monkeypatch.setattr(rx, "decode_steps", fn)
        got = {}
        Engine(wl, device=dev, inputs=GatherInputs(wl, vals, [0]), layers=[0], kv8_block=1,
               on_decode_wave=lambda s, rids, ctx, outs, info: got.__setitem__(
                   s, tuple(x.clone() for x in outs[0]))).run()
        torch.cuda.synchronize()
        assert rx.device_check() == 0
        runs.append(got)
    assert runs[0] and kept and runs[0].keys() == runs[1].keys()
    for k in runs[0]:
        assert torch.equal(runs[0][k][0], runs[1][k][0])
        assert torch.equal(runs[0][k][1], runs[1][k][1])
