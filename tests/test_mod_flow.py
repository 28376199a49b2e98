"""What serves a model's layer around the radix pool, as it is used together:
requests over a shared prompt prefilled batch after batch (the keys normalised,
rotated and stored in the pass that turns the queries, then attention under a
cap, a window and slopes), decoded steps of one window plan, and a draft tree.

The pool's rows are checked against the norm and rotation in 64 bits, the
attention against the formula in 64 bits over the pool's own rows.
"""

import math

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx

from test_rope import freqs, reference
from test_score_mod import _check, _reference


class Layer:
    """Raw projections of token t at position p, the same wherever it occurs."""

    def __init__(self, hq, hkv, d, rot, mod, seed=0, layout="half", eps=1e-6):
        import torch
        self.hq, self.hkv, self.d, self.rot, self.mod, self.eps = hq, hkv, d, rot, mod, eps
        self.layout = layout
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16)
                  for _ in range(2)]
        self.norm = rx.head_norm(*self.w, eps)
        self.rope = rx.rope(rot, layout=layout, scaling="linear", factor=2.0)
        self.table = torch.randn((4096, (hq + 2 * hkv) * d), generator=g,
                                 device="cuda").to(torch.bfloat16)

    def raw(self, tokens):
        """q, k, v side by side as one projection gives them."""
        import torch
        x = self.table[torch.as_tensor(np.asarray(tokens), device="cuda").long() % 4096]
        x = x.view(len(tokens), self.hq + 2 * self.hkv, self.d).clone()
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def turned(self, x, pos, which):
        return reference(x.float().cpu().numpy(), pos, self.d, self.rot, self.layout,
                         dict(scaling="linear", factor=2.0), "weight",
                         self.w[which].float().cpu().numpy(), self.eps)


def _up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Flow:
    def __init__(self, layer, page, n_slots=4096, rows=8, width=1024):
        import torch
        self.y, self.page = layer, page
        self.cache = rx.RadixCache(n_slots, page)
        y = layer
        self.pools = [torch.full((2, y.hkv, n_slots, y.d), float("nan"), dtype=torch.bfloat16,
                                 device="cuda") for _ in range(2)]
        self.pool = rx.pool_desc(*self.pools)
        self.host = np.zeros((rows, width), np.int32)
        self.scale = 1 / math.sqrt(y.d)

    def store(self, tokens, pos, slots):
        """A pass over new tokens; checks what it wrote.  Returns the queries."""
        import torch
        q, k, v = self.y.raw(tokens)
        out = torch.empty((len(tokens), self.y.hq, self.y.d), dtype=torch.bfloat16, device="cuda")
        rx.qkv_store(self.pool, 1, self.y.rope, _up(pos), _up(slots), q, k, v, out, self.y.norm)
        s = _up(slots).long()
        for got, x, which in ((out, q, 0), (self.pools[0][1, :, s].transpose(0, 1), k, 1)):
            want, tol = self.y.turned(x, pos, which)
            assert np.all(np.abs(got.float().cpu().numpy() - want) <= tol)
        assert torch.equal(self.pools[1][1, :, s].transpose(0, 1), v)
        return out

    def check(self, q, out, lse, slots, pos):
        """One request's queries at `pos` over its keys in `slots`."""
        import torch
        m, G = self.y.mod, self.y.hq // self.y.hkv
        s = _up(slots).long()
        p = torch.as_tensor(np.asarray(pos), device="cuda")
        for h in range(self.y.hkv):
            hs = slice(h * G, (h + 1) * G)
            _check(out[:, hs], lse[:, hs], _reference(
                q[:, hs], self.pools[0][1, h, s], self.pools[1][1, h, s], p, self.scale,
                softcap=m["softcap"], window=m["window"], slopes=m["slopes"][hs]))

    def prefill(self, prompts, rows):
        """One extend batch of requests in the rows of the table."""
        import torch
        y, R = self.y, len(prompts)
        ind = np.concatenate([[0], np.cumsum([len(p) for p in prompts])]).astype(np.int64)
        toks = np.concatenate(prompts).astype(np.int32)
        table = np.zeros((R, self.host.shape[1]), np.int32)
        prefix, nodes, new = self.cache.extend_begin(toks, ind, table)
        sfx = [len(p) - int(m) for p, m in zip(prompts, prefix)]
        pos = np.concatenate([np.arange(m, len(p)) for p, m in zip(prompts, prefix)])
        q = self.store(np.concatenate([p[m:] for p, m in zip(prompts, prefix)]), pos, new)
        qo = np.concatenate([[0], np.cumsum(sfx)]).astype(np.int32)
        tiles, nt = rx.extend_plan(qo, y.hq, y.hkv, y.d)
        out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        mod = rx.score_mod(**y.mod)
        rx.extend_attention_mod(self.pool, 1, q, y.hq, _up(table), _up(np.arange(R)), _up(prefix),
                                _up(qo), _up(tiles), R, nt, self.scale, mod, out, lse)
        for r, p in enumerate(prompts):
            a = slice(int(qo[r]), int(qo[r + 1]))
            self.check(q[a], out[a], lse[a], table[r, :len(p)], np.arange(prefix[r], len(p)))
        done, _ = self.cache.extend_end(toks, ind, table, prefix, nodes)
        self.host[rows] = table
        return [int(x) for x in prefix], [int(x) for x in done]


SHAPES = [(8, 2, 128, 128, 1, 50), (8, 2, 128, 64, 16, 200), (16, 4, 256, 256, 16, 33),
          (4, 4, 128, 32, 64, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_requests_prefilled_and_decoded(shape):
    import torch
    hq, hkv, d, rot, page, window = shape
    mod = dict(softcap=20.0, window=window,
               slopes=torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq) * 0.1)
    f = Flow(Layer(hq, hkv, d, rot, mod, seed=d + page), page)
    rng = np.random.default_rng(3)
    common = rng.integers(0, 4000, 150)
    prompts = [np.concatenate([common, 4000 + rng.integers(0, 90, n)])
               for n in (1, 40, 7, 130, 64)]
    pre, nodes = f.prefill(prompts[:1], [0])
    assert pre == [0]
    more, got = f.prefill(prompts[1:], [1, 2, 3, 4])
    assert all(m == 150 // page * page for m in more)
    nodes += got
    # decode: three steps of one plan, a token stored and attended a step
    B, steps = len(prompts), 3
    ctx = np.array([len(p) + 1 for p in prompts], np.int32)
    last = [f.host[b, len(p) - 1] for b, p in enumerate(prompts)]
    slots = f.cache.alloc_decode_steps(ctx - 1, last, steps)
    for t in range(steps):
        f.host[np.arange(B), ctx - 1 + t] = slots[t]
    plan, info = f.cache.plan_decode(nodes, ctx, np.arange(B), hq, hkv, d, n_steps=steps,
                                     window=window)
    dplan, table = _up(plan[:info.plan_words]), _up(f.host)
    ws = torch.full((int(info.workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
    m = rx.score_mod(ctx_len=_up(ctx), **mod)
    for t in range(steps):
        q = f.store(rng.integers(0, 4000, B), ctx - 1 + t, slots[t])
        out = torch.empty((B, hq, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((B, hq), dtype=torch.float32, device="cuda")
        rx.decode_attention_mod(f.pool, 1, q, hq, table, dplan, info, B, f.scale, m, out, lse, ws,
                                step=t)
        for b in range(B):
            n = int(ctx[b]) + t
            f.check(q[b:b + 1], out[b:b + 1], lse[b:b + 1], f.host[b, :n], [n - 1])
    # drafts behind the last step of two requests
    parents, counts = [-1, 0, 0, -1, 0, 1], [3, 3]
    draft_slots = f.cache.alloc(-(-6 // page) * page)[:6] if page == 1 else \
        f.cache.alloc(6 * page)[::page][:6]
    pl = [int(ctx[b]) + steps - 1 for b in (1, 3)]
    rows, dctx, dpos = rx.verify_rows(pl, f.host[[1, 3]], np.concatenate([[0], np.cumsum(counts)]),
                                      parents, draft_slots, f.host.shape[1])
    q = f.store(rng.integers(0, 4000, 6), dpos, draft_slots)
    plan, info = f.cache.plan_decode([nodes[1]] * 3 + [nodes[3]] * 3, dctx, np.arange(6), hq, hkv,
                                     d, window=window)
    ws = torch.full((int(info.workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty((6, hq, d), dtype=torch.float32, device="cuda")
    lse = torch.empty((6, hq), dtype=torch.float32, device="cuda")
    rx.decode_attention_mod(f.pool, 1, q, hq, _up(rows), _up(plan[:info.plan_words]), info, 6,
                            f.scale, rx.score_mod(ctx_len=_up(dctx), **mod), out, lse, ws)
    for i in range(6):
        n = int(dctx[i])
        f.check(q[i:i + 1], out[i:i + 1], lse[i:i + 1], rows[i, :n], [n - 1])
    assert rx.device_check() == 0


@pytest.mark.gpu
def test_a_decode_step_captured_with_its_store():
    """Store and attention of a step in one graph, replayed for new tokens."""
    import torch
    hq, hkv, d = 8, 2, 128
    mod = dict(softcap=30.0, window=64, slopes=torch.full((hq,), 0.01, device="cuda"))
    f = Flow(Layer(hq, hkv, d, d, mod, seed=5, layout="interleaved"), 1)
    rng = np.random.default_rng(8)
    prompts = [rng.integers(0, 4000, n) for n in (90, 33)]
    _, nodes = f.prefill(prompts, [0, 1])
    ctx = np.array([len(p) + 1 for p in prompts], np.int32)
    slots = f.cache.alloc(2)
    f.host[np.arange(2), ctx - 1] = slots
    plan, info = f.cache.plan_decode(nodes, ctx, np.arange(2), hq, hkv, d, window=64)
    dplan, table, dslots, dpos = _up(plan[:info.plan_words]), _up(f.host), _up(slots), _up(ctx - 1)
    ws = torch.empty(int(info.workspace_bytes), dtype=torch.uint8, device="cuda")
    m = rx.score_mod(ctx_len=_up(ctx), **mod)
    tok = torch.zeros(2, dtype=torch.int64, device="cuda")
    q = torch.empty((2, hq, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((2, hq), device="cuda")

    def step():
        x = f.y.table[tok].view(2, hq + 2 * hkv, d)
        rx.qkv_store(f.pool, 1, f.y.rope, dpos, dslots, x[:, :hq], x[:, hq:hq + hkv],
                     x[:, hq + hkv:], q, f.y.norm)
        rx.decode_attention_mod(f.pool, 1, q, hq, table, dplan, info, 2, f.scale, m, out, lse, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for toks in ([5, 77], [3000, 9]):
        tok.copy_(torch.tensor(toks))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(2):
            n = int(ctx[b])
            f.check(q[b:b + 1], out[b:b + 1], lse[b:b + 1], f.host[b, :n], [n - 1])
    assert rx.device_check() == 0


@pytest.mark.gpu
def test_a_pool_beyond_four_gigabytes():
    """Slots whose byte and element offsets pass 32 bits, in the last layer."""
    import torch
    hq, hkv, d, n_slots = 4, 2, 128, 9_000_000
    mod = dict(softcap=0.0, window=0, slopes=torch.zeros(hq, device="cuda"))
    y = Layer(hq, hkv, d, d, mod)
    pools = [torch.empty((2, hkv, n_slots, d), dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    assert pools[0].numel() > 1 << 32
    f = Flow.__new__(Flow)
    f.y, f.pools, f.pool, f.scale = y, pools, rx.pool_desc(*pools), 0.1
    n = 300
    slots = np.concatenate([np.arange(n_slots - 200, n_slots), np.arange(n_slots - 900,
                                                                          n_slots - 800)])
    q = f.store(np.arange(n), np.arange(n), slots)
    table = np.zeros((1, n), np.int32)
    table[0] = slots
    qo = np.array([0, n], np.int32)
    tiles, nt = rx.extend_plan(qo, hq, hkv, d)
    out, lse = torch.empty_like(q), torch.empty((n, hq), device="cuda")
    rx.extend_attention_mod(f.pool, 1, q, hq, _up(table), _up([0]), _up([0]), _up(qo), _up(tiles),
                            1, nt, f.scale, None, out, lse)
    f.check(q, out, lse, slots, np.arange(n))
    cache = rx.RadixCache(n_slots)
    plan, info = cache.plan_decode([0], [n], [0], hq, hkv, d)
    ws = torch.empty(int(info.workspace_bytes), dtype=torch.uint8, device="cuda")
    rx.decode_attention_mod(f.pool, 1, q[-1:].contiguous(), hq, _up(table),
                            _up(plan[:info.plan_words]), info, 1, f.scale, None, out, lse, ws)
    f.check(q[-1:], out[:1], lse[:1], slots, [n - 1])
    assert rx.device_check() == 0
    del pools
    f.pools = None
    torch.cuda.empty_cache()
