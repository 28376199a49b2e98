"""Cases of what stands between a model's projections and its logits around
the KV pool: the norm and position rotation of queries and keys, their append
to the pool, and extend and decode attention whose scores are modified (capped
by a tanh, biased by distance, limited to a window, a document or a prefix).

The pool holds bf16 keys and values, ``[Hkv, num_slots, d]`` a layer, and a
request reads it through its row of a slot table.  Head counts, head
dimensions and lengths are those of this package's workloads (an agent loop
over a shared preamble, a multi-turn chat, a batch over one long document).

``own`` chooses between the operators' plain form (elementary torch
operations in 32 bits, angles in 64, rounded once at the end) and the
package's calls.
"""

import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16
INF = math.inf


# --------------------------------------------------------------------- cases
def listed():
    rope = dict(layout="half", base=10000.0, scaling="none", factor=1.0, orig=0, low=0.0,
                high=0.0)
    mod = dict(softcap=0.0, window=0, slopes=False, docs=0, bidir=0)
    return [
        # one request's next token: the latency of the smallest call
        dict(rope, name="rope_one", op="rope", tokens=1, run=1, q_heads=32, kv_heads=8, d=128,
             rot=128, norm="weight", far=4000, fused=False),
        # a long prompt out of one fused projection, a part of each head
        # rotated, positions scaled to a longer context
        dict(rope, name="rope_long_prompt", op="rope", tokens=32767, run=32767, q_heads=32,
             kv_heads=8, d=128, rot=64, norm="none", far=0, fused=True, layout="interleaved",
             scaling="parts", factor=8.0, orig=4096, low=1.0, high=32.0),
        # one decode step of a chat wave: a token each for 256 sessions
        dict(rope, name="store_chat_step", op="store", tokens=256, run=1, q_heads=16, kv_heads=4,
             d=256, rot=256, norm="plus_one", far=4000, fused=False, page=16),
        # the new tokens of an agent loop's calls, far into a scaled context
        dict(rope, name="store_agent_calls", op="store", tokens=8017, run=200, q_heads=32,
             kv_heads=8, d=128, rot=128, norm="none", far=100000, fused=True, page=1,
             base=500000.0, scaling="wavelength", factor=8.0, orig=8192, low=1.0, high=4.0),
        # a chat wave's turn: 256 user turns of 200 tokens in pages of 16
        dict(rope, name="store_chat_turn", op="store", tokens=51200, run=200, q_heads=16,
             kv_heads=4, d=256, rot=256, norm="weight", far=3000, fused=False, page=16),
        # an agent loop's calls: short suffixes over a shared preamble
        dict(mod, name="extend_agent_cap", op="extend", batch=40, shared=3000, lo=0, hi=0,
             sfx_lo=150, sfx_hi=250, q_heads=32, kv_heads=8, d=128, page=1, softcap=50.0),
        # a chat turn whose scores fall with distance
        dict(mod, name="extend_chat_distance", op="extend", batch=64, shared=2000, lo=0, hi=1624,
             sfx_lo=200, sfx_hi=200, q_heads=16, kv_heads=4, d=256, page=16, slopes=True),
        # one long prompt of an odd length in a layer that sees a window
        dict(mod, name="extend_prompt_window", op="extend", batch=1, shared=0, lo=0, hi=0,
             sfx_lo=8191, sfx_hi=8191, q_heads=32, kv_heads=8, d=128, page=64, softcap=30.0,
             window=1024),
        # prompts of several documents each, their instructions seen by all
        # of the tokens both ways
        dict(mod, name="extend_documents", op="extend", batch=5, shared=0, lo=0, hi=0,
             sfx_lo=1500, sfx_hi=2500, q_heads=32, kv_heads=8, d=128, page=1, docs=400,
             bidir=300),
        # a single request's token
        dict(mod, name="decode_one_cap", op="decode", batch=1, shared=0, lo=3201, hi=3201,
             steps=64, q_heads=32, kv_heads=8, d=128, page=1, softcap=50.0),
        # a chat wave's step in a layer that sees a window
        dict(mod, name="decode_chat_window", op="decode", batch=256, shared=2000, lo=201, hi=1833,
             steps=32, q_heads=16, kv_heads=4, d=256, page=16, softcap=50.0, window=1024),
        # many users over one long document, scores that fall with distance
        dict(mod, name="decode_long_distance", op="decode", batch=64, shared=32768, lo=1025,
             hi=1152, steps=128, q_heads=64, kv_heads=8, d=128, page=1, slopes=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: both head dimensions, one to eight query
    heads a KV head, one token to the longest, every rotation and score."""
    op = rng.choice(["rope", "store", "extend", "extend", "decode", "decode"])
    d = rng.choice([128, 256])
    kv = rng.choice([1, 2, 4, 8]) if d == 128 else rng.choice([1, 2, 4])
    q = kv * rng.choice([1, 2, 4, 4, 8])
    if op in ("rope", "store"):
        # at most the elements of the listed chat turn
        n = _log(rng, 1, min(50000, 310000000 // ((q + 2 * kv) * d)))
        scaling = rng.choice(["none", "none", "linear", "base", "parts", "wavelength"])
        c = dict(op=op, tokens=n, run=min(n, _log(rng, 1, 2000)), q_heads=q, kv_heads=kv, d=d,
                 rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                 layout=rng.choice(["half", "interleaved"]),
                 base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                 norm=rng.choice(["none", "weight", "plus_one"]), far=_log(rng, 1, 500000),
                 fused=rng.choice([False, True]),
                 factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), orig=0, low=0.0,
                 high=0.0)
        if scaling == "parts":
            c.update(orig=4096, low=1.0, high=32.0)
        if scaling == "wavelength":
            c.update(orig=8192, low=1.0, high=4.0)
        return dict(c, page=rng.choice([1, 16, 64])) if op == "store" else c
    c = dict(op=op, q_heads=q, kv_heads=kv, d=d, page=rng.choice([1, 1, 16, 64]),
             softcap=rng.choice([0.0, 20.0, 30.0, 50.0]),
             window=rng.choice([0, 0, _log(rng, 1, 8000)]), slopes=rng.random() < 0.35,
             docs=rng.choice([0, 0, _log(rng, 8, 2000)]), bidir=0)
    if not (c["softcap"] or c["window"] or c["slopes"] or c["docs"]):
        c["softcap"] = 50.0
    shared = rng.choice([0, _log(rng, 20, 30000)])
    if op == "decode":
        batch = _log(rng, 1, 256)
        # at most the gathered keys of the listed long document
        top = 2.2e9 / (kv * d * batch)
        shared = min(shared, int(top / 2))
        top = max(2, min(16000, 300000 // batch, int(top / 2)))
        lo = _log(rng, 1, top)
        hi = _log(rng, lo, top) if lo < top else lo
        return dict(c, batch=batch, shared=shared, lo=lo, hi=hi, steps=rng.choice([0, 1, 16, 64]))
    batch = _log(rng, 1, 64)
    hi_s = _log(rng, 1, 8000 // batch)
    lo_s = _log(rng, 1, hi_s)
    # at most the pairs of the listed long prompt
    shared = min(shared, int(3.2e7 * 8 / q / (batch * hi_s)))
    hi = _log(rng, 1, max(1, min(4000, int(3.2e7 * 8 / q / (batch * hi_s)))))
    return dict(c, batch=batch, shared=shared, lo=rng.randint(0, hi), hi=hi, sfx_lo=lo_s,
                sfx_hi=hi_s, bidir=rng.choice([0, _log(rng, 1, 1000)]))


def _spread(lo, hi, n):
    """n lengths between lo and hi, the same for every seed (the work of a
    case follows from its sizes alone)."""
    if hi <= lo:
        return np.full(n, lo, dtype=np.int64)
    i = np.arange(n, dtype=np.int64)
    return lo + (i * 7919 + (hi - lo)) % (hi - lo + 1)


def _lengths(c):
    """(private tokens before the queries, query tokens) of each request; a
    decode request's query is the last of its private tokens."""
    part = _spread(c["lo"], c["hi"], c["batch"])
    if c["op"] == "decode":
        return part - 1, np.ones(c["batch"], dtype=np.int64)
    return part, _spread(c["sfx_lo"], c["sfx_hi"], c["batch"])


def _document_begins(c, n):
    """The first position of the document that each of n positions lies in:
    documents of c["docs"] tokens, give or take half."""
    lens = _spread(max(1, c["docs"] // 2), c["docs"] * 3 // 2 + 1, max(1, 4 * n // c["docs"] + 4))
    ends = np.cumsum(lens)
    begins = np.concatenate([[0], ends])
    return begins[np.searchsorted(ends, np.arange(n), side="right")]


def _limits(c):
    """For each request the positions of its queries, and the first and one
    past the last key that each of them sees (empty when first >= last)."""
    priv, sfx = _lengths(c)
    out = []
    for b in range(c["batch"]):
        pre = c["shared"] + int(priv[b])
        n = pre + int(sfx[b])
        pos = np.arange(pre, n)
        lo = np.zeros(len(pos), dtype=np.int64)
        if c["window"]:
            lo = np.maximum(lo, pos - c["window"] + 1)
        if c["docs"]:
            lo = np.maximum(lo, _document_begins(c, n)[pos])
        out.append((pos, lo, np.maximum(pos + 1, min(c["bidir"], n))))
    return out


def work(c):
    H, d = c["kv_heads"], c["d"]
    if c["op"] in ("rope", "store"):
        n = c["tokens"]
        rows = c["q_heads"] + (2 if c["op"] == "store" else 1) * H
        return {"bytes": n * rows * d * 4 + (8 if c["op"] == "store" else 4) * n,
                "flops": 6 * n * (c["q_heads"] + H) * d}
    lim = _limits(c)
    shared, first, keys, pairs, nq = c["shared"], c["shared"], 0, 0, 0
    for pos, lo, hi in lim:
        pairs += int(np.maximum(hi - lo, 0).sum())
        nq += len(pos)
        seen = lo < hi
        if seen.any():
            # (the keys between two documents' are some query's own)
            a, e = int(lo[seen].min()), int(hi[seen].max())
            first = min(first, a)
            keys += max(0, e - max(a, shared))
    keys += shared - first
    return {"bytes": keys * (2 * H * d * 2 + 4) + nq * c["q_heads"] * (4 * d + 4),
            "flops": 4 * d * c["q_heads"] * pairs}


# -------------------------------------------------------------------- inputs
def _slots_of_runs(lengths, page, rng):
    """A slot list for each length, as the cache hands them out: whole pages,
    a request's positions in slot order within a page, the pages of the pool
    in an order that evictions and reuse have shuffled (for pages of one slot
    the runs are shuffled whole).  Page 0 is the pad page.  Returns the lists
    and the pool's slots."""
    lengths = [int(x) for x in lengths]
    if page > 1:
        n_pages = [-(-x // page) for x in lengths]
        total = sum(n_pages) + 3
        order = 1 + rng.permutation(total - 1)
        out, at = [], 0
        for x, p in zip(lengths, n_pages):
            ids = order[at:at + p]
            at += p
            out.append((ids[:, None] * page + np.arange(page)[None, :]).reshape(-1)[:x])
        return out, total * page
    starts = np.zeros(len(lengths), dtype=np.int64)
    at = 1
    for i in rng.permutation(len(lengths)):
        starts[i] = at
        at += lengths[i]
    return [np.arange(s, s + x) for s, x in zip(starts, lengths)], at + 64


def _rows(n, heads, d, gen, dev):
    """bf16 rows of n tokens: normal, with the magnitudes of tokens and of
    channels spread."""
    tok = torch.exp(0.4 * torch.randn((n, heads, 1), generator=gen, device=dev))
    chan = torch.exp(0.3 * torch.randn((1, heads, d), generator=gen, device=dev))
    return (torch.randn((n, heads, d), generator=gen, device=dev) * tok * chan).to(BF16)


def _pool(H, slots, d, gen, dev):
    """A pool's keys or values as earlier steps left them."""
    out = torch.empty((H, slots, d), dtype=BF16, device=dev)
    step = max(1, (1 << 26) // (H * d))
    for a in range(0, slots, step):
        b = min(slots, a + step)
        out[:, a:b] = _rows(b - a, H, d, gen, dev).permute(1, 0, 2)
    return out


def _up(a, dev, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(dev)


def _prepare_rope(c, st, rng, gen, dev):
    n, Hq, H, d = c["tokens"], c["q_heads"], c["kv_heads"], c["d"]
    lens = [c["run"]] * (n // c["run"]) + ([n % c["run"]] if n % c["run"] else [])
    pos = [int(rng.integers(0, c["far"] + 1)) + np.arange(x) for x in lens]
    st.update(d=d, rot=c["rot"], layout=c["layout"], pos=_up(np.concatenate(pos), dev), eps=1e-6,
              norm=c["norm"], rope=dict((k, c[k]) for k in ("rot", "base", "scaling", "factor",
                                                            "orig", "low", "high")))
    if c["norm"] != "none":
        off = 0.0 if c["norm"] == "plus_one" else 1.0
        st["qw"], st["kw"] = ((off + 0.2 * torch.randn(d, generator=gen, device=dev)).to(BF16)
                              for _ in range(2))
    if c["fused"]:  # q, k and v side by side, as one projection writes them
        x = _rows(n, Hq + 2 * H, d, gen, dev)
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    else:
        st["q"], st["k"], st["v"] = (_rows(n, h, d, gen, dev) for h in (Hq, H, H))
    st["q_out"] = torch.empty((n, Hq, d), dtype=BF16, device=dev)
    if c["op"] == "rope":
        st["k_out"] = torch.empty((n, H, d), dtype=BF16, device=dev)
        return
    # a run of new tokens shorter than a page lands inside one
    page = c["page"]
    lead = [int(rng.integers(0, page)) if x < page else 0 for x in lens]
    lists, slots = _slots_of_runs([x + y for x, y in zip(lens, lead)], page, rng)
    st["slots"] = _up(np.concatenate([s[y:] for s, y in zip(lists, lead)]), dev)
    st["kp"], st["vp"] = (_pool(H, slots, d, gen, dev) for _ in range(2))


def _prepare_attention(c, st, rng, gen, dev):
    Hq, H, d, page = c["q_heads"], c["kv_heads"], c["d"], c["page"]
    priv, sfx = _lengths(c)
    B, shared = c["batch"], c["shared"]
    # the shared part ends on a page, as in the tree; the rest of it is private
    cut = shared // page * page
    # the tokens decoded so far got their slots step by step: at a page of
    # one slot they lie a batch apart
    tail = np.zeros(B, dtype=np.int64)
    if c["op"] == "decode" and page == 1:
        tail = np.minimum(priv + 1, c["steps"])
    lens = [cut] + [int(x) for x in (shared - cut) + priv + sfx - tail]
    lists, slots = _slots_of_runs(lens, page, rng)
    ctx = shared + priv + sfx
    table = np.zeros((B, int(ctx.max())), dtype=np.int32)
    for b in range(B):
        t = int(tail[b])
        table[b, :cut] = lists[0]
        table[b, cut:cut + lens[1 + b]] = lists[1 + b]
        table[b, cut + lens[1 + b]:ctx[b]] = slots + np.arange(t) * B + b
    slots += int(tail.max()) * B
    lim = _limits(c)
    nq = int(sfx.sum())
    # queries of several magnitudes: scores from near zero to the cap's bend
    q = 1.5 * _rows(nq, Hq, d, gen, dev).float()
    st.update(hq=Hq, batch=B, scale=1.0 / math.sqrt(d), table=_up(table, dev), ctx=_up(ctx, dev),
              q=q.to(BF16), softcap=c["softcap"], window=c["window"], slopes=None,
              key_begin=None, bidir_end=None,
              out=torch.empty((nq, Hq, d), dtype=BF16, device=dev),
              lse=torch.empty((nq, Hq), dtype=torch.float32, device=dev))
    if c["slopes"]:  # 2^(-8 (h + 1) / Hq), the usual geometric row
        st["slopes"] = torch.exp2(-8.0 / Hq * torch.arange(1, Hq + 1, device=dev)).float()
    if c["docs"]:
        st["key_begin"] = _up(np.concatenate([_document_begins(c, int(x[0][-1]) + 1)[x[0]]
                                              for x in lim]), dev)
    if c["bidir"]:
        st["bidir_end"] = _up(np.minimum(c["bidir"], ctx), dev)
    qo = np.concatenate([[0], np.cumsum(sfx)])
    st.update(qo=_up(qo, dev), prefix=_up(shared + priv, dev), rows=_up(np.arange(B), dev),
              width=int(sfx.max()))
    st["kp"], st["vp"] = (_pool(H, slots, d, gen, dev) for _ in range(2))
    if not own:
        return
    # what a serving program keeps: a wave's tile schedule or decode plan
    from radix_tree_prefix_gb300 import rx
    st["mod"] = rx.score_mod(softcap=st["softcap"], window=st["window"], slopes=st["slopes"],
                             key_begin=st["key_begin"], bidir_end=st["bidir_end"],
                             ctx_len=st["ctx"] if c["op"] == "decode" else None)
    if c["op"] == "extend":
        tiles, st["n_tiles"] = rx.extend_plan(qo, Hq, H, d)
        st["tiles"] = _up(tiles, dev)
        return
    cache = rx.RadixCache(slots // page * page, page)
    nodes = []
    for b in range(B):
        keep = int(ctx[b] - min(int(priv[b]) + 1, c["steps"]))
        ids = np.arange(keep, dtype=np.int32)
        ids[cut:] += 100000 * (b + 1)
        nodes.append(cache.insert(ids, table[b, :keep])[1])
    plan, st["info"] = cache.plan_decode(nodes, ctx, np.arange(B), Hq, H, d, window=c["window"])
    st["plan"] = _up(plan[:int(st["info"].plan_words)], dev)
    st["ws"] = torch.empty(int(st["info"].workspace_bytes), dtype=torch.uint8, device=dev)


def prepare(c, seed):
    dev = torch.device("cuda")
    rng = np.random.Generator(np.random.PCG64(seed))
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = {"op": c["op"]}
    make = _prepare_rope if c["op"] in ("rope", "store") else _prepare_attention
    make(c, st, rng, gen, dev)
    if own:
        from radix_tree_prefix_gb300 import rx
        st["rx"] = rx
        if "kp" in st:
            st["pool"] = rx.pool_desc(st["kp"][None], st["vp"][None])
        if "rope" in st:
            r = st["rope"]
            st["turn"] = rx.rope(r["rot"], base=r["base"], layout=st["layout"],
                                 scaling=r["scaling"], factor=r["factor"],
                                 original_len=r["orig"], low=r["low"], high=r["high"])
            st["hn"] = None if st["norm"] == "none" else rx.head_norm(
                st["qw"], st["kw"], st["eps"], plus_one=st["norm"] == "plus_one")
    return st


# ----------------------------------------------------------------- operators
def _frequencies(r):
    """(angle a position of each pair in 64 bits, factor on cos and sin)."""
    rot, base, s = r["rot"], r["base"], r["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if r["scaling"] == "base" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if r["scaling"] == "linear":
        return f / s, 1.0
    if r["scaling"] == "parts":
        # a ramp over the pairs between those that turn `high` and `low`
        # times over the original length, kept above it and divided below it
        def pair(turns):
            return rot * math.log(r["orig"] / (turns * 2 * math.pi)) / (2 * math.log(base))
        a = max(0, math.floor(pair(r["high"])))
        b = min(rot - 1, math.ceil(pair(r["low"])))
        ramp = ((i - a) / max(b - a, 0.001)).clamp(0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    if r["scaling"] == "wavelength":
        turns = r["orig"] * f / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        return f / s * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _plain_rotated(st, x, w):
    """x [T, H, d] with its heads normalised and its pairs rotated, in fp32."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(dim=2, keepdim=True) + st["eps"])
        y = y * (w.float() + 1.0 if st["norm"] == "plus_one" else w.float())
    rot = st["rot"]
    f, m = _frequencies(st["rope"])
    t = st["pos"].double()[:, None] * f.to(x.device)[None, :]
    cos, sin = ((g * m).float()[:, None, :] for g in (torch.cos(t), torch.sin(t)))
    if st["layout"] == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=2)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=3).flatten(2)
    return torch.cat([turned, y[..., rot:]], dim=2).to(BF16)


def _plain_rope(st):
    return (_plain_rotated(st, st["q"], st.get("qw")), _plain_rotated(st, st["k"], st.get("kw")))


def _plain_store(st):
    q, k = _plain_rope(st)
    s = st["slots"].long()
    st["kp"][:, s] = k.permute(1, 0, 2)
    st["vp"][:, s] = st["v"].permute(1, 0, 2)
    return q, st["kp"], st["vp"]


def _plain_attention(st):
    """Each request's queries, padded to the longest, over its row of the slot
    table: softmax(score) v and the log of the sum of exponentials."""
    qo, S, G = st["qo"].long(), st["width"], st["hq"] // st["kp"].shape[0]
    dev = qo.device
    i = torch.arange(S, device=dev)
    real = i[None, :] < (qo[1:] - qo[:-1])[:, None]                  # [B, S]
    at = torch.where(real, qo[:-1, None] + i[None, :], torch.zeros_like(i)[None, :])
    q = st["q"][at]                                                 # [B, S, Hq, d]
    pos = st["prefix"].long()[:, None] + i[None, :]
    slot = st["table"].long()
    k, v = st["kp"][:, slot].float(), st["vp"][:, slot].float()     # [H, B, N, d]
    H, B, N, d = k.shape
    j = torch.arange(N, device=dev)
    s = torch.matmul(q.float().reshape(B, S, H, G, d).permute(2, 0, 1, 3, 4).reshape(H, B, S * G, d),
                     k.transpose(2, 3)).view(H, B, S, G, N).mul_(st["scale"])
    if st["softcap"]:
        s.div_(st["softcap"]).tanh_().mul_(st["softcap"])
    away = pos[:, :, None] - j                                      # [B, S, N]
    if st["slopes"] is not None:
        s.sub_(st["slopes"].view(H, 1, 1, G, 1) * away.abs()[None, :, :, None, :].float())
    seen = away >= 0
    if st["bidir_end"] is not None:
        seen |= j[None, None, :] < st["bidir_end"].long()[:, None, None]
    if st["window"]:
        seen &= away < st["window"]
    if st["key_begin"] is not None:
        seen &= j >= st["key_begin"].long()[at][:, :, None]
    # past a request's own tokens the table holds no keys of it
    seen &= j[None, None, :] < st["ctx"].long()[:, None, None]
    s.masked_fill_(~seen[None, :, :, None, :], -INF)
    m = s.amax(dim=4, keepdim=True).clamp_(min=-1e30)
    s.sub_(m).exp_()
    l = s.sum(dim=4, keepdim=True)
    o = torch.matmul(s.view(H, B, S * G, N), v).view(H, B, S, G, d) / l.clamp(min=1e-30)
    lse = (m + torch.log(l))[..., 0]
    return (o.permute(1, 2, 0, 3, 4).reshape(B, S, H * G, d)[real].to(BF16),
            lse.permute(1, 2, 0, 3).reshape(B, S, H * G)[real])


def run(st):
    op = st["op"]
    if not own:
        return {"rope": _plain_rope, "store": _plain_store}.get(op, _plain_attention)(st)
    rx = st["rx"]
    if op == "rope":
        rx.qk_rope(st["turn"], st["pos"], st["q"], st["k"], st["q_out"], st["k_out"], st["hn"])
        return st["q_out"], st["k_out"]
    if op == "store":
        rx.qkv_store(st["pool"], 0, st["turn"], st["pos"], st["slots"], st["q"], st["k"], st["v"],
                     st["q_out"], st["hn"])
        return st["q_out"], st["kp"], st["vp"]
    if op == "extend":
        rx.extend_attention_mod(st["pool"], 0, st["q"], st["hq"], st["table"], st["rows"],
                                st["prefix"], st["qo"], st["tiles"], st["batch"], st["n_tiles"],
                                st["scale"], st["mod"], st["out"], st["lse"])
    else:
        rx.decode_attention_mod(st["pool"], 0, st["q"], st["hq"], st["table"], st["plan"],
                                st["info"], st["batch"], st["scale"], st["mod"], st["out"],
                                st["lse"], st["ws"])
    return st["out"], st["lse"]


# ------------------------------------------------------------ in 64 bits
def _exact_angles(r):
    """Pair by pair, the angle of one position, and the magnitude."""
    out = []
    rot, s, two_pi = r["rot"], r["factor"], 2 * math.pi
    b = r["base"]
    if r["scaling"] == "base" and rot > 2:
        b = math.exp(math.log(b) + rot / (rot - 2) * math.log(s))
    for i in range(rot // 2):
        f = math.exp(-(2 * i / rot) * math.log(b))
        if r["scaling"] == "linear":
            f /= s
        elif r["scaling"] == "wavelength":
            wave = two_pi / f
            if wave > r["orig"] / r["low"]:
                f /= s
            elif wave >= r["orig"] / r["high"]:
                w = (r["orig"] / wave - r["low"]) / (r["high"] - r["low"])
                f = w * f + (1 - w) * f / s
        elif r["scaling"] == "parts":
            first, last = (math.log(r["orig"] / two_pi / n) / math.log(b) * rot / 2
                           for n in (r["high"], r["low"]))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
            w = min(1.0, max(0.0, (i - first) / (last - first if last > first else 0.001)))
            f = f * (1 - w + w / s)
        out.append(f)
    return out, 1 + math.log(s) / 10 if r["scaling"] == "parts" else 1.0


def _exact_rotated(st, x, w):
    y = x.double()
    if w is not None:
        g = w.double() + (1 if st["norm"] == "plus_one" else 0)
        y = y / torch.sqrt(torch.mean(y * y, 2, True) + st["eps"]) * g
    f, m = _exact_angles(st["rope"])
    z = y.clone()
    p = st["pos"].double()
    for i, w in enumerate(f):
        a, b = (i, i + st["rot"] // 2) if st["layout"] == "half" else (2 * i, 2 * i + 1)
        turn = torch.polar(torch.full_like(p, m), p * w)[:, None]
        both = torch.complex(y[..., a], y[..., b]) * turn
        z[..., a], z[..., b] = both.real, both.imag
    return z


def exact(c, seed):
    """The definition in 64 bits, pair by pair and request by request."""
    st = prepare(c, seed)
    if c["op"] in ("rope", "store"):
        q = _exact_rotated(st, st["q"], st.get("qw"))
        k = _exact_rotated(st, st["k"], st.get("kw"))
        if c["op"] == "rope":
            return q, k
        kp, vp = st["kp"].double(), st["vp"].double()
        s = st["slots"].long()
        for h in range(c["kv_heads"]):
            kp[h].index_copy_(0, s, k[:, h])
            vp[h].index_copy_(0, s, st["v"][:, h].double())
        return q, kp, vp
    H, d = c["kv_heads"], c["d"]
    G = c["q_heads"] // H
    q = st["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -INF, dtype=torch.float64, device=q.device)
    at = 0
    for b, (pos, lo, hi) in enumerate(_limits(c)):
        n, s = int(pos[-1]) + 1, len(pos)
        slot = st["table"][b, :n].long()
        p, lo, hi = (torch.from_numpy(x).to(q.device)[:, None, None] for x in (pos, lo, hi))
        j = torch.arange(n, device=q.device)[None, None, :]
        for h in range(H):
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("sgd,nd->sgn", q[at:at + s, heads], st["kp"][h, slot].double())
            x /= math.sqrt(d)
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if c["slopes"]:
                x -= st["slopes"][heads].double()[None, :, None] * (p - j).abs()
            x = torch.where((j >= lo) & (j < hi), x, torch.full_like(x, -INF))
            l = torch.logsumexp(x, dim=2)
            lse[at:at + s, heads] = l
            some = torch.isfinite(l)[..., None]
            wt = torch.where(some, torch.exp(x - torch.where(some, l[..., None], 0.0)), 0.0)
            out[at:at + s, heads] = wt @ st["vp"][h, slot].double()
        at += s
    return out, lse
