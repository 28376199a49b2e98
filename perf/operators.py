"""Cases of the 8-bit KV cache: storing into it, reading it back, and decode
and extend attention over it.

The cache holds keys and values as e4m3 codes, ``[Hkv, num_slots, d]`` a
layer, with one fp32 scale for each KV head and block of ``block`` consecutive
slots (a K and a V scale side by side, ``[Hkv, num_slots / block, 2]``); a key
is its code times its block's K scale.  The cases take their head counts, head
dimensions and lengths from this package's workloads (an agent loop over a
shared preamble, a multi-turn chat, a batch over one long document).

``own`` chooses between the operators' plain form (elementary torch
operations in 32 bits, rounded once at the end) and the package's calls.
"""

import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
FP8 = torch.float8_e4m3fn


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a chat wave: each of 256 sessions appends a token
        # somewhere inside a page
        dict(name="store_chat_step", op="store", tokens=256, run=1, kv_heads=4, d=256, block=16,
             page=16),
        # the new tokens of an agent loop's calls, token-granular slots
        dict(name="store_agent_calls", op="store", tokens=8017, run=200, kv_heads=8, d=128,
             block=1, page=1),
        # a chat wave's turn: 256 user turns of 200 tokens in pages of 16
        dict(name="store_chat_turn", op="store", tokens=51200, run=200, kv_heads=4, d=256,
             block=16, page=16),
        # a shared system prompt read back (to move it to another pool)
        dict(name="load_system_prompt", op="load", tokens=2000, run=2000, kv_heads=4, d=256,
             block=16, page=16),
        # a long document read back from token-granular slots
        dict(name="load_document", op="load", tokens=32768, run=500, kv_heads=8, d=128, block=1,
             page=1),
        # a single request's token: the latency of the smallest call
        dict(name="decode_one", op="decode", batch=1, shared=0, lo=3201, hi=3201, steps=64,
             q_heads=32, kv_heads=8, d=128, block=1, page=1),
        # a chat wave's step: a shared system prompt and each session's history
        dict(name="decode_chat", op="decode", batch=256, shared=2000, lo=201, hi=1833, steps=32,
             q_heads=16, kv_heads=4, d=256, block=16, page=16),
        # many users over one long document
        dict(name="decode_long_shared", op="decode", batch=64, shared=32768, lo=1025, hi=1152,
             steps=128, q_heads=64, kv_heads=8, d=128, block=1, page=1),
        # long contexts with nothing in common: bound by reading the cache
        dict(name="decode_private", op="decode", batch=32, shared=0, lo=7001, hi=16001, steps=64,
             q_heads=32, kv_heads=8, d=128, block=16, page=16),
        # an agent loop's calls: short suffixes over a shared preamble
        dict(name="extend_agent", op="extend", batch=40, shared=3000, lo=0, hi=0, sfx_lo=150,
             sfx_hi=250, q_heads=32, kv_heads=8, d=128, block=1, page=1),
        # a chat turn: a system prompt, each session's history, 200 new tokens
        dict(name="extend_chat", op="extend", batch=64, shared=2000, lo=0, hi=1624, sfx_lo=200,
             sfx_hi=200, q_heads=16, kv_heads=4, d=256, block=16, page=16),
        # one long prompt with nothing cached, an odd length
        dict(name="extend_prompt", op="extend", batch=1, shared=0, lo=0, hi=0, sfx_lo=8191,
             sfx_hi=8191, q_heads=32, kv_heads=8, d=128, block=64, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: both head dimensions, one to eight query
    heads a KV head, scale blocks of 1 to 64 slots, one token to the longest."""
    op = rng.choice(["store", "load", "decode", "decode", "extend", "extend"])
    block = rng.choice([1, 1, 2, 4, 8, 16, 16, 32, 64])
    page = max(block, rng.choice([1, 16, 64])) if block > 1 else rng.choice([1, 1, 16])
    d = rng.choice([128, 256])
    kv = rng.choice([1, 2, 4, 8]) if d == 128 else rng.choice([1, 2, 4])
    q = kv * rng.choice([1, 2, 4, 4, 8])
    c = dict(op=op, kv_heads=kv, d=d, block=block, page=page)
    if op in ("store", "load"):
        n = _log(rng, 1, 50000)
        return dict(c, tokens=n, run=min(n, _log(rng, 1, 2000)))
    c["q_heads"] = q
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
                sfx_hi=hi_s)


def _spread(lo, hi, n):
    """n lengths between lo and hi, the same for every seed (the work of a
    case follows from its sizes alone)."""
    if hi <= lo:
        return np.full(n, lo, dtype=np.int64)
    i = np.arange(n, dtype=np.int64)
    return lo + (i * 7919 + (hi - lo)) % (hi - lo + 1)


def _lengths(c):
    """(private tokens already in the cache, new tokens) of each request."""
    own_part = _spread(c["lo"], c["hi"], c["batch"])
    if c["op"] == "decode":
        return own_part, np.zeros(c["batch"], dtype=np.int64)
    return own_part, _spread(c["sfx_lo"], c["sfx_hi"], c["batch"])


def work(c):
    H, d = c["kv_heads"], c["d"]
    block = c["block"]
    if c["op"] in ("store", "load"):
        n = c["tokens"]
        scales = 8 * H * (n if c["run"] < block else -(-n // block))
        return {"bytes": n * H * d * 2 * (2 + 1) + scales + 4 * n, "flops": 0}
    priv, sfx = _lengths(c)
    distinct = c["shared"] + int((priv + sfx).sum())
    nq = c["batch"] if c["op"] == "decode" else int(sfx.sum())
    kv = distinct * (2 * H * d + 4) + -(-distinct // block) * H * 8
    qo = nq * c["q_heads"] * (2 * d + 2 * d + 4)
    if c["op"] == "decode":
        pairs = c["batch"] * c["shared"] + int(priv.sum())
    else:
        pairs = int((sfx * (c["shared"] + priv) + sfx * (sfx + 1) // 2).sum())
    return {"bytes": kv + qo, "flops": 4 * d * c["q_heads"] * pairs}


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
    order = rng.permutation(len(lengths))
    at = 1
    for i in order:
        starts[i] = at
        at += lengths[i]
    return [np.arange(s, s + x) for s, x in zip(starts, lengths)], at + 64


def _rows(n, heads, d, gen, dev):
    """bf16 keys or values of n tokens: normal, with the magnitudes of tokens
    and of channels spread."""
    tok = torch.exp(0.4 * torch.randn((n, heads, 1), generator=gen, device=dev))
    chan = torch.exp(0.3 * torch.randn((1, heads, d), generator=gen, device=dev))
    return (torch.randn((n, heads, d), generator=gen, device=dev) * tok * chan).to(torch.bfloat16)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, from -126 on."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp_(min=-126)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _filled_pool(H, slots, d, block, gen, dev):
    """A pool as earlier stores left it: every slot holds some token."""
    pads = -(-slots // block) * block
    codes, scales = [], []
    for _ in range(2):
        c = torch.empty((H, pads, d), dtype=FP8, device=dev)
        s = torch.empty((H, pads // block), dtype=torch.float32, device=dev)
        step = max(block, (1 << 26) // (H * d) // block * block)
        for a in range(0, pads, step):
            b = min(pads, a + step)
            x = _rows(b - a, H, d, gen, dev).permute(1, 0, 2).float()
            x = x.reshape(H, (b - a) // block, block * d)
            sc = _pow2(_exponent(x.abs().amax(dim=2)))
            c[:, a:b] = (x / sc[:, :, None]).reshape(H, b - a, d).to(FP8)
            s[:, a // block:b // block] = sc
        codes.append(c)
        scales.append(s)
    return codes[0], codes[1], torch.stack(scales, dim=2).contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    rng = np.random.Generator(np.random.PCG64(seed))
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    H, d, block, page = c["kv_heads"], c["d"], c["block"], c["page"]
    st = {"op": c["op"], "block": block}

    def up(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)

    if c["op"] in ("store", "load"):
        n, run = c["tokens"], c["run"]
        lens = [run] * (n // run) + ([n % run] if n % run else [])
        # a run of new tokens shorter than a page lands inside one, after the
        # tokens the sequence already has there
        lead = [int(rng.integers(0, page)) if x < page else 0 for x in lens]
        lists, slots = _slots_of_runs([x + y for x, y in zip(lens, lead)], page, rng)
        slot = np.concatenate([s[y:] for s, y in zip(lists, lead)])
        slots = -(-slots // block) * block
        st["slots"] = up(slot)
    else:
        priv, sfx = _lengths(c)
        B, shared = c["batch"], c["shared"]
        # the shared part ends on a page, as in the tree; the rest of it is private
        cut = shared // page * page
        # the tokens decoded so far got their slots step by step: at a page of
        # one slot they lie a batch apart
        tail = np.minimum(priv, c.get("steps", 0)) if page == 1 else np.zeros(B, dtype=np.int64)
        lens = [cut] + [int(x) for x in (shared - cut) + priv + sfx - tail]
        lists, slots = _slots_of_runs(lens, page, rng)
        ctx = shared + priv + sfx
        table = np.zeros((B, int(ctx.max())), dtype=np.int32)
        for b in range(B):
            body = lens[1 + b]
            table[b, :cut] = lists[0]
            table[b, cut:cut + body] = lists[1 + b]
            t = int(tail[b])
            table[b, cut + body:cut + body + t] = slots + np.arange(t) * B + b
        slots += int(tail.max()) * B if page == 1 else 0
        slots = -(-slots // block) * block
        nq = B if c["op"] == "decode" else int(sfx.sum())
        Hq = c["q_heads"]
        st.update(hq=Hq, batch=B, scale=1.0 / math.sqrt(d), table=up(table), ctx=up(ctx),
                  q=torch.randn((nq, Hq, d), generator=gen, device=dev).to(torch.bfloat16),
                  out=torch.empty((nq, Hq, d), dtype=torch.bfloat16, device=dev),
                  lse=torch.empty((nq, Hq), dtype=torch.float32, device=dev))
        if c["op"] == "extend":
            qo = np.concatenate([[0], np.cumsum(sfx)])
            st.update(qo=up(qo), prefix=up(shared + priv), rows=up(np.arange(B)),
                      width=int(sfx.max()))
    st["kc"], st["vc"], st["sc"] = _filled_pool(H, slots, d, block, gen, dev)
    if c["op"] in ("store", "load"):
        shape = (len(slot), H, d)
        if c["op"] == "store":
            st["k"], st["v"] = (_rows(len(slot), H, d, gen, dev) for _ in range(2))
        else:
            st["k"], st["v"] = (torch.empty(shape, dtype=torch.bfloat16, device=dev)
                                for _ in range(2))
    if own:
        # what a serving program keeps: the pool's description, and for a wave
        # of requests its tile schedule or decode plan
        from radix_tree_prefix_gb300 import rx
        st["rx"] = rx
        st["pool"] = rx.kv8_pool_desc(st["kc"][None], st["vc"][None], st["sc"][None])
        if c["op"] == "extend":
            tiles, st["n_tiles"] = rx.extend_plan(qo, c["q_heads"], H, d)
            st["tiles"] = up(tiles)
        if c["op"] == "decode":
            cache = rx.RadixCache(slots // page * page if page > 1 else slots, page)
            nodes = []
            for b in range(B):
                keep = int(ctx[b] - min(int(priv[b]), c["steps"]))
                ids = np.arange(keep, dtype=np.int32)
                ids[cut:] += 100000 * (b + 1)
                nodes.append(cache.insert(ids, table[b, :keep])[1])
            plan, st["info"] = cache.plan_decode(nodes, ctx, np.arange(B), c["q_heads"], H, d)
            st["plan"] = up(plan[:int(st["info"].plan_words)])
            st["ws"] = torch.empty(int(st["info"].workspace_bytes), dtype=torch.uint8, device=dev)
    return st


# ----------------------------------------------------------------- operators
def _plain_store(st):
    """Rows to e4m3 with power-of-two block scales.  A block's scale is the
    least power of two that holds its largest magnitude; a token in a block's
    first slot opens the block, any other keeps the tokens before it, which
    are rounded again if the scale grows."""
    block, slots = st["block"], st["slots"].long()
    blk, off = slots // block, slots % block
    ub, inv = torch.unique(blk, return_inverse=True)
    U = ub.numel()
    first = torch.full((U,), block, dtype=torch.int64, device=slots.device)
    first.scatter_reduce_(0, inv, off, "amin")
    for x, codes, which in ((st["k"], st["kc"], 0), (st["v"], st["vc"], 1)):
        xf = x.float()                                             # [T, H, d]
        H, d = xf.shape[1:]
        amax = torch.zeros((U, H), device=xf.device)
        amax.scatter_reduce_(0, inv[:, None].expand(-1, H), xf.abs().amax(dim=2), "amax")
        new = _pow2(_exponent(amax))                                # [U, H]
        old = st["sc"][:, ub, which].t()                            # [U, H]
        now = torch.where((first == 0)[:, None], new, torch.maximum(old, new))
        if block > 1:
            rows = codes.view(H, -1, block, d)
            kept = rows[:, ub].float()                              # [H, U, block, d]
            again = (kept * (old / now).t()[:, :, None, None]).to(FP8)
            before = torch.arange(block, device=xf.device)[None, :] < first[:, None]
            grew = (now > old).t()[:, :, None] & before[None]
            rows[:, ub] = torch.where(grew[..., None], again.float(), kept).to(FP8)
        codes[:, slots] = (xf / now[inv][:, :, None]).to(FP8).permute(1, 0, 2)
        st["sc"][:, ub, which] = now.t()
    return st["kc"], st["vc"], st["sc"]


def _values(st, which, slots):
    """fp32 keys (0) or values (1) of a tensor of slots: [Hkv, *slots, d]."""
    codes = st["vc" if which else "kc"]
    s = slots.long()
    return codes[:, s].float() * st["sc"][:, s // st["block"], which][..., None]


def _plain_load(st):
    return tuple(_values(st, w, st["slots"]).permute(1, 0, 2).to(torch.bfloat16).contiguous()
                 for w in (0, 1))


def _plain_attention(st, q, lim):
    """q [B, S, Hq, d] over each request's row of the slot table, query (b, s)
    seeing its first lim[b, s] keys: softmax(scale q . k) v, and the log of
    the sum of exponentials."""
    B, S, Hq, d = q.shape
    k, v = (_values(st, w, st["table"]) for w in (0, 1))           # [Hkv, B, N, d]
    H, _, N, _ = k.shape
    G = Hq // H
    qh = q.float().reshape(B, S, H, G, d).permute(2, 0, 1, 3, 4).reshape(H, B, S * G, d)
    s = torch.matmul(qh, k.transpose(2, 3)).view(H, B, S, G, N).mul_(st["scale"])
    hide = torch.arange(N, device=q.device)[None, None, :] >= lim[:, :, None]
    s.masked_fill_(hide[None, :, :, None, :], -math.inf)
    m = s.amax(dim=4, keepdim=True)
    s.sub_(m).exp_()
    l = s.sum(dim=4, keepdim=True)
    o = torch.matmul(s.view(H, B, S * G, N), v).view(H, B, S, G, d) / l
    lse = (m + torch.log(l))[..., 0]
    return (o.permute(1, 2, 0, 3, 4).reshape(B, S, Hq, d),
            lse.permute(1, 2, 0, 3).reshape(B, S, Hq))


def _plain_decode(st):
    o, lse = _plain_attention(st, st["q"][:, None], st["ctx"][:, None].long())
    return o[:, 0].to(torch.bfloat16), lse[:, 0].contiguous()


def _plain_extend(st):
    n = st["q"].shape[0]
    qo, S = st["qo"].long(), st["width"]
    i = torch.arange(S, device=qo.device)
    at = qo[:-1, None] + i[None, :]                                 # query of (request, i)
    real = i[None, :] < (qo[1:] - qo[:-1])[:, None]
    q = st["q"][torch.where(real, at, torch.zeros_like(at))]
    lim = torch.where(real, st["prefix"].long()[:, None] + i[None, :] + 1,
                      torch.ones_like(at))
    o, lse = _plain_attention(st, q, lim)
    return o[real].to(torch.bfloat16).view(n, *o.shape[2:]), lse[real].view(n, -1)


def run(st):
    op = st["op"]
    if not own:
        return {"store": _plain_store, "load": _plain_load, "decode": _plain_decode,
                "extend": _plain_extend}[op](st)
    rx = st["rx"]
    if op == "store":
        rx.kv8_store(st["pool"], 0, st["slots"], st["k"], st["v"])
        return st["kc"], st["vc"], st["sc"]
    if op == "load":
        rx.kv8_load(st["pool"], 0, st["slots"], st["k"], st["v"])
        return st["k"], st["v"]
    if op == "decode":
        rx.kv8_decode_attention(st["pool"], 0, st["q"], st["hq"], st["table"], st["plan"],
                                st["info"], st["batch"], st["scale"], st["out"], st["lse"],
                                st["ws"])
    else:
        rx.kv8_extend_attention(st["pool"], 0, st["q"], st["hq"], st["table"], st["rows"],
                                st["prefix"], st["qo"], st["tiles"], st["batch"], st["n_tiles"],
                                st["scale"], st["out"], st["lse"])
    return st["out"], st["lse"]


# ------------------------------------------------------------ in 64 bits
def _e4m3(x):
    """float64 values rounded to the nearest e4m3 value, ties to even."""
    a = np.abs(x)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    e = np.where(np.ldexp(1.0, e.astype(int)) > a, e - 1, e)
    q = np.ldexp(1.0, np.maximum(e, -6).astype(int) - 3)
    return np.sign(x) * np.minimum(np.rint(a / q) * q, E4M3_MAX)


def _exact_store(st):
    block = st["block"]
    slots = st["slots"].cpu().numpy().astype(np.int64)
    sc = st["sc"].double().cpu().numpy()
    out = []
    ub, inv = np.unique(slots // block, return_inverse=True)
    first = np.full(len(ub), block)
    np.minimum.at(first, inv, slots % block)
    for x, codes, w in ((st["k"], st["kc"], 0), (st["v"], st["vc"], 1)):
        x = x.double().cpu().numpy()
        c = codes.double().cpu().numpy()
        amax = np.zeros((len(ub), x.shape[1]))
        np.maximum.at(amax, inv, np.abs(x).max(axis=2))
        e = np.ceil(np.log2(np.where(amax > 0, amax, 1.0) / E4M3_MAX)).astype(int)
        e = np.where(np.ldexp(E4M3_MAX, e - 1) >= amax, e - 1, e)   # log2 rounds
        e = np.where(np.ldexp(E4M3_MAX, e) < amax, e + 1, e)
        e = np.where(amax > 0, np.maximum(e, -126), -126)
        new = np.ldexp(1.0, e)
        old = sc[:, ub, w].T
        now = np.where((first == 0)[:, None], new, np.maximum(old, new))
        for u in np.nonzero((first > 0) & (now > old).any(axis=1))[0]:
            r = slice(int(ub[u]) * block, int(ub[u]) * block + int(first[u]))
            f = (old[u] / now[u])[:, None, None]
            c[:, r] = np.where(f < 1, _e4m3(c[:, r] * f), c[:, r])
        c[:, slots] = _e4m3(x / now[inv][:, :, None]).transpose(1, 0, 2)
        sc[:, ub, w] = now.T
        out.append(c)
    return out[0], out[1], sc


def exact(c, seed):
    """The definition in 64 bits, request by request."""
    st = prepare(c, seed)
    if c["op"] == "store":
        if st["kc"].numel() > 1 << 25:
            return None                    # minutes of host arithmetic
        return _exact_store(st)
    kd, vd = st["kc"].double(), st["vc"].double()
    kd *= st["sc"][..., 0].double().repeat_interleave(c["block"], 1)[..., None]
    vd *= st["sc"][..., 1].double().repeat_interleave(c["block"], 1)[..., None]
    if c["op"] == "load":
        s = st["slots"].long()
        return kd[:, s].transpose(0, 1).contiguous(), vd[:, s].transpose(0, 1).contiguous()
    Hq, H, d = c["q_heads"], c["kv_heads"], c["d"]
    G = Hq // H
    ctx = st["ctx"].tolist()
    sfx = [1] * c["batch"] if c["op"] == "decode" else _lengths(c)[1].tolist()
    q = st["q"].double()
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    at = 0
    for b in range(c["batch"]):
        n, s = int(ctx[b]), int(sfx[b])
        slot = st["table"][b, :n].long()
        lim = n - s + 1 + torch.arange(s, device=q.device)
        for h in range(H):
            qq = q[at:at + s, h * G:(h + 1) * G]                    # [s, G, d]
            sco = torch.einsum("sgd,nd->sgn", qq, kd[h, slot]) / math.sqrt(d)
            seen = torch.arange(n, device=q.device)[None, :] < lim[:, None]
            sco = torch.where(seen[:, None, :], sco, torch.full_like(sco, -math.inf))
            l = torch.logsumexp(sco, dim=2)
            out[at:at + s, h * G:(h + 1) * G] = torch.exp(sco - l[..., None]) @ vd[h, slot]
            lse[at:at + s, h * G:(h + 1) * G] = l
        at += s
    return out, lse
