"""Runs of decode steps over the 8-bit KV pool (rx_kv8_decode_steps), whose
kernels overlap: a run gives the bits of its steps called one at a time, also
where a step reads what the store just before it wrote.
"""

import ctypes as C

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx


def _plan_words(plan, info):
    n = int(info.n_work)
    return np.asarray(plan[int(info.off_work):int(info.off_work) + 8 * n]).reshape(n, 8)


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("Hq,H,d", [(32, 8, 128), (16, 4, 256), (64, 2, 128)])
def test_plans_mark_shared_segments_that_a_step_stores_into(page, Hq, H, d):
    """Word 7 of a work item is 0 only if no step of the plan stores a token in
    the item's segment: a request whose context ends with the shared path has
    its first step's token at that path's end."""
    cache = rx.RadixCache(8192, page)
    slots = np.arange(1, 1 + 2048, dtype=np.int32) + page - 1
    path = np.arange(960, dtype=np.int32)
    mid = cache.insert(path[:640], slots[:640])[1]
    end = cache.insert(path, slots[:960])[1]
    B = 40
    for n_steps in (1, 5):
        # every context ends past the shared path: nothing is stored into it
        plan, info = cache.plan_decode([end] * B, [961 + b for b in range(B)], np.arange(B), Hq, H,
                                       d, n_steps=n_steps)
        w = _plan_words(plan, info)
        assert (w[w[:, 4] > 1, 7] == 0).all() and (w[w[:, 2] > 960, 7] > 960).all()
        # request 3 ends at the path's end, or at the end of its first part
        for node, depth in ((end, 960), (mid, 640)):
            nodes, ctx = [end] * B, [961 + b for b in range(B)]
            nodes[3], ctx[3] = node, depth
            plan, info = cache.plan_decode(nodes, ctx, np.arange(B), Hq, H, d, n_steps=n_steps)
            w = _plan_words(plan, info)
            into = (w[:, 1] < depth) & (depth <= w[:, 2]) & (w[:, 4] > 1)
            assert into.any() and (w[into, 7] == depth).all()
            shared = w[w[:, 4] > 1]
            first = depth if node == mid else 0     # the segment that ends at `depth`
            rest = shared[shared[:, 1] >= first] if node == mid else shared[:0]
            assert (rest[:, 7] == 0).all()
            # the keys of every step are those of before: the whole segment
            for t in range(n_steps):
                ends = np.where(w[into, 7] > 0, np.minimum(w[into, 2], w[into, 7] + t), w[into, 2])
                assert (ends == w[into, 2]).all()
            assert info.tails_private == 0
            assert info.distinct_kv_tokens == 960 + sum(max(0, c - 960) for c in ctx)


class Steps:
    """A pool filled by rx_kv8_store, table rows of given lengths that may share
    their first part with another row, and lists of decode steps over them."""

    def __init__(self, torch, Hq, H, d, block, lens, parent, seed):
        """Row b has lens[b] positions; parent[b] is None or (row, n): its
        first n positions are that row's."""
        self.torch, self.Hq, self.H, self.d, self.block = torch, Hq, H, d, block
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        own = [n - (p[1] if p else 0) for n, p in zip(lens, parent)]
        pages = [-(-n // block) for n in own]
        order = 1 + rng.permutation(sum(pages))
        self.N = (1 + sum(pages)) * block
        self.table = np.zeros((len(lens), max(lens)), dtype=np.int32)
        at = 0
        for b, (n, p) in enumerate(zip(own, parent)):
            if p:
                self.table[b, :p[1]] = self.table[p[0], :p[1]]
            ids = order[at:at + pages[b]]
            at += pages[b]
            s = (ids[:, None] * block + np.arange(block)).reshape(-1)[:n]
            self.table[b, lens[b] - n:lens[b]] = s
        self.start = self.empty_pool()
        pool = self.desc(self.start)
        for b in range(len(lens)):
            s = self.table[b, lens[b] - own[b]:lens[b]]
            if len(s):
                self.store(pool, 0, self.up(s), *self.rows(len(s), H, 0.5))
        self.d_table = self.up(self.table)
        self.keep = []

    store = staticmethod(rx.kv8_store)

    def empty_pool(self):
        torch = self.torch
        return (*(torch.zeros((1, self.H, self.N, self.d), dtype=torch.uint8, device="cuda")
                  for _ in range(2)),
                torch.zeros((1, self.H, self.N // self.block, 2), device="cuda"))

    def desc(self, tensors):
        return rx.kv8_pool_desc(*tensors)

    def up(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def rows(self, n, heads, mag):
        t = self.torch
        return [(t.randn((n, heads, self.d), generator=self.gen, device="cuda") * mag)
                .to(t.bfloat16) for _ in range(2)]

    def plan(self, rows, ctx, depth, n_steps=1):
        """A plan of the given table rows; the first depth[b] positions of a
        row are its cached path (equal slots are equal tokens)."""
        cache = rx.RadixCache(self.N, self.block)
        nodes = [cache.insert(self.table[r, :n], self.table[r, :n])[1]
                 for r, n in zip(rows, depth)]
        plan, info = cache.plan_decode(nodes, ctx, rows, self.Hq, self.H, self.d, n_steps=n_steps)
        d_plan = self.up(plan[:int(info.plan_words)])
        self.keep.append((d_plan, info))
        return d_plan, info, list(rows), list(ctx)

    def entries(self, entries, mag=2.0):
        """Decode steps [(plan, step)], each with new K and V for its tokens."""
        torch, B = self.torch, len(entries[0][0][2])
        rec = np.zeros(len(entries), dtype=rx.DECODE_STEP_DTYPE)
        ins = []
        for i, ((d_plan, info, rows, ctx), t) in enumerate(entries):
            slots = np.array([self.table[r, c + t - 1] for r, c in zip(rows, ctx)])
            assert len(set(slots.tolist())) == B
            q, _ = self.rows(B, self.Hq, 1.0)
            k, v = self.rows(B, self.H, mag)
            ins.append((q, k, v, self.up(slots)))
            rec["d_q"][i], rec["d_k"][i], rec["d_v"][i], rec["d_slots"][i] = (
                x.data_ptr() for x in ins[-1])
            rec["d_plan"][i], rec["info"][i] = d_plan.data_ptr(), C.addressof(info)
            rec["step"][i] = t
        need = max(int(e[0][1].workspace_bytes) for e in entries) + 4 * len(entries)
        self.keep.append(ins)

        def run(one_by_one, graph=False):
            tensors = [x.clone() for x in self.start]
            pool = self.desc(tensors)
            out = torch.full((len(entries), B, self.Hq, self.d), 9.0, device="cuda")
            lse = torch.full((len(entries), B, self.Hq), 9.0, device="cuda")
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            r = rec.copy()
            for i in range(len(entries)):
                r["d_out"][i], r["d_lse"][i] = out[i].data_ptr(), lse[i].data_ptr()
            torch.cuda.synchronize()
            if graph:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    rx.decode_steps(pool, 0, self.Hq, self.d_table, r, B, self.d ** -0.5, ws)
                for _ in range(3):      # (blocks of one slot: a token stored again is the same)
                    out.fill_(9.0)
                    g.replay()
                torch.cuda.synchronize()
            for part in () if graph else [r[i:i + 1] for i in range(len(r))] if one_by_one else [r]:
                rx.decode_steps(pool, 0, self.Hq, self.d_table, part, B, self.d ** -0.5, ws)
                if one_by_one:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            assert rx.device_check() == 0
            return (out, lse, *tensors)
        run.inputs = ins
        return run


def _equal(torch, run, times=8, graph=False):
    want = run(True)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    for i in range(times):
        got = run(False, graph and i == 0)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d", [(64, 2, 128), (32, 2, 256)])
@pytest.mark.parametrize("block", [1, 4])
def test_more_tiles_than_sms_read_the_new_tokens(Hq, H, d, block):
    """Large groups: the tails are tile items too, more of them than the device
    has SMs, so that one follows another on an SM that has read the pool before
    the step's store (slots of the shared path and of the tails mixed, so that
    their scales share sectors)."""
    torch = pytest.importorskip("torch")
    B, depth, steps = 84, 2048, 12
    lens = [depth + steps + 1 + 5 * (b % 7) // block * block for b in range(B)]
    c = Steps(torch, Hq, H, d, block, lens, [None] + [(0, depth)] * (B - 1), 12)
    p = c.plan(range(B), [n - steps + 1 for n in lens], [depth] * B, n_steps=steps)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert p[1].n_work == p[1].n_work_tc and p[1].n_work_tc * H > sms
    _equal(torch, c.entries([(p, t) for t in range(steps)]))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d,block", [(32, 8, 128, 1), (32, 8, 128, 4), (16, 4, 256, 1),
                                          (16, 4, 256, 16)])
@pytest.mark.parametrize("B,depth", [(48, 2048), (12, 4096)])
def test_streams_beside_tiles_read_the_new_tokens(Hq, H, d, block, B, depth):
    """The shared path in tiles, the tails in streams that start beside them:
    every tail holds the token that the store just before wrote."""
    torch = pytest.importorskip("torch")
    steps = 24
    lens = [depth + steps + 1 + 37 * (b % 11) // block * block for b in range(B)]
    c = Steps(torch, Hq, H, d, block, lens, [None] + [(0, depth)] * (B - 1), 13)
    p = c.plan(range(B), [n - steps + 1 for n in lens], [depth] * B, n_steps=steps)
    assert 0 < p[1].n_work_tc < p[1].n_work
    _equal(torch, c.entries([(p, t) for t in range(steps)]))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d", [(32, 8, 128), (16, 4, 256), (64, 2, 128)])
@pytest.mark.parametrize("block", [1, 16])
def test_new_tokens_at_the_end_of_a_shared_segment(Hq, H, d, block):
    """One request of 40 ends with the path that all share, so each step stores
    into a segment that tiles read (its token anew at every step)."""
    torch = pytest.importorskip("torch")
    B, depth = 40, 1024
    lens = [depth] + [depth + 1 + 3 * b for b in range(1, B)]
    c = Steps(torch, Hq, H, d, block, lens, [None] + [(0, depth)] * (B - 1), 11)
    p = c.plan(range(B), lens, [depth] * B)
    assert p[1].n_work_tc > 0
    _equal(torch, c.entries([(p, 0)] * 6), graph=block == 1)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d", [(32, 8, 128), (16, 4, 256), (64, 2, 128)])
@pytest.mark.parametrize("block", [1, 16])
def test_a_plan_over_what_the_plan_before_stored(Hq, H, d, block):
    """A list of two plans: the first one's steps append to a context that the
    second one's requests share, so its tiles read the rows that the entries
    just before stored."""
    torch = pytest.importorskip("torch")
    B, end = 40, 1024
    lens = [end] + [60 + b for b in range(1, B)] + [end + 9 + b for b in range(B)]
    c = Steps(torch, Hq, H, d, block, lens, [None] * B + [(0, end)] * B, 14)
    steps = 4
    first = c.plan(range(B), [n - steps + 1 for n in lens[:B]], [0] * B, n_steps=steps)
    then = c.plan(range(B, 2 * B), [n - 3 for n in lens[B:]], [end] * B, n_steps=3)
    assert then[1].n_work_tc > 0
    _equal(torch, c.entries([(first, t) for t in range(steps)] + [(then, t) for t in range(3)] +
                            [(first, steps - 1), (then, 0)]), graph=block == 1)
