"""Runs of decode steps over the bf16 pool (rx_decode_steps): steps of one plan
against softmax attention in 64 bits, and lists of several plans.
"""

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx

from test_kv8_steps import Steps, _equal


class Bf16Steps(Steps):
    store = staticmethod(rx.kv_store)

    def empty_pool(self):
        torch = self.torch
        return tuple(torch.zeros((1, self.H, self.N, self.d), dtype=torch.bfloat16, device="cuda")
                     for _ in range(2))

    def desc(self, tensors):
        return rx.pool_desc(*tensors)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d", [(32, 8, 128), (64, 2, 128), (128, 1, 128), (32, 2, 256)])
@pytest.mark.parametrize("depth,own,steps", [(0, [3, 131, 700], 9), (640, [1, 1, 90, 20], 9),
                                             (0, [1, 100], 700)])
def test_a_step_sees_no_token_of_a_later_step(Hq, H, d, depth, own, steps):
    """Rows of later steps lie in the table and hold anything; groups of more
    than 16 heads (8 at head_dim 256) have their tails in tiles, and a long plan
    has items that no step has reached yet.

    A softmax weight is rounded to bf16 (2^-8 of it), a score carries fp32
    rounding of its d products (2^-20 of the sum of their magnitudes), and the
    weights' sum is taken before or after their rounding (2^-8)."""
    torch = pytest.importorskip("torch")
    B = len(own)
    lens = [depth + n + steps - 1 for n in own]
    c = Bf16Steps(torch, Hq, H, d, 1, lens, [None] + [(0, depth) if depth else None] * (B - 1), 21)
    p = c.plan(range(B), [depth + n for n in own], [depth] * B, n_steps=steps)
    run = c.entries([(p, t) for t in range(steps)], mag=1.0)
    k, v = (x[0].double() for x in c.start)     # the last step's rows are nobody's before it
    out, lse = run(False)[:2]
    for t in range(steps):
        q, kn, vn, slots = run.inputs[t]
        k[:, slots.long()] = kn.double().transpose(0, 1)
        v[:, slots.long()] = vn.double().transpose(0, 1)
        if steps > 20 and t not in (0, 1, 300, steps - 1):
            continue
        for b in range(B):
            ix = torch.from_numpy(c.table[b, :depth + own[b] + t].astype(np.int64)).cuda()
            kk, vv = (x[:, ix].repeat_interleave(Hq // H, 0) for x in (k, v))
            qd = q[b].double()
            s = torch.einsum("hd,hnd->hn", qd, kk) * d ** -0.5
            mag = torch.einsum("hd,hnd->hn", qd.abs(), kk.abs()) * d ** -0.5
            w = s.softmax(-1)
            want = torch.einsum("hn,hnd->hd", w, vv)
            ds = 2 * mag.amax(-1) * 2.0 ** -20 + 2.0 ** -20
            bound = (2.0 ** -7 + ds)[:, None] * torch.einsum("hn,hnd->hd", w, vv.abs())
            assert ((out[t, b].double() - want).abs() <= bound).all(), (t, b)
            assert ((lse[t, b].double() - s.logsumexp(-1)).abs() <= 2.0 ** -8 + ds).all(), (t, b)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H,d", [(32, 8, 128), (16, 4, 256), (64, 2, 128)])
@pytest.mark.parametrize("first_end", [1024, 300])
def test_a_list_of_two_plans(Hq, H, d, first_end):
    """Plans of other sizes in one list, the second one's shared path appended
    to by the first one's steps: the entries called one at a time give the same
    bits."""
    torch = pytest.importorskip("torch")
    B, end, steps = 40, first_end, 4
    lens = [end] + [60 + b for b in range(1, B)] + [end + 9 + b for b in range(B)]
    c = Bf16Steps(torch, Hq, H, d, 1, lens, [None] * B + [(0, end)] * B, 22)
    first = c.plan(range(B), [n - steps + 1 for n in lens[:B]], [0] * B, n_steps=steps)
    then = c.plan(range(B, 2 * B), [n - 3 for n in lens[B:]], [end] * B, n_steps=3)
    assert then[1].n_work_tc > 0 and first[1].n_parts != then[1].n_parts
    _equal(torch, c.entries([(first, t) for t in range(steps)] + [(then, t) for t in range(3)] +
                            [(first, steps - 1), (then, 0)]), graph=True)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [dict(q_heads=64, kv_heads=2),
                                   dict(q_heads=32, kv_heads=2, head_dim=256)])
def test_flow_with_large_groups_matches_the_oracle(heads):
    """The request flow where every tail is a tile: tolerances of the other
    flows' comparisons with the oracle."""
    pytest.importorskip("torch")
    from parity_util import DeviceRun

    from radix_tree_prefix_gb300 import workloads
    wl = workloads.agent_loop(calls=6, preamble=300, lo=20, hi=400, decode_steps=7, **heads)
    DeviceRun(wl, layers=[0], extend_tokens=5).assert_close()
