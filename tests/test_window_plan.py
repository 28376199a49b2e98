"""A decode plan made for a window says so, and no call that needs its other keys takes it."""

import ctypes as C

import numpy as np
import pytest

from radix_tree_prefix_gb300 import rx
from test_score_mod import _tree

X = 1 << 24


def _info(window=0):
    cache, nodes, ctx, _ = _tree([5, 9], shared=30)
    return cache.plan_decode(nodes, ctx, np.arange(2), 4, 2, 128, window=window)[1]


def test_a_plan_says_its_window():
    assert _info(7).window == 7 and _info(1000).window == 1000
    assert _info().window == 0
    cache, nodes, ctx, _ = _tree([5, 9], shared=30)
    assert cache.plan_decode(nodes, ctx, np.arange(2), 4, 2, 128, n_steps=3)[1].window == 0
    plan = np.zeros(1000, np.int32)
    assert cache.plan_decode(nodes, ctx, np.arange(2), 4, 2, 128, plan=plan, n_steps=3,
                             window=4)[1].window == 4


@pytest.mark.parametrize("window", [0, 8, 2 ** 31 - 1, None])
def test_wider_windows_are_refused(window):
    pool = rx.rx_pool_desc(X, X, 64, 2, 2, 128, 0)
    info = _info(7)
    mod = None if window is None else C.byref(rx.rx_score_mod(0.0, window, None, None, None, X))
    st = rx._lib.rx_decode_attention_mod(C.byref(pool), 0, X, 4, X, 64, X, C.byref(info), 2, 0, 0.1,
                                         mod, X, 0, X, X, 1 << 30, None)
    assert st == rx.RX_ERR_INVALID
    assert "window" in rx.last_error()


def test_calls_without_a_window_refuse_such_a_plan():
    pool = rx.rx_pool_desc(X, X, 64, 2, 2, 128, 0)
    pool8 = rx.rx_kv8_pool_desc(X, X, X, 64, 2, 2, 128, 16)
    info = _info(7)
    steps = (rx.rx_decode_step * 1)(rx.rx_decode_step(X, X, X, X, X, C.addressof(info), X, X, 0, 0))
    p, p8, i = C.byref(pool), C.byref(pool8), C.byref(info)
    for st in (rx._lib.rx_decode_attention(p, 0, X, 4, X, 64, X, i, 2, 0.1, X, X, X, 1 << 30, None),
               rx._lib.rx_decode_attention_static(p, 0, X, 4, X, 64, X, i, 2, 0.1, X, X, None),
               rx._lib.rx_verify_attention(p, 0, X, 4, X, 64, X, i, 2, 0.1, X, X, X, 1 << 30, None),
               rx._lib.rx_decode_steps(p, 0, 4, X, 64, steps, 1, 2, 0.1, X, 1 << 30, None),
               rx._lib.rx_kv8_decode_attention(p8, 0, X, 4, X, 64, X, i, 2, 0, 0.1, X, 0, X, X,
                                               1 << 30, None),
               rx._lib.rx_kv8_decode_steps(p8, 0, 4, X, 64, steps, 1, 2, 0.1, X, 1 << 30, None)):
        assert st == rx.RX_ERR_INVALID
        assert "window" in rx.last_error()
