"""An 8-bit pool's memory is free as soon as nobody holds its descriptor."""

import gc
import weakref

import pytest

from radix_tree_prefix_gb300 import rx


def _released(torch, device):
    kc, vc = (torch.zeros((1, 2, 64, 128), dtype=torch.uint8, device=device) for _ in range(2))
    sc = torch.ones((1, 2, 16, 2), device=device)
    pool = rx.kv8_pool_desc(kc, vc, sc)
    refs = [weakref.ref(x) for x in (pool, kc, vc, sc)]
    if device != "cpu":
        s = torch.arange(1, 4, dtype=torch.int32, device=device)
        x = torch.ones((3, 2, 128), dtype=torch.bfloat16, device=device)
        rx.kv8_store(pool, 0, s, x, x)
        rx.kv8_load(pool, 0, s, x.clone(), x.clone())
        torch.cuda.synchronize()
    del kc, vc, sc
    assert all(r() is not None for r in refs)    # the descriptor keeps its tensors
    del pool
    return [r() is None for r in refs]


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_a_dropped_descriptor_frees_its_tensors(device):
    torch = pytest.importorskip("torch")
    on = gc.isenabled()
    gc.disable()
    try:
        assert all(_released(torch, device))
    finally:
        if on:
            gc.enable()
