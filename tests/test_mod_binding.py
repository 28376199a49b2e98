"""What the binding of attention with modified scores answers to head counts that are none."""

import pytest

from radix_tree_prefix_gb300 import rx


@pytest.mark.parametrize("hq", [0, -4])
def test_no_query_heads_are_refused(hq):
    torch = pytest.importorskip("torch")
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rx.extend_attention_mod(rx.rx_pool_desc(1, 1, 8, 1, 1, 128, 0), 0, q, hq, i.view(1, 4), i,
                                i, i, i, 1, 1, 1.0, rx.score_mod(), q, q)
    with pytest.raises(ValueError):
        rx.decode_attention_mod(rx.rx_pool_desc(1, 1, 8, 1, 1, 128, 0), 0, q, hq, i.view(1, 4), i,
                                rx.rx_decode_plan_info(), 1, 1.0, rx.score_mod(), q, q, q)


@pytest.mark.gpu
def test_no_query_heads_are_an_error_of_the_call():
    import torch
    pool = [torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    lse = torch.zeros(4, device="cuda")
    for hq in (0, -4):
        with pytest.raises((rx.RxError, ValueError)):
            rx.extend_attention_mod(rx.pool_desc(*pool), 0, q, hq, i.view(1, 4), i, i, i, i, 1, 1,
                                    1.0, None, q.clone(), lse)
