"""Elements that no rotation and no norm touches come out bit for bit, whatever they are
and whatever lies beside them."""

import pytest

from radix_tree_prefix_gb300 import rx


def _odd_rows(T, H, d, seed):
    """bf16 [T, H, d] with infinities, NaN (of several payloads), both zeros and the
    smallest numbers strewn in."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = torch.randn((T, H, d), generator=g, device="cuda").to(torch.bfloat16).view(torch.int16)
    odd = torch.tensor([0x7f80, 0xff80, 0x7fc0, 0xffc1, 0x7f81, 0x8000, 0, 1, 0x8001, 0x7f7f],
                       dtype=torch.int32, device="cuda").to(torch.int16)
    at = torch.randint(0, 40, (T, H, d), generator=g, device="cuda")
    return torch.where(at < 10, odd[at.clamp(max=9)], bits).view(torch.bfloat16)


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [None, 0, 2, 34, 64, 100, 126])
@pytest.mark.parametrize("T", [1, 77, 6000])
def test_elements_that_are_not_turned(d, layout, rot, T):
    import torch
    x, k, v = (_odd_rows(T, h, d, s) for h, s in ((5, 1), (2, 2), (2, 3)))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    out, ko = torch.empty_like(x), torch.empty_like(k)
    rope = None if rot is None else rx.rope(rot, layout=layout, magnitude=0.7)
    r = rot or 0
    rx.qk_rope(rope, pos, x, k, out, ko)
    assert torch.equal(_bits(out[..., r:]), _bits(x[..., r:]))
    assert torch.equal(_bits(ko[..., r:]), _bits(k[..., r:]))
    pool = [torch.zeros((1, 2, T + 1, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rx.qkv_store(rx.pool_desc(*pool), 0, rope, pos, torch.arange(1, T + 1, dtype=torch.int32,
                                                                 device="cuda"), x, k, v, out)
    for got, want, n in ((out, x, r), (pool[0][0, :, 1:].transpose(0, 1), k, r),
                         (pool[1][0, :, 1:].transpose(0, 1), v, 0)):
        assert torch.equal(_bits(got[..., n:]), _bits(want[..., n:]))
    # in place, and one side's norm leaves the other side's tail alone
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    kept = k.clone()
    rx.qk_rope(rope, pos, x, k, x, k, rx.head_norm(w, None, 1e-6))
    assert torch.equal(_bits(k[..., r:]), _bits(kept[..., r:]))
    assert rx.device_check() == 0
