"""The adapters' workspace: one made for the largest batch serves every smaller
one, of fewer tokens, adapters or ranks."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq
from w8a8_int8_quantized_token_gb300 import build_lib


@pytest.fixture(scope="module")
def size():
    build_lib.build()
    return wq.lib().wq_lora_add_workspace_size


@pytest.mark.parametrize("n,r", [(1, 8), (1, 64), (8, 16), (8, 64), (32, 16), (5, 24), (300, 128), (8192, 32)])
def test_more_tokens_never_take_less(size, n, r):
    sizes = [size(T, n, r) for T in range(0, 45000)] + [size(T, n, r) for T in range(45000, 1 << 24, 99991)]
    assert sizes == sorted(sizes) and sizes[256] == 0 and sizes[257] > 0


@pytest.mark.parametrize("T", [257, 300, 577, 1024, 1536, 1537, 1600, 3000, 8831, 8832, 20000, 38912, 50000])
def test_more_adapters_or_ranks_never_take_less(size, T):
    by_n = [[size(T, n, r) for n in range(1, 8193, 13)] for r in (8, 24, 64, 128)]
    by_r = [[size(T, n, r) for r in range(8, 129, 8)] for n in (1, 8, 70, 8192)]
    assert all(s == sorted(s) for s in by_n + by_r)


def z(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("most,T,n,r", [(8832, 8831, 8, 64), (20000, 18559, 8, 64), (20000, 15487, 32, 16), (2000, 500, 3, 64)])
def test_smaller_batches_in_the_largest_ones_workspace(most, T, n, r):
    """Also with fewer adapters, and within the workspace's bounds."""
    H, N, g = 136, 72, torch.Generator().manual_seed(T)
    x, y = torch.randn(T, H, generator=g).bfloat16().cuda(), torch.randn(T, N, generator=g).bfloat16().cuda()
    A, B = (torch.randn(*s, generator=g).mul(0.1).bfloat16().cuda() for s in ((n, r, H), (n, N, r)))
    ids = torch.randint(0, 2, (T,), generator=g).to(torch.int32).cuda()
    need = wq.lora_add_workspace(z(most, N), z(most, H), A).numel()
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for k in (n, 2):
        want, got = y.clone(), y.clone()
        wq.lora_add(want, x, A[:k], B[:k], ids)
        wq.lora_add(got, x, A[:k], B[:k], ids, ws=room[:need])
        assert torch.equal(got, want) and not torch.equal(got, y) and (room[need:] == 0x5A).all()
