"""Offsets past 2^31 elements: caches, weights and adapters where a 32-bit offset
would reach other elements.  Each call is compared with the same one on tensors
of the size that it needs."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HKV, D = 4, 128


def randn(*shape, seed=0, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def in_large(c):
    """The pages of c behind others, past 2^31 elements."""
    per = c[0].numel()
    ahead = 2 ** 31 // per + 3
    big = torch.empty(ahead + len(c), *c.shape[1:], dtype=c.dtype, device="cuda")
    big[ahead:] = c
    return big, ahead


def far_rows(t, pitch):
    """A copy of t whose first dimension has this pitch."""
    big = torch.empty((t.shape[0] - 1) * pitch + t[0].numel(), dtype=t.dtype, device="cuda")
    v = big.as_strided(t.shape, (pitch, *t.stride()[1:]))
    v.copy_(t)
    return v


@pytest.mark.parametrize("q,page", [(1, 64), (150, 64), (3, 12)])
def test_weights(q, page):
    B, L = 2, 600
    ns = -(-L // page)
    k, n = randn(B * ns, HKV, page, D), torch.tensor([L, 431], dtype=torch.int32).cuda()
    pt = torch.randperm(B * ns, generator=torch.Generator().manual_seed(1)).to(torch.int32).reshape(B, ns).cuda()
    a = dict(q=randn(B * q, 8, D, seed=2), key_len=n, max_len=L, lse=torch.full((B * q, 8), 5.0).cuda())
    w = torch.rand(B, HKV, L, generator=torch.Generator().manual_seed(3)).cuda()
    want = wq.attention_weights_paged(k_cache=k, page_table=pt, weights=w.clone(), **a)
    big, ahead = in_large(k)
    st = wq.new_status()
    got = wq.attention_weights_paged(k_cache=big, page_table=pt + ahead, weights=far_rows(w, 2 ** 31 + 8), status=st, **a)
    assert int(st) == 0
    for b, m in enumerate(n.tolist()):
        assert torch.equal(got[b, :, :m], want[b, :, :m])


@pytest.mark.parametrize("apart", [False, True])
def test_eviction(apart):
    B, L, page, budget = 2, 600, 64, 200
    ns, no = -(-L // page), -(-budget // page)
    k, v = randn(B * (ns + no), HKV, page, D, seed=1), randn(B * (ns + no), HKV, page, D, seed=2)
    pages = torch.randperm(B * (ns + no), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    pt, out = pages[:B * ns].reshape(B, ns), pages[B * ns:].reshape(B, no) if apart else None
    n, w = torch.tensor([L, 431], dtype=torch.int32).cuda(), torch.rand(B, HKV, L, generator=torch.Generator().manual_seed(3)).cuda()
    (bk, ahead), (bv, _), bw = in_large(k), in_large(v), far_rows(w, 2 ** 31 + 8)
    a, st = dict(key_len=n, max_len=L, budget=budget, recent=20, first=2), wq.new_status()
    want = wq.evict_paged(w, k, v, pt, out_table=out, **a)
    got = wq.evict_paged(bw, bk, bv, pt + ahead, out_table=out + ahead if apart else None, status=st, **a)
    assert int(st) == 0 and all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(bk[ahead:], k) and torch.equal(bv[ahead:], v) and torch.equal(bw[..., :budget], w[..., :budget])


@pytest.mark.parametrize("T", [40, 400, 2200])
def test_adapters(T):
    H, N, r, n = 2056, 136, 64, 3
    A, B = randn(n, r, H, seed=1) * H ** -0.5, randn(n, N, r, seed=2) * r ** -0.5
    x, y = randn(T, H, seed=3), randn(T, N, seed=4)
    ids = torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    pitch = (2 ** 31 // (T - 1) + 64) // 8 * 8
    far = far_rows(y, max(pitch, N))
    wq.lora_add(y, x, A, B, ids)
    st = wq.new_status()
    wq.lora_add(far, far_rows(x, max(pitch, H)), A, B, ids, status=st)
    assert int(st) == 0 and torch.equal(far, y)


@pytest.mark.parametrize("T", [40, 400, 2200])
def test_many_adapters(T):
    """Which numbers the tokens' adapters have changes nothing."""
    H, N, r, n = 2056, 2056, 128, 8192
    assert n * r * H > 2 ** 31
    A0, B0 = randn(4, r, H, seed=1) * H ** -0.5, randn(4, N, r, seed=2) * r ** -0.5
    ids = torch.randint(-1, 4, (T,), generator=torch.Generator().manual_seed(5))
    x, y = randn(T, H, seed=3), randn(T, N, seed=4)
    got, st = [], wq.new_status()
    for numbers in ([0, 1, 2, 3], [0, 4001, 8190, 8191]):
        at = torch.tensor(numbers)
        A, B = torch.zeros(n, r, H, dtype=BF, device="cuda"), torch.zeros(n, N, r, dtype=BF, device="cuda")
        A[at.cuda()], B[at.cuda()] = A0, B0
        of = at[ids.clamp(min=0)].where(ids >= 0, -1).to(torch.int32).cuda()
        got.append(wq.lora_add(y.clone(), x, A, B, of, status=st))
    assert int(st) == 0 and torch.equal(got[0], got[1]) and not torch.equal(got[0], y)
