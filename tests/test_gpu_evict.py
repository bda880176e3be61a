"""Eviction from a paged cache on the GPU against a plain definition; which keys
stay, and what moves, is exact."""
import math

import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def rng(seed):
    return torch.Generator().manual_seed(seed)


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def chosen(w, n, budget, recent, first):
    """Places that stay of n keys with weights w (a list)."""
    if n <= budget:
        return list(range(n))
    value = [-math.inf if math.isnan(x) else x for x in w[:n]]
    nan = [math.isnan(x) for x in w[:n]]
    mid = sorted(range(first, n - recent), key=lambda i: (nan[i], -value[i], i))
    return sorted(list(range(first)) + mid[:budget - first - recent] + list(range(n - recent, n)))


def problem(lens, Hkv, dk, dv, page, dtype, budget, apart, token_major=False, seed=0, weights=None):
    B, ns, no = len(lens), -(-max(max(lens), 1) // page), -(-budget // page)
    pages = B * (ns + no) + 1
    order = torch.randperm(pages, generator=rng(seed)).to(torch.int32)

    def cache(d, s):
        c = torch.randn(pages, page, Hkv, d, generator=rng(s)).to(dtype).cuda()
        return c.transpose(1, 2) if token_major else c.transpose(1, 2).contiguous()

    w = torch.randn(B, Hkv, max(lens) + 3, generator=rng(seed + 1)).exp()
    w = w if weights is None else weights(w)
    out = order[B * ns:B * (ns + no)].reshape(B, no).contiguous().cuda() if apart else None
    return dict(weights=w.cuda(), k_cache=cache(dk, 5), v_cache=cache(dv, 6),
                page_table=order[:B * ns].reshape(B, ns).contiguous().cuda(), key_len=i32(lens), max_len=max(lens),
                budget=budget, out_table=out)


def check(a, recent, first, weights_out=None):
    w, kc, vc = a["weights"].cpu(), a["k_cache"].cpu().clone(), a["v_cache"].cpu().clone()
    src = a["page_table"].cpu().long()
    dst = src if a["out_table"] is None else a["out_table"].cpu().long()
    lens, (B, Hkv, _), page, budget = a["key_len"].tolist(), w.shape, kc.shape[2], a["budget"]
    wo = w.clone() if weights_out is None else weights_out.cpu().clone()
    want = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    k0, v0 = kc.clone(), vc.clone()
    for b in range(B):
        for h in range(Hkv):
            at = torch.tensor(chosen(w[b, h].tolist(), lens[b], budget, recent, first), dtype=torch.long)
            j = torch.arange(len(at))
            want[b, h, :len(at)] = at.to(torch.int32)
            wo[b, h, :len(at)] = w[b, h, at]
            for c, c0 in ((kc, k0), (vc, v0)):
                c[dst[b, j // page], h, j % page] = c0[src[b, at // page], h, at % page]
    st = wq.new_status()
    new_len, kept = wq.evict_paged(**a, recent=recent, first=first, weights_out=weights_out, status=st)
    assert int(st) == 0
    assert new_len.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(kept.cpu(), want)
    got = a["weights"] if weights_out is None else weights_out
    assert torch.equal(got.cpu().view(torch.int32), wo.view(torch.int32))
    assert torch.equal(a["k_cache"].cpu(), kc) and torch.equal(a["v_cache"].cpu(), vc)


CASES = [  # lengths, Hkv, dk, dv, page, dtype, budget, recent, first, token-major
    ([1], 1, 64, 64, 16, BF, 1, 0, 0, False),
    ([2], 1, 64, 64, 16, BF, 1, 0, 0, False),
    ([2], 2, 64, 32, 16, BF, 1, 1, 0, False),
    ([0, 5, 40, 33], 2, 128, 128, 16, BF, 32, 4, 2, True),
    ([100, 700, 64, 65], 3, 80, 96, 48, FP, 64, 10, 4, False),
    ([300, 20, 301], 2, 66, 34, 5, BF, 100, 0, 3, False),
    ([50, 60], 1, 33, 7, 1, FP, 49, 20, 29, False),
    ([3000, 2999, 10], 2, 128, 64, 64, BF, 2998, 100, 0, False),
    ([2100], 8, 128, 128, 32, BF, 512, 64, 4, False),
    ([5000, 4000], 1, 520, 8, 16, BF, 1300, 7, 1, True),
    ([60000, 49153], 2, 8, 8, 64, BF, 5000, 9, 4, False),  # past what shared memory holds
    ([70, 80, 90], 2, 64, 64, 16, BF, 200, 10, 10, False),  # nothing to evict
]


@pytest.mark.parametrize("lens,Hkv,dk,dv,page,dtype,budget,recent,first,token_major", CASES)
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("same_weights", [False, True])
def test_evict_paged(lens, Hkv, dk, dv, page, dtype, budget, recent, first, token_major, apart, same_weights):
    a = problem(lens, Hkv, dk, dv, page, dtype, budget, apart, token_major)
    out = None if same_weights else torch.full((len(lens), Hkv, budget + 2), 7.0, device="cuda")
    check(a, recent, first, out)


SPECIAL = [
    lambda w: torch.zeros_like(w),                                      # all equal: the earlier ones
    lambda w: torch.where(w > 1, 0.0, -0.0),                            # both zeros are equal
    lambda w: (w * 2).round() / 2,                                      # many ties
    lambda w: torch.where(w > 1.5, torch.tensor(math.nan), w),          # NaN goes first
    lambda w: torch.where(w > 2, torch.tensor(math.inf), torch.where(w < 0.5, torch.tensor(-math.inf), w)),
    lambda w: -w * 1e-40,                                               # subnormal, negative
    lambda w: torch.full_like(w, math.nan),
]


@pytest.mark.parametrize("weights", SPECIAL)
@pytest.mark.parametrize("budget,recent,first", [(1, 0, 0), (100, 0, 0), (150, 30, 4), (299, 0, 1)])
def test_ties_and_special_weights(weights, budget, recent, first):
    check(problem([300, 299, 200], 2, 64, 64, 16, BF, budget, False, weights=weights), recent, first)


def test_strided_weights_and_a_second_call():
    a = problem([400, 120], 2, 64, 64, 16, BF, 100, False)
    wide = torch.full((2, 2, 500), 7.0, device="cuda")
    wide[:, :, 20:423] = a["weights"].transpose(0, 1)
    b = {**a, "weights": wide[:, :, 20:423].transpose(0, 1), "k_cache": a["k_cache"].clone(), "v_cache": a["v_cache"].clone()}
    check(a, 10, 2)
    check(b, 10, 2)
    assert torch.equal(a["k_cache"], b["k_cache"]) and (wide[:, :, :20] == 7).all() and (wide[:, :, 423:] == 7).all()
    a["key_len"], a["budget"], a["max_len"] = i32([100, 100]), 60, 100
    check(a, 0, 0)


def test_bad_pages_and_lengths_are_reported_and_skipped():
    a = problem([100, 90], 2, 64, 64, 16, BF, 40, True)
    a["page_table"][0, 1], a["out_table"][1, 0] = 10 ** 6, -1
    k0, st = a["k_cache"].clone(), wq.new_status()
    _, kept = wq.evict_paged(**a, recent=5, status=st)
    assert int(st) == -6
    out, src, kept = a["out_table"].cpu(), a["page_table"].cpu(), kept.cpu()
    for b in range(2):
        for j in range(40):
            for h in range(2):
                i, to = int(kept[b, h, j]), int(out[b, j // 16])
                if to < 0:
                    continue
                page = int(src[b, i // 16])
                want = k0[to, h, j % 16] if page == 10 ** 6 else k0[page, h, i % 16]
                assert torch.equal(a["k_cache"][to, h, j % 16], want)
    for lens in ([101, 50], [-3, 50]):
        b, st = problem([100, 50], 2, 64, 64, 16, BF, 40, False), wq.new_status()
        b["key_len"] = i32(lens)
        new_len, _ = wq.evict_paged(**b, status=st)
        assert int(st) == -6 and new_len.tolist() == [40 if lens[0] > 0 else 0, 40]


def test_replayed_in_a_graph_with_other_lengths():
    a = problem([200, 200], 2, 64, 64, 16, BF, 60, True)
    ws, out = wq.evict_paged_workspace(a["weights"], 200, 60), torch.zeros(2, 2, 60, device="cuda")
    res = dict(new_len=torch.empty(2, dtype=torch.int32, device="cuda"),
               kept=torch.empty(2, 2, 60, dtype=torch.int32, device="cuda"), weights_out=out, ws=ws)
    a["key_len"].copy_(i32([200, 30]))
    wq.evict_paged(**a, **res, recent=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.evict_paged(**a, **res, recent=5)
    a["key_len"].copy_(i32([61, 199]))
    a["weights"].copy_(torch.rand(a["weights"].shape, generator=rng(3)))
    graph.replay()
    got = [res["kept"].clone(), out.clone(), a["k_cache"].clone()]
    wq.evict_paged(**a, **res, recent=5)
    assert res["new_len"].tolist() == [60, 60]
    assert all(torch.equal(x, y) for x, y in zip(got, (res["kept"], out, a["k_cache"])))


def test_last_pages_of_a_cache_past_32_bits():
    pages, Hkv, page, D = 16500, 8, 128, 128
    kc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    vc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    for c in (kc, vc):
        c[-2] = torch.randn(Hkv, page, D, generator=rng(1)).to(BF).cuda()
    w = torch.rand(1, Hkv, page, generator=rng(2)).cuda()
    _, kept = wq.evict_paged(w, kc, vc, i32([[pages - 2]]), i32([page]), page, 50, out_table=i32([[pages - 1]]))
    for h in range(Hkv):
        at = kept[0, h].long()
        assert torch.equal(kc[-1, h, :50], kc[-2, h, at]) and torch.equal(vc[-1, h, :50], vc[-2, h, at])
    assert not kc[-1, :, 50:].any() and not kc[0].any()


def test_attention_over_the_keys_that_stayed():
    """The whole run: weights of an attention choose the keys, and attention over
    the packed cache is attention over those keys."""
    Hkv, G, D, page, L, T = 2, 4, 64, 16, 500, 3
    a = problem([L, L - 77], Hkv, D, D, page, BF, 128, False, weights=torch.zeros_like)
    k0, v0, table = a["k_cache"].clone(), a["v_cache"].clone(), a["page_table"]
    q = (torch.randn(2 * T, Hkv * G, D, generator=rng(9)) * 2).to(BF).cuda()
    lse = torch.empty(2 * T, Hkv * G, device="cuda")
    wq.attention_shared_prefix(q, a["k_cache"], a["v_cache"], None, 0, table, a["key_len"], L, lse=lse)
    wq.attention_weights_paged(q, a["k_cache"], table, a["key_len"], L, lse, a["weights"])
    new_len, kept = wq.evict_paged(**a, recent=T)
    got = wq.attention_shared_prefix(q, a["k_cache"], a["v_cache"], None, 0, table, new_len, 128)
    assert (a["weights"][0, :, :128].sum(-1) > 0).all()
    for b in range(2):
        for h in range(Hkv):
            at = kept[b, h].long()
            k, v = (c[table[b, at // page].long(), h, at % page].double() for c in (k0, v0))
            qs = q[b * T:(b + 1) * T, h * G:(h + 1) * G].double()
            x = (qs @ k.T) * D ** -0.5  # [T, G, keys]
            x = x.masked_fill((torch.arange(128, device="cuda") > 128 - T + torch.arange(T, device="cuda")[:, None])[:, None], -math.inf)
            want = torch.softmax(x, -1) @ v
            # bf16 weights and output: 2^-8 of the values that are weighed, and as much of the result
            tol = 2 ** -8 * (torch.softmax(x, -1) @ v.abs() + want.abs()) + 1e-4
            assert ((got[b * T:(b + 1) * T, h * G:(h + 1) * G].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("at,dv", [(0, 96), (0, 64), (32, 64), (5, 40)])
def test_values_that_are_part_of_the_keys(apart, at, dv):
    """Elements that keys and values share move once, in place too."""
    a = problem([1500, 70, 9], 1 if at else 2, 96, dv, 16, BF, 64, apart, seed=at + dv)
    a["v_cache"] = a["k_cache"][..., at:at + dv]
    check(a, 8, 2)


@pytest.mark.parametrize("n", [131, 515, 2050, 6000, 40000])
@pytest.mark.parametrize("kind", ["equal", "three", "last bits", "middle bits"])
def test_weights_that_share_their_digits(n, kind):
    """Keys that the first digits do not tell apart, more and fewer than a block
    gathers or ranks, and equal ones."""
    i = torch.arange(n + 3)
    mixed = (i * 7919) % 4099
    w = {"equal": torch.full((n + 3,), 0.5), "three": (mixed % 3).float(),
         "last bits": 1 + mixed * 2.0 ** -23, "middle bits": 1 + (mixed % 300) * 2.0 ** -16}[kind]
    a = problem([n, n // 2], 1, 32, 32, 64, BF, max(n // 3, 8), True, weights=lambda x: w.float().expand_as(x).contiguous())
    check(a, 3, 1)
