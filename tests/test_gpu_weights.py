"""Accumulated attention weights of cached keys on the GPU against a float64
definition.  Tolerances are derived in serve_ref."""
import math

import pytest
import torch

import serve_ref as R
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def randn(*shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 7919 * len(shape) + sum(shape))
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def problem(ql, kl, Hkv, G, dk, page, dtype, token_major=False, lead=0, tail=0, spread=0.5):
    """Inputs whose unwritten places hold NaN: cache places past a length, rows
    of no sequence, weights of the tokens' own keys."""
    B, ns, T = len(ql), -(-max(max(kl), 1) // page), lead + sum(ql) + tail
    pages = B * ns + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(3))[:B * ns].reshape(B, ns)
    kc = randn(pages, page, Hkv, dk, dtype=dtype, seed=1)
    for b in range(B):
        for p in range(ns):
            kc[order[b, p], max(0, min(page, kl[b] - p * page)):] = math.nan
    kc = kc.transpose(1, 2) if token_major else kc.transpose(1, 2).contiguous()
    q = randn(T, Hkv * G, dk, dtype=dtype, seed=2, scale=1.5)
    cu = [lead + sum(ql[:b]) for b in range(B + 1)]
    q[:lead], q[cu[-1]:] = math.nan, math.nan
    w = randn(B, Hkv, max(kl) + 5, seed=4).abs()
    for b in range(B):
        w[b, :, max(0, kl[b] - ql[b]):kl[b]] = math.nan
    # log-sum-exps of a size that leaves weights between 0 and 1
    lse = torch.full((T, Hkv * G), math.nan)
    for b in range(B):
        if ql[b]:
            rows = slice(cu[b], cu[b + 1])
            lse[rows] = (1 + randn(ql[b], Hkv * G, seed=5).cpu() * spread) + 0.5 * dk ** 0.5 / 4 + math.log(1 + kl[b])
            hidden = torch.arange(ql[b]) < ql[b] - kl[b]  # tokens that see no key
            lse[rows][hidden] = -math.inf
    return dict(q=q, k_cache=kc, page_table=order.to(torch.int32).cuda(), key_len=i32(kl), max_len=max(kl),
                lse=lse.cuda(), weights=w, cu_q=i32(cu), max_q=max(max(ql), 1))


def check(a, decay=1.0, scale=None, **kw):
    want, tol = R.attention_weights(a["q"], a["k_cache"], a["page_table"], a["key_len"], a["cu_q"], a["lse"],
                                    a["weights"], a["q"].shape[2] ** -0.5 if scale is None else scale, decay)
    st = wq.new_status()
    got = wq.attention_weights_paged(**a, decay=decay, scale=scale, status=st, **kw)
    assert got is a["weights"] and int(st) == 0
    R.check(got, want, tol, "weights")


CASES = [  # tokens and keys of each sequence, Hkv, G, dk, page, dtype, token-major
    ([1], [1], 1, 1, 64, 16, BF, False),
    ([1], [300], 2, 4, 128, 64, BF, False),
    ([1, 1, 1], [17, 1, 530], 2, 8, 128, 128, BF, True),
    ([1, 1], [40, 257], 1, 16, 96, 8, FP, False),
    ([1] * 9, [3, 70, 64, 65, 128, 0, 255, 256, 257], 1, 7, 80, 48, BF, False),
    ([4, 1, 3], [9, 1, 130], 2, 5, 64, 32, FP, False),
    ([1, 0, 33, 2], [1, 5, 33, 300], 1, 4, 128, 16, BF, False),
    ([70, 129], [200, 129], 2, 2, 64, 16, BF, True),
    ([3, 2], [1, 0], 2, 1, 64, 16, FP, False),       # tokens that see nothing
    ([2, 2], [0, 1], 1, 33, 128, 64, BF, False),
    ([1] * 40, list(range(0, 120, 3)), 2, 8, 128, 64, BF, False),
    ([1, 2], [700, 40], 1, 128, 64, 128, FP, False),
    ([600, 37, 300], [700, 900, 300], 2, 3, 64, 16, BF, False),
    ([257], [1030], 3, 6, 128, 32, FP, False),
    ([5, 1, 40], [90, 33, 40], 2, 4, 72, 5, BF, True),    # any page size
    ([1, 0], [70, 9], 1, 2, 8, 1, FP, False),
    ([0, 0], [300, 9], 2, 2, 64, 16, BF, False),
]


@pytest.mark.parametrize("ql,kl,Hkv,G,dk,page,dtype,token_major", CASES)
@pytest.mark.parametrize("decay", [1.0, 0.9])
def test_attention_weights(ql, kl, Hkv, G, dk, page, dtype, token_major, decay):
    check(problem(ql, kl, Hkv, G, dk, page, dtype, token_major, lead=2 if sum(ql) else 0, tail=3 if sum(ql) else 0), decay)


@pytest.mark.parametrize("B,q,L", [(3, 1, 400), (2, 3, 70), (1, 300, 300)])
def test_even_tokens_without_cu_q(B, q, L):
    a = problem([q] * B, [L] * B, 2, 4, 64, 16, BF)
    b = {**a, "cu_q": None, "max_q": None, "weights": a["weights"].clone()}
    check(a, scale=0.3)
    wq.attention_weights_paged(**b, scale=0.3)
    assert torch.equal(a["weights"].nan_to_num(), b["weights"].nan_to_num())


@pytest.mark.parametrize("lse", [-80.0, -60.0, 60.0, 95.0, math.inf])
@pytest.mark.parametrize("ql,kl,G", [([1, 1], [200, 31], 4), ([200, 31], [300, 40], 4), ([90], [90], 5)])
def test_weights_far_from_one(lse, ql, kl, G):
    """Log-sum-exps that are not the scores' own: weights up to 2^120 and down
    to nothing, in some rows only."""
    a = problem(ql, kl, 2, G, 64, 16, BF)
    a["lse"][::3] = lse
    a["lse"][1::7] = lse / 2
    check(a)


@pytest.mark.parametrize("ql,kl", [([1, 1], [200, 31]), ([200, 31], [300, 40])])
def test_nonfinite_queries_and_sums_reach_the_keys_they_see(ql, kl):
    a = problem(ql, kl, 2, 4, 64, 16, BF)
    a["weights"] = a["weights"].nan_to_num()
    b = {**a, "q": a["q"].clone(), "lse": a["lse"].clone(), "weights": a["weights"].clone()}
    wq.attention_weights_paged(**a)
    row = ql[0] - 1  # the last token of the first sequence sees all its keys
    for name, value in (("q", math.nan), ("lse", math.nan), ("q", math.inf)):
        c = {k: v.clone() if k in ("q", "lse", "weights") else v for k, v in b.items()}
        c[name][row, 5] = value  # a query head of key head 1
        wq.attention_weights_paged(**c)
        n = kl[0]
        assert not c["weights"][0, 1, :n].isfinite().all() and (name == "q" and value == math.inf or
                                                                c["weights"][0, 1, :n].isnan().all())
        c["weights"][0, 1, :n], mine = 0, a["weights"].clone()
        mine[0, 1, :n] = 0
        assert torch.equal(c["weights"], mine)


def test_weights_in_other_strides_and_repeated_calls():
    a = problem([2, 7], [100, 300], 3, 2, 64, 16, BF)
    b = problem([2, 7], [100, 300], 3, 2, 64, 16, BF)
    wide = torch.full((3, 2, 400), 7.0, device="cuda")
    wide[:, :, 10:10 + 305] = a["weights"].transpose(0, 1)
    b["weights"] = wide[:, :, 10:10 + 305].transpose(0, 1)
    first = a["weights"].clone()
    check(a)
    wq.attention_weights_paged(**b)
    assert torch.equal(a["weights"].nan_to_num(), b["weights"].nan_to_num())
    assert (wide[:, :, :10] == 7).all() and (wide[:, :, 315:] == 7).all()
    again = {**a, "weights": first}
    wq.attention_weights_paged(**again)
    assert torch.equal(first.nan_to_num(), a["weights"].nan_to_num())


def test_weights_of_one_softmax_add_up():
    """With the attention's own lse, over its prefix too, a token's weights over
    all keys are one for each query head."""
    Hkv, G, D, page, P, L, T = 2, 4, 64, 16, 40, 333, 5
    kc, vc = randn(40, Hkv, page, D, dtype=BF, seed=1), randn(40, Hkv, page, D, dtype=BF, seed=2)
    q, lse = randn(T, Hkv * G, D, dtype=BF, seed=3), torch.empty(T, Hkv * G, device="cuda")
    table, prefix = torch.arange(22, dtype=torch.int32).cuda()[None], torch.arange(30, 33, dtype=torch.int32).cuda()
    wq.attention_shared_prefix(q, kc, vc, prefix, P, table, i32([L]), L, lse=lse)
    w = torch.zeros(1, Hkv, L, device="cuda")
    wq.attention_weights_paged(q, kc, table, i32([L]), L, lse, w)
    # the prefix's keys, as a sequence whose tokens come behind them all
    wp = torch.zeros(1, Hkv, P, device="cuda")
    for t in range(T):
        wq.attention_weights_paged(q[t:t + 1], kc, prefix[None], i32([P]), P, lse[t:t + 1], wp)
        if t + 1 < T:
            keep = wp[..., -1].clone() if t == 0 else keep + wp[..., -1]
    wp[..., -1] += keep  # each call begins its last key anew
    total = w.sum(-1) + wp.sum(-1)
    # lse and weights are each within the tolerances of their own tests, 1e-5 of the sum here
    assert (total / (T * G) - 1).abs().max() < 1e-5


def test_bad_pages_lengths_and_tokens_are_reported():
    for page, dk in ((16, 64), (5, 64)):
        a = problem([1, 1], [100, 100], 2, 4, dk, page, BF)
        want = {**a, "page_table": a["page_table"].clone(), "weights": a["weights"].clone()}
        a["page_table"][0, 2], a["page_table"][1, 0] = -1, 10 ** 6
        kc = a["k_cache"]
        for b, p in ((0, 2), (1, 0)):  # keys of a page that is none count as zeros
            kc[want["page_table"][b, p].long()] = 0
        st = wq.new_status()
        wq.attention_weights_paged(**a, status=st)
        assert int(st) == -6
        check(want)
        assert torch.equal(a["weights"].nan_to_num(), want["weights"].nan_to_num())
    for kw in (dict(key_len=i32([100, 101])), dict(key_len=i32([-1, 50])), dict(cu_q=i32([0, 1, 3]))):
        b, st = {**problem([1, 1], [100, 100], 2, 4, 64, 16, BF), **kw}, wq.new_status()
        wq.attention_weights_paged(**b, status=st)
        assert int(st) == -6


def test_replayed_in_a_graph_with_other_lengths():
    for ql, kl, more in (([1, 1], [60, 200], [61, 201]), ([200, 31], [300, 40], [300, 40])):
        a = problem(ql, [max(kl)] * 2, 2, 4, 64, 16, BF)
        a["key_len"].copy_(i32(kl))
        w0 = a["weights"].nan_to_num().clone()
        ws = wq.attention_weights_paged_workspace(a["q"], a["k_cache"], 2, a["max_len"], a["max_q"])
        a["weights"] = w0.clone()
        wq.attention_weights_paged(**a, ws=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            wq.attention_weights_paged(**a, ws=ws)
        a["weights"].copy_(w0)
        a["key_len"].copy_(i32(more))
        a["q"].copy_(randn(*a["q"].shape, dtype=BF, seed=8))
        graph.replay()
        got = a["weights"].clone()
        a["weights"].copy_(w0)
        wq.attention_weights_paged(**a, ws=ws)
        assert torch.equal(got, a["weights"]) and not torch.equal(got, w0)


def test_last_page_of_a_cache_past_32_bits():
    pages, Hkv, page, D = 16500, 8, 128, 128
    kc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    kc[0] = randn(Hkv, page, D, dtype=BF, seed=1)
    kc[-1] = kc[0]
    q, lse = randn(1, 16, D, dtype=BF, seed=2), torch.full((1, 16), 4.0, device="cuda")
    outs = []
    for p in (0, pages - 1):
        w = torch.zeros(1, Hkv, page, device="cuda")
        outs.append(wq.attention_weights_paged(q, kc, i32([[p]]), i32([page]), page, lse, w))
    assert torch.equal(outs[0], outs[1]) and (outs[0] > 0).all()


def test_on_another_stream_beside_a_busy_one():
    a = problem([1] * 4, [500, 3, 260, 90], 2, 4, 128, 16, BF)
    b = {**a, "weights": a["weights"].clone()}
    wq.attention_weights_paged(**a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        wq.attention_weights_paged(**b)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a["weights"].nan_to_num(), b["weights"].nan_to_num())
