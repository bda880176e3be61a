"""Norms of query and key heads with the rotary position in the same pass, and
on the way into a paged cache, on the GPU against float64 definitions.
Tolerances are derived in serve_ref."""
import pytest
import torch

import serve_ref as R
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def randn(*shape, dtype=F32, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 7919 * len(shape) + sum(shape))
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def weight(D, dtype, seed=9):
    return (1 + 0.3 * randn(D, seed=seed)).to(dtype)


HEADS = [  # T, heads, D, rot, lead, layout, dtype
    (1, 1, 2, 2, 0, "half", F32), (3, 5, 66, 34, 1, "inter", BF), (17, 8, 128, 128, 0, "half", BF),
    (5, 3, 64, 64, 128, "inter", FP), (7, 2, 80, 32, 0, "half", FP), (4, 4, 96, 48, 8, "half", BF),
    (6, 3, 72, 24, 0, "inter", BF), (9, 7, 40, 40, 0, "half", BF), (300, 16, 128, 64, 0, "half", F32),
    (2, 2, 512, 512, 0, "half", BF), (2, 3, 520, 520, 0, "half", FP), (3, 2, 256, 32, 0, "inter", F32),
    (5, 3, 80, 0, 0, "half", BF), (2, 1, 1000, 6, 0, "half", BF), (1, 1, 8, 0, 0, "inter", FP),
    (1100, 33, 128, 128, 0, "half", BF), (2300, 24, 80, 80, 0, "half", FP), (2200, 40, 80, 32, 0, "inter", F32),
]


@pytest.mark.parametrize("T,heads,D,rot,lead,layout,dtype", HEADS)
@pytest.mark.parametrize("weighted", [True, False])
def test_head_norm_rope(T, heads, D, rot, lead, layout, dtype, weighted):
    tab = wq.rope_table(5000, rot) if rot else None
    x = randn(T, heads, lead + D, dtype=dtype, scale=3.0)[:, :, lead:]
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32).cuda()
    w = weight(D, dtype) if weighted else None
    st = wq.new_status()
    got = wq.head_norm_rope(x, w, pos, tab, eps=EPS, layout=layout, status=st)
    want, mag = R.head_norm_rotate(x, w, pos, tab, layout, EPS)
    R.check(got, want, R.head_norm_tol(want, mag, dtype, D), "y")
    assert int(st) == 0
    same = x.clone()
    assert torch.equal(wq.head_norm_rope(same, w, pos, tab, eps=EPS, layout=layout, out=same), got)


def test_zero_and_nonfinite_heads_stay_apart():
    tab = wq.rope_table(10, 64)
    x = randn(4, 4, 64, dtype=BF)
    x[1, 2] = 0
    x[2, 1, 3] = float("nan")
    x[3, 0, 5] = float("inf")
    clean = x.clone()
    clean[2, 1], clean[3, 0] = 1.0, 1.0
    pos = torch.arange(4, dtype=torch.int32).cuda()
    got, ref = (wq.head_norm_rope(t, None, pos, tab) for t in (x, clean))
    assert (got[1, 2] == 0).all() and got[2, 1].isnan().all() and got[3, 0].isnan().any()
    for t, n in ((0, 0), (1, 0), (2, 0), (2, 2), (3, 1), (3, 3)):
        assert torch.equal(got[t, n], ref[t, n]) and got[t, n].isfinite().all()


def test_bad_position_is_reported_and_skipped():
    tab = wq.rope_table(10, 64)
    x = randn(4, 2, 64, dtype=BF)
    for D in (64, 63):  # the vector kernel, the element-wise one
        out = torch.full((4, 2, D), 7.0, dtype=BF, device="cuda")
        st = wq.new_status()
        wq.head_norm_rope(x[:, :, :D], None, torch.tensor([3, 10, -1, 9], dtype=torch.int32).cuda(),
                          tab if D == 64 else wq.rope_table(10, 62), out=out, status=st)
        assert int(st) == -6
        assert (out[1:3] == 7).all() and not (out[0] == 7).all() and not (out[3] == 7).all()


APPENDS = [  # T, Hq, Hkv, dk, dv, rot, page, layout, dtype, token-major pages
    (1, 1, 1, 64, 64, 64, 16, "half", BF, False), (13, 8, 2, 128, 128, 128, 64, "half", BF, True),
    (40, 28, 7, 80, 80, 32, 5, "half", FP, False), (9, 3, 3, 66, 34, 10, 1, "inter", BF, False),
    (33, 4, 1, 96, 64, 48, 48, "inter", FP, True), (8, 0, 2, 64, 64, 0, 16, "half", BF, False),
    (7, 2, 2, 64, 520, 64, 16, "half", BF, False), (2000, 40, 8, 128, 128, 128, 64, "inter", BF, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,dk,dv,rot,page,layout,dtype,token_major", APPENDS)
def test_head_norm_rope_append_paged(T, Hq, Hkv, dk, dv, rot, page, layout, dtype, token_major):
    pages = T // page + 4

    def paged(d, seed):
        if token_major:
            return randn(pages, page, Hkv, d, dtype=dtype, seed=seed).transpose(1, 2)
        return randn(pages, Hkv, page, d, dtype=dtype, seed=seed)

    kc, vc = paged(dk, 1), paged(dv, 2)
    slots = torch.randperm(pages * page)[:T]
    if T > 4:
        slots[2] = -1
    tab = wq.rope_table(777, rot) if rot else None
    pos = torch.randint(0, 777, (T,), dtype=torch.int32).cuda()
    qk = randn(T, Hq + Hkv, dk, dtype=dtype, seed=3, scale=2.0)
    q, k, v = (qk[:, :Hq] if Hq else None), qk[:, Hq:], randn(T, Hkv, dv, dtype=dtype, seed=4)
    wk, wqt = weight(dk, dtype, 5), (weight(dk, dtype, 6) if Hq else None)
    rk, mk = R.head_norm_rotate(k, wk, pos, tab, layout, EPS)
    tk = R.head_norm_tol(rk, mk, dtype, dk)
    want_k, want_v = R.f64(kc), R.f64(vc)
    tol = torch.zeros_like(want_k)
    on = slots >= 0
    p, o = slots[on] // page, slots[on] % page
    want_k[p, :, o], want_v[p, :, o], tol[p, :, o] = rk[on], R.f64(v)[on], tk[on]
    st = wq.new_status()
    got = wq.head_norm_rope_append_paged(k, v, pos, slots.cuda(), tab, kc, vc, k_weight=wk, q=q, q_weight=wqt,
                                         eps=EPS, layout=layout, status=st)
    R.check(kc, want_k, tol, "k_cache")
    R.check(vc, want_v, 0.0, "v_cache")
    if q is not None:
        want, mag = R.head_norm_rotate(q, wqt, pos, tab, layout, EPS)
        R.check(got, want, R.head_norm_tol(want, mag, dtype, dk), "q")
    assert int(st) == 0


@pytest.mark.parametrize("D", [64, 62])
def test_append_bad_slots_and_positions(D):
    kc, vc = torch.zeros(2, 2, 16, D, dtype=BF).cuda(), torch.zeros(2, 2, 16, D, dtype=BF).cuda()
    k, v = randn(3, 2, D, dtype=BF, seed=1), randn(3, 2, D, dtype=BF, seed=2)
    st = wq.new_status()
    wq.head_norm_rope_append_paged(k, v, torch.tensor([1, 2, 8], dtype=torch.int32).cuda(),
                                   torch.tensor([32, 3, 5]).cuda(), wq.rope_table(8, D), kc, vc, status=st)
    assert int(st) == -6
    assert torch.equal(vc[0, :, 3], v[1]) and int((vc != 0).any(-1).sum()) == 2 and int((kc != 0).any(-1).sum()) == 2


def test_last_page_of_a_cache_past_32_bits():
    """A cache of more than 2^32 bytes: the last page's places are as the first's."""
    pages, Hkv, page, D = 16500, 8, 128, 128
    assert pages * Hkv * page * D > 2 ** 31
    kc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    vc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    k, v, tab = randn(9, Hkv, D, dtype=BF, seed=1), randn(9, Hkv, D, dtype=BF, seed=2), wq.rope_table(100, D)
    pos = torch.arange(9, dtype=torch.int32).cuda()
    for p in (0, pages - 1):
        wq.head_norm_rope_append_paged(k, v, pos, p * page + torch.arange(9).cuda(), tab, kc, vc)
    assert torch.equal(kc[0], kc[-1]) and torch.equal(vc[0], vc[-1]) and kc[0, :, :9].any()


def test_replayed_in_a_graph():
    tab = wq.rope_table(64, 64)
    x, pos = randn(8, 4, 64, dtype=BF), torch.arange(8, dtype=torch.int32).cuda()
    kc, vc = torch.zeros(4, 4, 16, 64, dtype=BF).cuda(), torch.zeros(4, 4, 16, 64, dtype=BF).cuda()
    slots, out = torch.arange(8).cuda(), torch.empty_like(x)
    call = lambda: wq.head_norm_rope_append_paged(x, x, pos, slots, tab, kc, vc, q=x, q_out=out)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(randn(8, 4, 64, dtype=BF, seed=5))
    pos.add_(3)
    slots.add_(20)
    graph.replay()
    got = out.clone(), kc.clone()
    call()
    assert torch.equal(got[0], out) and torch.equal(got[1], kc) and kc[1, :, 4:12].any()
