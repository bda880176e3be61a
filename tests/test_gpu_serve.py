"""The serving operators on the GPU against plain float64 definitions: block
norms, rotary positions, the rotated append to a paged cache, attention behind
a shared prefix.  Tolerances are derived in serve_ref."""
import math

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


# ---------------------------------------------------------------- norms
NORMS = [  # T, H, dtype, post, pre, gate, scale
    (1, 1, BF, "rms", "rms", "none", 1.0),
    (3, 7, FP, "layer", "rms", "token", 0.5),
    (5, 64, BF, "none", "rms", "shared", 1.0),
    (9, 264, BF, "rms", "layer", "token", 0.3),
    (300, 128, FP, "none", "rms", "none", 1.0),
    (33, 257, F32, "layer", "layer", "shared", 2.0),
    (4, 1000, F32, "rms", "none", "none", 1.0),
    (1, 7168, BF, "none", "rms", "none", 1.0),
    (400, 7168, BF, "rms", "rms", "none", 1.0),
    (17, 4099, FP, "layer", "layer", "token", 0.5),
    (310, 4101, BF, "rms", "rms", "none", 1.0),
    (2, 32768, BF, "rms", "rms", "shared", 1.0),
    (2, 32767, F32, "layer", "rms", "none", 1.0),
    (306, 32768, F32, "rms", "layer", "none", 1.0),
]


def norm_inputs(T, H, dtype, post, pre, gate):
    w = lambda k, kind: None if kind == "none" else 1 + 0.2 * randn(H, dtype=F32, seed=k)
    cast = lambda t: None if t is None else t.to(dtype)
    b = lambda k, kind: randn(H, dtype=dtype, seed=k, scale=0.1) if kind == "layer" else None
    return dict(block=randn(T, H, dtype=dtype, seed=1, scale=3), residual=randn(T, H, dtype=dtype, seed=2),
                gate={"none": None, "shared": randn(H, dtype=dtype, seed=3),
                      "token": randn(T, H, dtype=dtype, seed=3)}[gate],
                post_weight=cast(w(4, post)), post_bias=b(5, post), pre_weight=cast(w(6, pre)), pre_bias=b(7, pre))


def norm_check(got, i, dtype, scale, post, pre):
    h, y, mh, my = R.block_norm(i["block"], i["residual"], i["gate"], scale, post, i["post_weight"],
                                i["post_bias"], pre, i["pre_weight"], i["pre_bias"], EPS)
    # sums of up to 32 elements a thread and ten levels of a tree, and about
    # ten roundings more: 64 E relative to the magnitudes
    if got[0] is not None:
        R.check(got[0], h, R.U[dtype] * h.abs() + 64 * R.E * mh + R.TINY[dtype], "h")
    if got[1] is not None:
        R.check(got[1], y, R.U[dtype] * y.abs() + 64 * R.E * my + R.TINY[dtype], "y")


@pytest.mark.parametrize("T,H,dtype,post,pre,gate,scale", NORMS)
def test_block_norm(T, H, dtype, post, pre, gate, scale):
    i = norm_inputs(T, H, dtype, post, pre, gate)
    got = wq.block_norm(scale=scale, post=post, pre=pre, eps=EPS, **i)
    norm_check(got, i, dtype, scale, post, pre)


@pytest.mark.parametrize("H", [96, 99, 2056])
def test_block_norm_pitches_and_missing_parts(H):
    """Rows of wider tensors, no residual, outputs into the inputs."""
    T = 6
    wide = randn(T, H + 24, dtype=BF, seed=1)
    i = norm_inputs(T, H, BF, "rms", "rms", "none")
    i.update(block=wide[:, 8:8 + H], residual=None)
    norm_check(wq.block_norm(post="rms", pre="rms", eps=EPS, **i), i, BF, 1.0, "rms", "rms")
    i = norm_inputs(T, H, BF, "rms", "rms", "none")
    keep = {k: None if v is None else v.clone() for k, v in i.items()}
    got = wq.block_norm(post="rms", pre="rms", eps=EPS, x_out=i["residual"], y=i["block"], **i)
    assert got[0].data_ptr() == i["residual"].data_ptr()
    norm_check(got, keep, BF, 1.0, "rms", "rms")


@pytest.mark.parametrize("T,H,dtype", [(5, 99, BF), (7, 4099, FP), (3, 1001, F32)])
def test_block_norm_rows_that_start_apart(T, H, dtype):
    """Tensors whose rows lie differently against 16-byte boundaries."""
    i = norm_inputs(T, H, dtype, "layer", "rms", "token")
    i["residual"] = randn(T, H + 3, dtype=dtype, seed=8)[:, 1:1 + H]
    norm_check(wq.block_norm(post="layer", pre="rms", eps=EPS, **i), i, dtype, 1.0, "layer", "rms")


def test_block_norm_zero_and_nonfinite_rows_stay_apart():
    i = norm_inputs(4, 512, BF, "rms", "rms", "none")
    i["block"][1] = 0
    i["residual"][1] = 0
    i["block"][2, 5] = math.nan
    got = wq.block_norm(post="rms", pre="rms", eps=EPS, **i)
    assert torch.equal(got[0][1], torch.zeros_like(got[0][1])) and torch.equal(got[1][1], got[0][1])
    assert got[1][2].isnan().all()
    for t in (0, 1, 3):
        assert torch.isfinite(got[1][t]).all()


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=40.0, trained=4096),
                                dict(scaling="yarn", factor=4.0, trained=8, mscale=0.7)])
@pytest.mark.parametrize("rot", [4, 64, 130])
def test_rope_table(rot, kw):
    n = 70001
    got = wq.rope_table(n, rot, base=10000.0, **kw)
    want = R.table(n, rot, 10000.0, **kw)
    # float64 angles up to 7e4: a few units of 2^-53 * 7e4, then one rounding
    R.check(got, want, R.E * want.abs() + 1e-10, "table")


ROPES = [  # T, heads, D, rot, lead, layout, dtype
    (1, 1, 2, 2, 0, "half", F32), (3, 5, 66, 34, 1, "inter", BF), (17, 8, 128, 128, 0, "half", BF),
    (5, 3, 64, 64, 128, "inter", FP), (7, 2, 80, 32, 0, "half", FP), (4, 4, 96, 48, 8, "half", BF),
    (6, 3, 72, 24, 0, "inter", BF), (9, 7, 40, 40, 0, "half", BF), (300, 16, 128, 64, 0, "half", F32),
]


@pytest.mark.parametrize("T,heads,D,rot,lead,layout,dtype", ROPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(T, heads, D, rot, lead, layout, dtype, inverse):
    tab = wq.rope_table(5000, rot)
    x = randn(T, heads, lead + D, dtype=dtype)[:, :, lead:]
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32).cuda()
    st = wq.new_status()
    got = wq.rope(x, pos, tab, layout=layout, inverse=inverse, status=st)
    want, mag = R.rotate(x, pos, tab, layout, inverse)
    R.check(got, want, R.rope_tol(want, mag, dtype), "rope")
    assert torch.equal(got[..., rot:], x[..., rot:]) and int(st) == 0
    same = x.clone()[:, :, :]
    assert torch.equal(wq.rope(same, pos, tab, layout=layout, inverse=inverse, out=same), got)


def test_rope_gradient_is_the_inverse():
    """The rotation is linear and orthogonal, so the gradient of sum(g *
    rope(x)) is rope(g, inverse): against differences, exactly linear here."""
    tab = wq.rope_table(100, 16)
    x, g = randn(3, 2, 16, seed=1), randn(3, 2, 16, seed=2)
    pos = torch.tensor([0, 7, 99], dtype=torch.int32).cuda()
    grad = R.f64(wq.rope(g, pos, tab, inverse=True))
    for e in range(16):
        step = torch.zeros_like(x)
        step[..., e] = 1.0
        d = (R.f64(g) * (R.f64(wq.rope(x + step, pos, tab)) - R.f64(wq.rope(x - step, pos, tab)))).sum(-1) / 2
        # 16 products of float32 values off by 4 E (|a| + |b|), both of the order 4
        R.check(d, grad[..., e], torch.tensor(16 * 4 * 4 * 4 * 2 * R.E, dtype=torch.float64), "gradient")


def test_rope_bad_position_is_reported_and_skipped():
    tab = wq.rope_table(10, 64)
    x = randn(4, 2, 64, dtype=BF)
    out = torch.full_like(x, 7.0)
    st = wq.new_status()
    wq.rope(x, torch.tensor([3, 10, -1, 9], dtype=torch.int32).cuda(), tab, out=out, status=st)
    assert int(st) == -6
    assert (out[1:3] == 7).all() and not (out[0] == 7).all() and not (out[3] == 7).all()


# ---------------------------------------------------------------- rotated append
APPENDS = [  # T, Hq, Hkv, dk, dv, rot, page, layout, dtype, token-major pages
    (1, 1, 1, 64, 64, 64, 16, "half", BF, False), (13, 8, 2, 128, 128, 128, 64, "half", BF, True),
    (40, 28, 7, 80, 80, 32, 5, "half", FP, False), (9, 3, 3, 66, 34, 10, 1, "inter", BF, False),
    (33, 4, 1, 96, 64, 48, 48, "inter", FP, True), (8, 0, 2, 64, 64, 0, 16, "half", BF, False),
]


def paged(pages, heads, page, d, dtype, token_major, seed):
    if token_major:
        return randn(pages, page, heads, d, dtype=dtype, seed=seed).transpose(1, 2)
    return randn(pages, heads, page, d, dtype=dtype, seed=seed)


@pytest.mark.parametrize("T,Hq,Hkv,dk,dv,rot,page,layout,dtype,token_major", APPENDS)
def test_rope_append_paged(T, Hq, Hkv, dk, dv, rot, page, layout, dtype, token_major):
    pages = T // page + 4
    kc, vc = paged(pages, Hkv, page, dk, dtype, token_major, 1), paged(pages, Hkv, page, dv, dtype, token_major, 2)
    slots = torch.randperm(pages * page)[:T]
    if T > 4:
        slots[2] = -1
    tab = wq.rope_table(777, rot) if rot else None
    pos = torch.randint(0, 777, (T,), dtype=torch.int32).cuda()
    qk = randn(T, Hq + Hkv, dk, dtype=dtype, seed=3)
    q, k, v = (qk[:, :Hq] if Hq else None), qk[:, Hq:], randn(T, Hkv, dv, dtype=dtype, seed=4)
    wk, wv = R.f64(kc), R.f64(vc)
    tol = torch.zeros_like(wk)
    rk, mk = R.rotate(k, pos, tab, layout) if rot else (R.f64(k), torch.zeros(T, Hkv, dk))
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            wk[s // page, :, s % page], wv[s // page, :, s % page] = rk[t], R.f64(v[t])
            tol[s // page, :, s % page] = R.rope_tol(rk[t], mk[t], dtype) if rot else 0.0
    st = wq.new_status()
    got = wq.rope_append_paged(k, v, pos, slots.cuda(), tab, kc, vc, layout=layout, q=q, status=st)
    R.check(kc, wk, tol, "k_cache")
    R.check(vc, wv, 0.0, "v_cache")
    if q is not None:
        want, mag = R.rotate(q, pos, tab, layout)
        R.check(got, want, R.rope_tol(want, mag, dtype), "q")
    assert int(st) == 0


def test_append_bad_slots_and_positions():
    kc, vc = torch.zeros(2, 2, 16, 64, dtype=BF).cuda(), torch.zeros(2, 2, 16, 64, dtype=BF).cuda()
    k, v = randn(3, 2, 64, dtype=BF, seed=1), randn(3, 2, 64, dtype=BF, seed=2)
    tab = wq.rope_table(8, 64)
    st = wq.new_status()
    wq.rope_append_paged(k, v, torch.tensor([1, 2, 8], dtype=torch.int32).cuda(),
                         torch.tensor([32, 3, 5]).cuda(), tab, kc, vc, status=st)
    assert int(st) == -6
    assert torch.equal(vc[0, :, 3], v[1]) and int((vc != 0).any(-1).sum()) == 2 and int((kc != 0).any(-1).sum()) == 2


def test_append_and_attention_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: the last page works
    as the first."""
    pages, Hkv, page, D = 16500, 8, 128, 128
    assert pages * Hkv * page * D > 2 ** 31
    kc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    vc = torch.zeros(pages, Hkv, page, D, dtype=BF, device="cuda")
    tab = wq.rope_table(100, D)
    n = 100
    k, v, q = randn(n, Hkv, D, dtype=BF, seed=1), randn(n, Hkv, D, dtype=BF, seed=2), randn(1, 16, D, dtype=BF, seed=3)
    pos = torch.arange(n, dtype=torch.int32).cuda()
    outs = []
    for p in (0, pages - 1):
        wq.rope_append_paged(k, v, pos, p * page + torch.arange(n).cuda(), tab, kc, vc)
        pt = torch.tensor([[p]], dtype=torch.int32).cuda()
        outs.append(wq.attention_shared_prefix(q, kc, vc, None, 0, pt, torch.tensor([n], dtype=torch.int32).cuda(), n))
    assert torch.equal(kc[0], kc[-1]) and torch.equal(vc[0], vc[-1]) and vc[0].any()
    assert torch.equal(outs[0], outs[1]) and outs[0].any()


# ---------------------------------------------------------------- attention
ATTN = [  # q tokens of each sequence, suffix lengths, P, Hkv, G, dk, dv, page, dtype, token-major
    ([1], [1], 0, 1, 1, 64, 64, 16, BF, False),
    ([1], [0], 1, 2, 4, 128, 128, 16, BF, False),
    ([1, 1, 1], [17, 1, 130], 333, 2, 8, 128, 128, 16, BF, True),
    ([1, 1], [40, 257], 0, 1, 16, 96, 96, 5, FP, False),
    ([1] * 9, [3, 70, 64, 65, 128, 0, 5, 200, 31], 65, 1, 7, 80, 64, 48, BF, False),
    ([4, 1, 3], [9, 1, 130], 100, 2, 5, 64, 128, 32, FP, False),
    ([1, 0, 33, 2], [1, 5, 33, 300], 48, 1, 4, 128, 64, 1, BF, False),
    ([70, 129], [200, 129], 150, 2, 2, 64, 64, 16, BF, True),
    ([3], [1], 0, 2, 1, 64, 64, 16, FP, False),      # tokens 0 and 1 see nothing
    ([2, 2], [0, 1], 0, 1, 33, 128, 128, 64, BF, False),
    ([1] * 40, list(range(0, 120, 3)), 1000, 2, 8, 128, 128, 64, BF, False),
    ([1] * 40, list(range(40, 0, -1)), 700, 1, 128, 64, 64, 128, FP, False),
    ([300], [900], 513, 1, 3, 128, 128, 256, BF, False),
    ([150, 7, 90], [150, 300, 91], 259, 2, 1, 96, 128, 24, FP, True),
    ([1] * 72, [2] * 72, 1500, 5, 8, 64, 64, 16, BF, False),   # pairs of row tiles, the last with one
    ([1] * 72, [2] * 72, 1500, 5, 8, 128, 128, 16, BF, False),
    ([1] * 290, [1] * 290, 700, 3, 8, 64, 64, 16, FP, False),  # ten pairs in gangs of eight or so
]


def attn_inputs(ql, sl, P, Hkv, G, dk, dv, page, dtype, token_major, hole=math.nan, seed=0):
    """A cache whose places past every length hold `hole`."""
    T, B = sum(ql), len(ql)
    npx, ns = -(-P // page), -(-max(max(sl), 1) // page)
    pages = npx + B * ns + 2
    kc, vc = paged(pages, Hkv, page, dk, dtype, token_major, 1 + seed), paged(pages, Hkv, page, dv, dtype, token_major, 2 + seed)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    pre, pt = order[:npx].contiguous(), order[npx:npx + B * ns].view(B, ns).contiguous()
    used = torch.zeros(pages, page, dtype=torch.bool)
    mark = lambda lst, n: [used.__setitem__((int(lst[i // page]), i % page), True) for i in range(n)]
    mark(pre.cpu(), P)
    for b in range(B):
        mark(pt[b].cpu(), sl[b])
    hide = ~used[:, None, :, None].cuda()
    kc.masked_fill_(hide, hole)
    vc.masked_fill_(hide, hole)
    cu = torch.tensor([sum(ql[:b]) for b in range(B + 1)], dtype=torch.int32).cuda()
    return dict(q=randn(T, Hkv * G, dk, dtype=dtype, seed=3 + seed, scale=2.0), k_cache=kc, v_cache=vc,
                prefix_pages=pre, page_table=pt, suffix_len=torch.tensor(sl, dtype=torch.int32).cuda(), cu_q=cu)


def attn_call(i, P, max_suffix, max_q, **kw):
    return wq.attention_shared_prefix(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], max_suffix, cu_q=i["cu_q"], max_q=max_q, **kw)


@pytest.mark.parametrize("ql,sl,P,Hkv,G,dk,dv,page,dtype,token_major", ATTN)
def test_attention(ql, sl, P, Hkv, G, dk, dv, page, dtype, token_major):
    i = attn_inputs(ql, sl, P, Hkv, G, dk, dv, page, dtype, token_major)
    lse = torch.full((sum(ql), Hkv * G), 7.0, device="cuda")
    st = wq.new_status()
    out = attn_call(i, P, max(sl), max(ql), lse=lse, status=st)
    scale = dk ** -0.5
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], scale, dtype)
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    assert int(st) == 0
    # a longer bound on the suffixes and on the tokens changes the split, not the result's meaning
    room = i["page_table"].shape[1] * page
    R.check(attn_call(i, P, room, max(ql) + 5), want, tol, "out under wider bounds")
    # the same call again gives the same bits
    assert torch.equal(attn_call(i, P, max(sl), max(ql)), out)


# enough row tiles for every SM: prefix and suffix in one walk, with tails at
# the end of either, of both and of none, and sequences that see the prefix alone
WALKS = [([200, 250, 170], [200, 300, 171], 333, 4, 16, 128, 16, BF), ([90, 1, 400], [90, 7, 650], 130, 8, 8, 64, 32, FP),
         ([300, 300], [384, 512], 256, 4, 16, 64, 16, BF), ([310, 300], [310, 0], 100, 4, 16, 128, 64, FP)]


@pytest.mark.parametrize("ql,sl,P,Hkv,G,D,page,dtype", WALKS)
def test_attention_walks_prefix_and_suffix(ql, sl, P, Hkv, G, D, page, dtype):
    i = attn_inputs(ql, sl, P, Hkv, G, D, D, page, dtype, False)
    lse = torch.full((sum(ql), Hkv * G), 7.0, device="cuda")
    st = wq.new_status()
    out = attn_call(i, P, max(sl), max(ql), lse=lse, status=st)
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], D ** -0.5, dtype)
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    for _ in range(100):  # the same bits whatever the timing, and no wait that ran out
        again = attn_call(i, P, max(sl), max(ql), status=st)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and int(st) == 0


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,sl,P", [([1, 1], [50, 90], 130), ([100, 60], [100, 90], 130)])
def test_attention_extreme_scores(dtype, ql, sl, P):
    """Scores of hundreds with one sign, then the other, and keys that meet
    later in the range with the largest ones: the running maximum moves."""
    i = attn_inputs(ql, sl, P, 1, 4, 64, 64, 16, dtype, False)
    ramp = torch.arange(P, dtype=F32)
    for n in range(P):
        i["k_cache"][i["prefix_pages"][n // 16].item(), 0, n % 16] = ((ramp[n] - 65) / 10).to(dtype)
    i["q"].copy_(torch.where(i["q"] > 0, 3.0, 2.0))
    i["q"][1] *= -1
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], 0.5, dtype)
    lse = torch.empty(sum(ql), 4, device="cuda")
    R.check(attn_call(i, P, max(sl), max(ql), lse=lse, scale=0.5), want, tol, "out")
    R.check(lse, wl, ltol, "lse")


@pytest.mark.parametrize("B,D", [(10, 64), (10, 128), (40, 64), (40, 128)])
@pytest.mark.parametrize("up", [True, False])
def test_attention_scores_that_keep_growing(B, D, up):
    """Each key outweighs those before it (or after it), by 2^8 every few
    tiles: the sums are scaled again and again, one row tile or two."""
    P, G = 2100, 8
    i = attn_inputs([1] * B, [3] * B, P, 1, G, D, D, 16, BF, False)
    ramp = torch.arange(P, dtype=F32, device="cuda") / P * 4
    pages, place = i["prefix_pages"].long()[torch.arange(P) // 16], torch.arange(P) % 16
    i["k_cache"][pages, 0, place] = (ramp if up else ramp.flip(0))[:, None].expand(P, D).to(BF)
    i["q"].copy_((i["q"].abs() + 0.5).to(BF))
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], 0.4, BF)
    for _ in range(20):
        lse = torch.empty(B, G, device="cuda")
        R.check(attn_call(i, P, 3, 1, lse=lse, scale=0.4), want, tol, "out")
        R.check(lse, wl, ltol, "lse")


@pytest.mark.parametrize("ql", [[1, 1], [64, 80]])
def test_attention_strided_views_and_other_stream(ql):
    """q as a slice of a wider row, out likewise, on a stream of its own."""
    sl, P, Hkv, G, D = [80, 100], 200, 2, 4, 64
    i = attn_inputs(ql, sl, P, Hkv, G, D, D, 16, BF, True)
    wide = torch.zeros(sum(ql), Hkv * G + 3, D + 8, dtype=BF, device="cuda")
    wide[:, 1:1 + Hkv * G, :D] = i["q"]
    plain = attn_call(i, P, 100, max(ql))
    i["q"] = wide[:, 1:1 + Hkv * G, :D]
    room = torch.full((sum(ql), Hkv * G, D + 6), 5.0, dtype=BF, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        attn_call(i, P, 100, max(ql), out=room[..., :D])
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(room[..., :D], plain) and (room[..., D:] == 5).all()


@pytest.mark.parametrize("ql,page", [([1, 1], 16), ([90, 70], 16), ([90, 70], 12)])
def test_attention_bad_pages_and_lengths_are_reported(ql, page):
    """Page ids outside the cache, lengths and token counts past their bounds:
    a status, finite in-bounds work, other sequences untouched."""
    sl, P = [100, 90], 64
    i = attn_inputs(ql, sl, P, 2, 4, 64, 64, page, BF, False, hole=0.0)
    good = attn_call(i, P, 100, max(ql))
    bad = dict(i, page_table=i["page_table"].clone())
    bad["page_table"][0, 2] = 10 ** 9
    bad["page_table"][0, 1] = -3
    st = wq.new_status()
    out = attn_call(bad, P, 100, max(ql), status=st)
    assert int(st) == -6 and torch.isfinite(out).all()
    assert torch.equal(out[ql[0]:], good[ql[0]:])
    st = wq.new_status()
    long = dict(i, suffix_len=torch.tensor([10 ** 6, 90], dtype=torch.int32).cuda())
    assert torch.isfinite(attn_call(long, P, 100, max(ql), status=st)).all() and int(st) == -6
    st = wq.new_status()
    short = dict(i, suffix_len=torch.tensor([-5, 90], dtype=torch.int32).cuda())
    assert torch.isfinite(attn_call(short, P, 100, max(ql), status=st)).all() and int(st) == -6


def test_attention_uniform_tokens_and_graph():
    """cu_q left out, recorded into a graph and replayed on new data."""
    ql, sl, P = [1] * 4, [20, 33, 64, 65], 130
    i = attn_inputs(ql, sl, P, 2, 8, 128, 128, 16, BF, False)
    out = torch.empty_like(i["q"])
    ws = wq.attention_shared_prefix_workspace(i["q"], i["k_cache"], i["v_cache"], 4, P, 65, 1)
    call = lambda: wq.attention_shared_prefix(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P,
                                              i["page_table"], i["suffix_len"], 65, out=out, ws=ws)
    call()
    assert torch.equal(out, attn_call(i, P, 65, 1))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    i["q"].copy_(randn(*i["q"].shape, dtype=BF, seed=99))
    i["suffix_len"].copy_(torch.tensor([1, 30, 0, 64], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, attn_call(i, P, 65, 1))
