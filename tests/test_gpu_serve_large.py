"""The serving operators at sizes that take the kernels for many rows and
tokens, against the float64 definitions, and one output alone."""
import ctypes

import pytest
import torch

import serve_ref as R
import test_gpu_serve as S
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6

# Norms of more than 6 x 152 rows of whole 16-byte pieces walk them, up to four
# blocks of 256 threads an SM: 1400 rows are two rounds or three, 3000 four or
# more, the last without a row for some.
STREAM = [  # T, H, dtype, post, pre, gate, scale
    (1400, 1024, BF, "rms", "rms", "none", 1.0),        # two pieces a thread, every thread full
    (3000, 1032, FP, "layer", "rms", "token", 0.5),     # ... the last ones with less
    (1400, 4096, BF, "rms", "layer", "shared", 0.3),    # two pieces, widest
    (913, 4104, BF, "layer", "layer", "token", 1.0),    # four pieces
    (1400, 8192, FP, "none", "rms", "none", 1.0),       # four pieces, widest
    (1400, 7168, BF, "rms", "rms", "token", 2.0),
    (3000, 260, F32, "layer", "rms", "none", 1.0),
    (1000, 2048, F32, "rms", "layer", "token", 0.5),
    (1000, 4096, F32, "none", "rms", "shared", 1.0),
    (1000, 515, BF, "rms", "rms", "token", 1.0),        # rows shifted against 16 bytes
    (1000, 1027, F32, "layer", "rms", "shared", 1.0),
    (1500, 8200, BF, "rms", "rms", "none", 1.0),        # wider than the walking kernel takes
]


@pytest.mark.parametrize("T,H,dtype,post,pre,gate,scale", STREAM)
def test_block_norm_of_many_rows(T, H, dtype, post, pre, gate, scale):
    i = S.norm_inputs(T, H, dtype, post, pre, gate)
    S.norm_check(wq.block_norm(scale=scale, post=post, pre=pre, eps=EPS, **i), i, dtype, scale, post, pre)


@pytest.mark.parametrize("T,H,dtype", [(1400, 1032, BF), (1000, 2048, F32), (1000, 515, FP)])
def test_block_norm_of_many_rows_in_place(T, H, dtype):
    """Outputs into the inputs while later rows are on their way, and no
    residual."""
    i = S.norm_inputs(T, H, dtype, "rms", "layer", "token")
    keep = {k: None if v is None else v.clone() for k, v in i.items()}
    got = wq.block_norm(post="rms", pre="layer", eps=EPS, x_out=i["residual"], y=i["block"], **i)
    S.norm_check(got, keep, dtype, 1.0, "rms", "layer")
    i = S.norm_inputs(T, H, dtype, "rms", "rms", "none")
    i["residual"] = None
    S.norm_check(wq.block_norm(post="rms", pre="rms", eps=EPS, **i), i, dtype, 1.0, "rms", "rms")


@pytest.mark.parametrize("T,H", [(3, 64), (5, 1000), (400, 2048), (1400, 1032), (6, 99), (2, 32768)])
@pytest.mark.parametrize("which", [0, 1])
def test_block_norm_one_output(T, H, which):
    """x_out or y alone, through the C interface."""
    i = S.norm_inputs(T, H, BF, "rms", "layer", "none")
    out = torch.full((T + 1, H), 7.0, dtype=BF, device="cuda")
    at = lambda t: None if t is None else t.data_ptr()
    wq._check(wq.lib().wq_block_norm(
        at(i["block"]), H, at(i["residual"]), H, None, 0, 1.0, wq.NORM["rms"], at(i["post_weight"]), None,
        wq.NORM["layer"], at(i["pre_weight"]), at(i["pre_bias"]), EPS, T, H, 0, None if which else at(out), H,
        at(out) if which else None, H, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)), "wq_block_norm")
    S.norm_check((None, out[:T]) if which else (out[:T], None), i, BF, 1.0, "rms", "layer")
    assert (out[T] == 7).all()


# Rotary launches of more than 622592 units of 16 elements give a thread four
# heads: head counts that four does not divide, heads that end inside a unit.
ROPES = [  # T, heads, D, rot, lead, layout, dtype
    (2900, 29, 128, 128, 0, "half", BF), (4200, 30, 80, 32, 0, "half", FP), (5300, 31, 64, 64, 128, "inter", BF),
    (4200, 27, 96, 56, 8, "inter", FP), (160000, 1, 64, 16, 0, "half", BF), (3000, 70, 40, 40, 0, "inter", BF),
]


@pytest.mark.parametrize("T,heads,D,rot,lead,layout,dtype", ROPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_of_many_tokens(T, heads, D, rot, lead, layout, dtype, inverse):
    rows = rot // 16 + (D - rot // 16 * 16 + 15) // 16
    assert T * heads * rows > 4 * 256 * 152 * 4
    tab = wq.rope_table(5000, rot)
    x = S.randn(T, heads, lead + D, dtype=dtype)[:, :, lead:]
    pos = torch.randint(0, 5000, (T,), dtype=torch.int32).cuda()
    st = wq.new_status()
    got = wq.rope(x, pos, tab, layout=layout, inverse=inverse, status=st)
    want, mag = R.rotate(x, pos, tab, layout, inverse)
    R.check(got, want, R.rope_tol(want, mag, dtype), "rope")
    assert torch.equal(got[..., rot:], x[..., rot:]) and int(st) == 0
    # the same numbers in launches that give a thread one head
    few = T // 7
    assert torch.equal(wq.rope(x[:few], pos[:few], tab, layout=layout, inverse=inverse), got[:few])


@pytest.mark.parametrize("Hq,Hkv,dk,dv,rot,page,layout,dtype", [
    (28, 7, 80, 80, 32, 16, "half", FP), (10, 3, 128, 64, 128, 48, "inter", BF), (0, 5, 64, 128, 64, 64, "half", BF),
    (6, 6, 96, 96, 0, 16, "half", BF)])
def test_append_of_many_tokens(Hq, Hkv, dk, dv, rot, page, layout, dtype):
    units = lambda D, r: r // 16 + (D - r // 16 * 16 + 15) // 16
    T = 4 * 256 * 152 * 4 // ((Hq + Hkv) * units(dk, rot) + Hkv * units(dv, 0)) + 3
    pages = T // page + 4
    kc, vc = S.paged(pages, Hkv, page, dk, dtype, False, 1), S.paged(pages, Hkv, page, dv, dtype, False, 2)
    slots = torch.randperm(pages * page)[:T]
    slots[::50] = -1
    tab = wq.rope_table(777, rot) if rot else None
    pos = torch.randint(0, 777, (T,), dtype=torch.int32).cuda()
    qk = S.randn(T, Hq + Hkv, dk, dtype=dtype, seed=3)
    q, k, v = (qk[:, :Hq] if Hq else None), qk[:, Hq:], S.randn(T, Hkv, dv, dtype=dtype, seed=4)
    wk, wv, tol = R.f64(kc), R.f64(vc), torch.zeros(kc.shape, dtype=torch.float64)
    rk, mk = R.rotate(k, pos, tab, layout) if rot else (R.f64(k), torch.zeros(T, Hkv, dk, dtype=torch.float64))
    keep = slots >= 0
    p, o = slots[keep] // page, slots[keep] % page
    wk[p, :, o], wv[p, :, o] = rk[keep], R.f64(v)[keep]
    if rot:
        tol[p, :, o] = R.rope_tol(rk, mk, dtype)[keep]
    st = wq.new_status()
    got = wq.rope_append_paged(k, v, pos, slots.cuda(), tab, kc, vc, layout=layout, q=q, status=st)
    R.check(kc, wk, tol, "k_cache")
    R.check(vc, wv, 0.0, "v_cache")
    if q is not None and rot:
        want, mag = R.rotate(q, pos, tab, layout)
        R.check(got, want, R.rope_tol(want, mag, dtype), "q")
    elif q is not None:
        assert torch.equal(got, q)
    assert int(st) == 0


# Attention: forms of the kernel for few rows beside those of test_gpu_serve
FEW_ROWS = [  # tokens, suffix lengths, P, Hkv, G, dk, dv, page, dtype
    ([4, 3, 2], [40, 300, 2], 70, 2, 8, 64, 64, 16, BF),                 # two row tiles, heads of 64
    ([4] * 20, [i * 7 + 4 for i in range(20)], 0, 4, 8, 128, 128, 16, BF),   # ... of 128, blocks of one warp
    ([2, 4] * 9, [90] * 18, 260, 5, 8, 128, 96, 32, FP),                 # ... behind a prefix by row tiles
    ([1, 1, 1], [33, 1, 140], 57, 2, 7, 64, 48, 5, FP),                  # pages off 16, heads of 64
    ([4, 1, 3], [33, 1, 140], 57, 2, 8, 64, 64, 6, BF),                  # ... two row tiles
    ([4, 2], [700, 41], 333, 1, 8, 128, 128, 7, BF),                     # ... heads of 128
    ([2, 1], [5000, 4500], 0, 2, 8, 128, 128, 16, BF),                   # long ranges in four-warp blocks
]


@pytest.mark.parametrize("ql,sl,P,Hkv,G,dk,dv,page,dtype", FEW_ROWS)
def test_attention_of_few_rows(ql, sl, P, Hkv, G, dk, dv, page, dtype):
    S.test_attention(ql, sl, P, Hkv, G, dk, dv, page, dtype, False)


@pytest.mark.parametrize("ql,sl", [([1] * 12, [20, 33, 64, 65, 1, 2, 3, 64, 40, 41, 42, 43]), ([3, 1, 4, 2] * 4, [65] * 16)])
def test_attention_chain_in_a_graph(ql, sl):
    """Prefix by row tiles, suffixes by warps, join: three kernels that overlap,
    recorded and replayed on new data, then with padding at the end."""
    P, B, most = 700, len(ql), max(ql)
    i = S.attn_inputs(ql, sl, P, 2, 8, 128, 128, 16, BF, False, hole=0.0)
    out = torch.empty_like(i["q"])
    lse = torch.empty(out.shape[:2], device="cuda")
    ws = wq.attention_shared_prefix_workspace(i["q"], i["k_cache"], i["v_cache"], B, P, 65, most)
    call = lambda **kw: wq.attention_shared_prefix(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P,
                                                   i["page_table"], i["suffix_len"], 65, cu_q=i["cu_q"], max_q=most, **kw)
    call(out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out=out, lse=lse, ws=ws)
    for step in range(4):
        i["q"].copy_(S.randn(*i["q"].shape, dtype=BF, seed=99 + step, scale=2.0))
        i["suffix_len"].copy_(torch.tensor([max(n - 7 * step, 1) for n in sl], dtype=torch.int32))
        if step == 3:  # the last three sequences are gone, and their tokens padding
            i["cu_q"][-3:] = i["cu_q"][-4].clone()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                          i["suffix_len"], i["cu_q"], 128 ** -0.5, BF)
        R.check(out, want, tol, "out")
        R.check(lse, wl, ltol, "lse")
        assert torch.equal(call(), out)
