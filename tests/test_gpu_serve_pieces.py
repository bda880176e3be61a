"""Attention by row tiles where a block walks several pieces of the prefix: the
end of one (query tokens, key head) item and the beginning of the next, with one
row tile in some and two in others."""
import pytest
import torch

import serve_ref as R
import test_gpu_serve as S
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

# An odd number of row tiles (128 / G tokens each) leaves one alone in its pair.
PIECES = [  # tokens, suffix lengths, P, Hkv, G, dk, dv, page, dtype
    ([51], [57], 18, 3, 128, 96, 96, 128, FP),
    ([120, 150, 150], [4, 2, 0], 32, 5, 5, 24, 128, 24, BF),
    ([16, 16, 16, 17], [0, 0, 0, 0], 1959, 8, 128, 128, 128, 16, BF),
    ([5, 18, 18, 18, 2], [2, 6, 6, 4, 4], 20, 5, 33, 128, 128, 64, FP),
    ([200], [201], 25, 8, 8, 96, 96, 256, BF),
    ([1] * 65, [3] * 65, 1300, 4, 128, 64, 64, 8, FP),
    ([2, 1] * 20 + [1], [2] * 41, 1636, 5, 33, 64, 64, 8, FP),
    ([1] * 33, [1] * 33, 3333, 8, 128, 128, 128, 64, BF),
    ([290], [300], 100, 16, 3, 64, 64, 32, BF),
]


@pytest.mark.parametrize("ql,sl,P,Hkv,G,dk,dv,page,dtype", PIECES)
def test_pieces_of_one_and_two_row_tiles(ql, sl, P, Hkv, G, dk, dv, page, dtype):
    i = S.attn_inputs(ql, sl, P, Hkv, G, dk, dv, page, dtype, False)
    T = sum(ql)
    assert -(-T // (128 // G)) % 2 == 1
    lse = torch.full((T, Hkv * G), 7.0, device="cuda")
    st = wq.new_status()
    out = S.attn_call(i, P, max(sl), max(ql), lse=lse, status=st)
    assert int(st) == 0
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], dk ** -0.5, dtype)
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    for _ in range(30):
        again = S.attn_call(i, P, max(sl), max(ql), status=st)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and int(st) == 0


@pytest.mark.parametrize("T,G", [(9, 8), (40, 8)])
def test_long_walks_with_heads_of_64(T, G):
    """Many key tiles a piece and a maximum that grows: the sums are scaled after
    products of which not every end is waited for."""
    P = 12000
    i = S.attn_inputs([1] * T, [1] * T, P, 8, G, 64, 64, 64, BF, False)
    ramp = (torch.arange(P, device="cuda", dtype=torch.float32) / P * 3).to(BF)
    pages, place = i["prefix_pages"].long()[torch.arange(P) // 64], torch.arange(P) % 64
    i["k_cache"][pages, :, place] = (i["k_cache"][pages, :, place].float() * 0.2 + ramp[:, None, None].float()).to(BF)
    i["q"].copy_((i["q"].abs() + 0.25).to(BF))
    st = wq.new_status()
    lse = torch.empty(i["q"].shape[:2], device="cuda")
    out = S.attn_call(i, P, 1, 1, scale=0.3, lse=lse, status=st)
    assert int(st) == 0
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], 0.3, BF)
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    for _ in range(30):
        assert torch.equal(S.attn_call(i, P, 1, 1, scale=0.3, status=st), out)
    assert int(st) == 0
