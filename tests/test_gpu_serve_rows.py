"""Attention: what every row of the output holds and how its weights round,
at the places where sequences, bounds and types end."""
import pytest
import torch

import serve_ref as R
import test_gpu_serve as S
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def padded_inputs(lead, ql, trail, sl, P, Hkv, G, D, page, dtype):
    """Inputs whose q has `lead` rows before the first sequence and `trail`
    after the last, as a batch has that was padded for a recorded graph."""
    i = S.attn_inputs(ql, sl, P, Hkv, G, D, D, page, dtype, False)
    i["q"] = S.randn(lead + sum(ql) + trail, Hkv * G, D, dtype=dtype, seed=11, scale=2.0)
    i["cu_q"] += lead
    return i


def poisoned(i, P, max_suffix, max_q, fill, **kw):
    """The call with workspace, out and lse full of `fill`."""
    T, Hq = i["q"].shape[:2]
    ws = wq.attention_shared_prefix_workspace(i["q"], i["k_cache"], i["v_cache"], len(i["suffix_len"]), P, max_suffix, max_q)
    ws[:ws.numel() // 4 * 4].view(torch.float32).fill_(fill)
    out = torch.full((T, Hq, i["v_cache"].shape[-1]), fill, dtype=i["q"].dtype, device="cuda")
    lse = torch.full((T, Hq), fill, device="cuda")
    S.attn_call(i, P, max_suffix, max_q, ws=ws, out=out, lse=lse, **kw)
    return out, lse


NO_SEQUENCE = [  # lead, tokens, trail, suffix lengths, P, Hkv, G, D, page, dtype
    (2, [1, 1], 3, [5, 20], 100, 2, 4, 64, 16, BF),              # few rows: prefix and suffix joined
    (1, [2, 0, 3], 2, [9, 0, 300], 40, 1, 3, 128, 5, FP),        # ... pages off 16
    (0, [1] * 40, 8, [30] * 40, 300, 2, 8, 128, 16, BF),         # prefix by row tiles, suffixes by warps
    (3, [1] * 70, 1, [2] * 70, 700, 4, 8, 64, 16, BF),           # ... blocks of one warp and of four
    (5, [70, 129], 31, [200, 129], 150, 2, 2, 64, 16, BF),       # both by row tiles, joined
    (7, [200, 250, 170], 33, [200, 300, 171], 333, 4, 16, 128, 16, FP),  # both in one walk
    (1, [1, 1], 2, [17, 60], 0, 2, 4, 128, 16, BF),              # suffixes alone, nothing to join
    (4, [70, 90], 40, [100, 120], 0, 2, 2, 64, 16, FP),          # ... by row tiles
    (1, [2, 1], 1, [0, 0], 90, 2, 4, 64, 16, BF),                # the prefix alone, nothing to join
    (2, [30, 0, 30], 9, [0, 0, 0], 100, 2, 4, 128, 16, BF),      # ... by row tiles
    (2, [30, 30], 9, [0, 0], 30000, 1, 4, 128, 16, BF),          # ... joined
    (300, [70], 500, [90], 100, 2, 2, 64, 16, BF),               # more padding than tokens
    (100, [40], 300, [0], 100, 2, 4, 64, 16, BF),                # ... and the prefix alone
    (2, [3, 1], 3, [0, 0], 0, 2, 4, 64, 16, BF),                 # no keys at all
    (0, [0, 0], 4, [8, 9], 50, 1, 2, 64, 16, BF),                # no sequence has a token
]


@pytest.mark.parametrize("lead,ql,trail,sl,P,Hkv,G,D,page,dtype", NO_SEQUENCE)
@pytest.mark.parametrize("fill", [float("nan"), 50.0])
def test_rows_of_no_sequence_are_zero(lead, ql, trail, sl, P, Hkv, G, D, page, dtype, fill):
    """Whatever the buffers held: zeros and -inf there, and the sequences'
    rows as the definition has them."""
    i = padded_inputs(lead, ql, trail, sl, P, Hkv, G, D, page, dtype)
    st = wq.new_status()
    out, lse = poisoned(i, P, max(sl), max(max(ql), 1), fill, status=st)
    want, wl, tol, ltol = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                      i["suffix_len"], i["cu_q"], D ** -0.5, dtype)
    own = torch.zeros(len(out), dtype=torch.bool)
    own[lead:lead + sum(ql)] = True
    assert (out.cpu()[~own] == 0).all() and (lse.cpu()[~own] == -float("inf")).all()
    R.check(out, want, tol, "out")
    R.check(lse, wl, ltol, "lse")
    assert int(st) == 0


CUT = [  # tokens, the bound given, suffix lengths, P, Hkv, G, D, page
    ([1, 4, 2], 2, [9, 30, 8], 100, 2, 4, 64, 16),       # few rows, joined
    ([1, 4, 2], 2, [9, 30, 8], 0, 2, 4, 128, 16),        # ... nothing to join
    ([60, 150, 50], 70, [90, 200, 60], 130, 2, 4, 64, 16),     # row tiles, joined
    ([200, 330, 170], 210, [200, 400, 171], 333, 4, 16, 64, 16),  # one walk
    ([1, 4, 2], 2, [0, 0, 0], 100, 2, 4, 64, 16),        # the prefix alone
    ([40, 90, 30], 40, [0, 0, 0], 100, 2, 4, 64, 16),    # ... by row tiles
]


@pytest.mark.parametrize("ql,most,sl,P,Hkv,G,D,page", CUT)
@pytest.mark.parametrize("fill", [float("nan"), 50.0])
def test_tokens_past_the_bound_are_zero_and_reported(ql, most, sl, P, Hkv, G, D, page, fill):
    i = S.attn_inputs(ql, sl, P, Hkv, G, D, D, page, BF, False)
    good = S.attn_call(i, P, max(sl), max(ql))
    st = wq.new_status()
    out, lse = poisoned(i, P, max(sl), most, fill, status=st)
    assert int(st) == -6
    t0 = 0
    for n in ql:
        cut = slice(t0 + most, t0 + n)
        assert (out[cut] == 0).all() and (lse[cut] == -float("inf")).all()
        assert torch.isfinite(out[t0:t0 + n]).all()
        if n <= most:  # another split of the same keys: within two roundings of weights and result
            d = (out[t0:t0 + n].float() - good[t0:t0 + n].float()).abs().max()
            assert float(d) <= 4 * R.U[BF] * float(i["v_cache"].float().nan_to_num().abs().max())
        t0 += n


KERNELS = [  # tokens of each sequence, suffix keys, Hkv, G, D, page: which kernel the keys take
    ([1, 1], 3, 1, 4, 64, 16),            # few rows, blocks of four warps
    ([1] * 3, 40, 2, 8, 128, 5),          # ... pages off 16
    ([4] * 16, 200, 4, 8, 128, 16),       # suffixes by blocks of one warp, prefix by row tiles
    ([1] * 9, 3, 1, 8, 64, 16),           # prefix by row tiles (one), heads of 64
    ([1] * 40, 3, 1, 8, 128, 16),         # ... two row tiles, heads of 128
    ([70, 90], 150, 2, 4, 64, 16),        # suffixes by row tiles
    ([70, 90], 150, 2, 4, 128, 32),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,L,Hkv,G,D,page", KERNELS)
def test_scores_too_large_for_one_octave(ql, L, Hkv, G, D, page, dtype):
    """Scores around 2^32, where neighbouring float32 numbers are 512 apart:
    the one key that is ahead of all others (by an eighth) has weight one,
    the others none, so the result is its value to the bit (a 16-bit weight
    times a 16-bit value is exact in float32)."""
    P, B = 150, len(ql)
    i = S.attn_inputs(ql, [L] * B, P, Hkv, G, D, D, page, dtype, False, hole=0.0)
    keys = i["k_cache"]
    keys.fill_(2.0 ** 14)
    top = 77
    keys[int(i["prefix_pages"][top // page]), :, top % page] = 1.125 * 2.0 ** 14
    # heads and tokens with other significands: the offset's rounding errs either way
    s = 1 + torch.arange(i["q"].shape[0] * Hkv * G, device="cuda").remainder(113).float() / 128
    i["q"].copy_((s.view(-1, Hkv * G, 1) * 2.0 ** 14).expand_as(i["q"]))
    lse = torch.empty(i["q"].shape[:2], device="cuda")
    out = S.attn_call(i, P, L, max(ql), scale=0.125, lse=lse)
    v = i["v_cache"][int(i["prefix_pages"][top // page]), :, top % page]
    assert torch.equal(out, v.repeat_interleave(G, 0).expand_as(out))
    want = s.double().view(-1, Hkv * G) * 1.125 * 2.0 ** 28 * D * 0.125
    # a product rounded to float32, times the scale (rounded twice), times ln 2 (rounded twice)
    R.check(lse, want.cpu(), (6 * R.E * want).cpu(), "lse")


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("ql,L,Hkv,G,D,page", [k for k in KERNELS if k[-1] >= 16])
def test_fp16_keeps_weights_far_below_the_largest(ql, L, Hkv, G, D, page, first):
    """One key far ahead of 2^14 others that weigh about 2^-26 of it each: in all
    they have 2^-12 of the result, and all of it where the key's value is 0."""
    P, B, q0 = 16384, len(ql), 16.0
    i = S.attn_inputs(ql, [L] * B, P, Hkv, G, D, D, page, FP, False, hole=0.0)
    i["k_cache"].zero_()
    i["v_cache"].fill_(1.0)
    i["v_cache"][..., 1::2] = 4096.0
    top = 5 if first else P - 5
    page_of = int(i["prefix_pages"][top // page])
    # score of the key: log2 e * 16 * k0 = 26 with q = (16, 0, ...), scale 1
    k0 = torch.tensor(26 / 1.4426950408889634 / q0).half()
    i["k_cache"][page_of, :, top % page, 0] = k0
    i["v_cache"][page_of, :, top % page] = 0.0
    i["q"].zero_()
    i["q"][..., 0] = q0
    out = S.attn_call(i, P, L, max(ql), scale=1.0)
    want, _, _, _ = R.attention(i["q"], i["k_cache"], i["v_cache"], i["prefix_pages"], P, i["page_table"],
                                i["suffix_len"], i["cu_q"], 1.0, FP)
    # A weight is off by half a subnormal step of fp16, 2^-25, where the
    # largest is at least 2^7; the exponential by 2^-22 and its argument's
    # rounding, 26 * 2^-24 octaves; a sum of n weights by n * 2^-24; the result
    # by its own rounding.
    n = P + L
    vmax = torch.tensor([1.0, 4096.0] * (D // 2), dtype=torch.float64)
    tol = R.U[FP] * want.abs() + n * 2.0 ** -32 * vmax + want.abs() * (n * R.E + 64 * R.E)
    R.check(out, want, tol, "out")


FEW_ROWS = [  # tokens of each sequence, suffix keys, P, Hkv, G, D, page: every part by the kernel for few rows
    ([1] * 3, 40, 150, 2, 8, 128, 5),        # pages off 16
    ([1, 1], 90, 200, 4, 16, 64, 16),        # blocks of four warps
    ([4] * 16, 300, 0, 4, 8, 128, 16),       # blocks of one warp, two row tiles
    ([1] * 64, 320, 0, 4, 8, 128, 32),       # ... one row tile
    ([2] * 4, 320, 0, 1, 16, 64, 16),        # two row tiles, heads of 64
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("ql,L,P,Hkv,G,D,page", FEW_ROWS)
def test_average_of_equal_values_is_the_value(ql, L, P, Hkv, G, D, page, dtype):
    """With the same value at every key the result is that value, however the
    weights round: they are divided by the sum of what multiplied.  Float32
    sums of n weights are off by n * 2^-24 (n <= 320: 2^-15.6), under half a
    step of either type (2^-9, 2^-12), so it is equal to the bit."""
    i = S.attn_inputs(ql, [L] * len(ql), P, Hkv, G, D, D, page, dtype, False, hole=0.0)
    v = S.randn(Hkv, 1, D, dtype=dtype, seed=21)
    i["v_cache"].copy_(v[None].expand_as(i["v_cache"]))
    out = S.attn_call(i, P, L, max(ql))
    assert torch.equal(out, v.view(Hkv, D).repeat_interleave(G, 0).expand_as(out))
