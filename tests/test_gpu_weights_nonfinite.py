"""Keys with an infinite or NaN element in the attention weights: the formula's
value for that key, whatever the query tiles' unused rows hold, and no other
key's weight changed."""
import math

import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 3, 5, 7, 8, 12, 100])
@pytest.mark.parametrize("ql,kl", [([400], [512]), ([130, 1, 77], [300, 200, 77]), ([1, 1], [300, 40]), ([9], [70])])
@pytest.mark.parametrize("dk,page,dtype", [(64, 16, torch.bfloat16), (128, 32, torch.float16), (64, 5, torch.bfloat16)])
def test_keys_that_are_not_finite(G, ql, kl, dk, page, dtype):
    g = torch.Generator().manual_seed(G + sum(ql))
    B, ns, T = len(ql), -(-max(kl) // page), sum(ql)
    q = torch.randn(T, 2 * G, dk, generator=g).to(dtype)
    q[..., 3], q[..., 4] = -q[..., 3].abs() - 0.1, q[..., 4].abs() + 0.1
    kc = torch.randn(B * ns, 2, page, dk, generator=g).to(dtype)
    table = torch.arange(B * ns, dtype=torch.int32).reshape(B, ns)
    lse = math.log(max(kl)) + torch.rand(T, 2 * G, generator=g)
    w = torch.rand(B, 2, max(kl), generator=g)
    args = dict(q=q.cuda(), page_table=table.cuda(), key_len=torch.tensor(kl, dtype=torch.int32).cuda(), max_len=max(kl),
                lse=lse.cuda(), cu_q=torch.tensor([sum(ql[:b]) for b in range(B + 1)], dtype=torch.int32).cuda(), max_q=max(ql))
    clean = wq.attention_weights_paged(k_cache=kc.cuda(), weights=w.cuda(), decay=0.5, **args).cpu()
    # (key, element, value): every score minus infinity, plus infinity, NaN; near the front, so that tokens see them
    bad = [(2, 3, math.inf), (5, 4, -math.inf), (11, 4, math.inf), (17, 0, math.nan), (18, 3, math.inf)]
    for b in range(B):
        for i, d, v in bad:
            kc[table[b, i // page], :, i % page, d] = v
    got = wq.attention_weights_paged(k_cache=kc.cuda(), weights=w.cuda(), decay=0.5, **args).cpu()
    for b in range(B):
        old = kl[b] - ql[b]
        for i, d, v in bad:
            if math.isnan(v):
                assert got[b, :, i].isnan().all()
            elif (d == 3) == (v > 0):  # no weight is added
                assert torch.equal(got[b, :, i], 0.5 * w[b, :, i] if i < old else torch.zeros(2))
            else:
                assert (got[b, :, i] == math.inf).all()
        for i, _, _ in bad:
            got[b, :, i] = clean[b, :, i]
    assert torch.equal(got, clean)
