"""Infinite values of x in the adapters, at ranks that the kernels pad: what the
formula gives, wherever the padding ends."""
import math

import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu


def randn(g, *shape):
    return torch.randn(shape, generator=g)


@pytest.mark.parametrize("T,r", [(1, 8), (9, 8), (9, 16), (9, 24), (9, 40), (9, 64), (9, 72), (9, 128), (300, 8), (700, 24),
                                 (1600, 8), (1600, 16), (1600, 24), (1000, 40), (1000, 64), (700, 72), (700, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_infinite_x(T, r, dtype):
    H, N, g = 72, 136, torch.Generator().manual_seed(T + r)
    A, B = randn(g, 1, r, H).to(dtype), (randn(g, 1, N, r).abs() + 0.1).to(dtype)
    A[0, :, 5] = A[0, :, 5].abs() + 0.1  # sums of one sign for this element of x, of both signs for the next
    x, y = randn(g, T, H).to(dtype), randn(g, T, N).to(dtype)
    clean = y.cuda()
    ids = torch.zeros(T, dtype=torch.int32).cuda()
    wq.lora_add(clean, x.cuda(), A.cuda(), B.cuda(), ids)
    rows = {T - 1: (5, math.inf)} if T == 1 else {3: (5, math.inf), 4: (5, -math.inf), T - 1: (6, math.inf), 6: (7, math.nan)}
    for t, (i, v) in rows.items():
        x[t, i] = v
    got = y.cuda()
    wq.lora_add(got, x.cuda(), A.cuda(), B.cuda(), ids)
    h = x.double() @ A[0].double().T
    want = y.double() + h @ B[0].double().T
    got, clean = got.cpu(), clean.cpu()
    for t in range(T):
        if t in rows:
            # of both signs: inf - inf, which is NaN, wherever a row of A^T has both
            assert torch.equal(got[t].isnan(), want[t].isnan()) and torch.equal(got[t].isinf(), want[t].isinf())
            assert torch.equal(got[t][want[t].isinf()].double(), want[t][want[t].isinf()])
    rest = [t for t in range(T) if t not in rows]
    assert torch.equal(got[rest], clean[rest])
