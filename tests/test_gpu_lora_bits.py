"""How many bits of x A^T reach the second product of the adapters: problems
whose every product and sum is a whole number below 2^24, which float32 holds.
Then nothing but y's own rounding is left, and y has to be equal to the rounded
whole number.

Rows of A come in pairs that differ by one in one place, and B takes a pair's
difference: each of the two is a number of 17 to 20 bits, what is left of them
one of 7.  An operand that drops bits of the first shows in the second."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def whole(T, H, N, r, n, dtype):
    g = torch.Generator().manual_seed(T + H + N + r)

    def ints(*shape, most):
        return torch.randint(-most, most + 1, shape, generator=g).double()

    x, A = ints(T, H, most=127), ints(n, r, H, most=126)
    A[:, 1::2] = A[:, 0::2]
    at = torch.randint(0, H, (n, r // 2, 1), generator=g)
    A[:, 1::2].scatter_add_(2, at, torch.ones(n, r // 2, 1, dtype=torch.float64))
    b = ints(n, N, r // 2, most=1)
    B = torch.stack([b, -b], -1).reshape(n, N, r)
    ids, y = torch.randint(0, n, (T,), generator=g), ints(T, N, most=100)
    h = torch.stack([A[a] @ x[t] for t, a in enumerate(ids.tolist())])
    d = torch.stack([B[a] @ h[t] for t, a in enumerate(ids.tolist())])
    # fp16 keeps 22 bits counted from a row's largest; a pair's sum is small before the next pair is added
    assert h.abs().max() < 2 ** 21 and (y + d).abs().max() < 2 ** 16
    want = (y + d).to(dtype)
    y, x, A, B = (t.to(dtype).cuda() for t in (y, x, A, B))
    return dict(y=y, x=x, A=A, B=B, adapters=ids.to(torch.int32).cuda()), want


@pytest.mark.parametrize("T,H,N,r,n", [
    (1, 4096, 64, 16, 1), (50, 4096, 72, 24, 3), (300, 4096, 64, 64, 2), (40, 2048, 64, 128, 2), (20, 2048, 520, 32, 2),
    (1600, 4096, 136, 24, 3), (1540, 4096, 64, 16, 2), (700, 4096, 72, 64, 2), (600, 4096, 136, 128, 2), (1300, 2048, 264, 32, 1)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_no_bit_of_the_first_product_is_lost(T, H, N, r, n, dtype):
    a, want = whole(T, H, N, r, n, dtype)
    wq.lora_add(**a)
    assert torch.equal(a["y"].cpu(), want)
