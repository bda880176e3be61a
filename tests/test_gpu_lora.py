"""Low-rank adapters beside a shared projection on the GPU against a float64
definition.  Tolerances are derived in serve_ref."""
import math

import pytest
import torch

import serve_ref as R
from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def randn(*shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 7919 * len(shape) + sum(shape))
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def ids_of(T, n, seed=0, none=0.15):
    g = torch.Generator().manual_seed(seed + T)
    ids = torch.randint(0, n, (T,), generator=g)
    ids[torch.rand(T, generator=g) < none] = -1
    return ids.to(torch.int32).cuda()


def problem(T, H, N, r, n, dtype, ids=None, **kw):
    return dict(y=randn(T, N, dtype=dtype, seed=1), x=randn(T, H, dtype=dtype, seed=2),
                A=randn(n, r, H, dtype=dtype, seed=3, scale=H ** -0.5), B=randn(n, N, r, dtype=dtype, seed=4, scale=r ** -0.5),
                adapters=ids_of(T, n, **kw) if ids is None else ids, scales=0.5 + torch.arange(n).float().cuda() / n)


def check(a, ws=None):
    dtype = a["y"].dtype
    want, tol = R.lora(a["y"], a["x"], a["A"], a["B"], a["adapters"], a["scales"], dtype)
    st = wq.new_status()
    assert wq.lora_add(**a, ws=ws, status=st) is a["y"] and int(st) == 0
    R.check(a["y"], want, tol, "y")


CASES = [  # T, H, N, r, n, dtype
    (1, 8, 8, 8, 1, BF), (1, 256, 264, 16, 3, FP), (1, 7168, 1024, 16, 8, BF), (2, 104, 8, 128, 2, BF),
    (17, 512, 256, 16, 1, BF), (33, 264, 520, 24, 2, FP), (128, 1000, 1032, 16, 40, BF), (256, 256, 128, 64, 5, BF),
    (256, 136, 328, 32, 256, FP), (257, 512, 256, 8, 3, BF), (300, 128, 264, 128, 7, FP), (1024, 72, 80, 16, 300, BF),
    (1025, 256, 136, 64, 2, BF), (1500, 264, 200, 24, 9, FP), (2000, 128, 128, 128, 8192, BF), (3100, 192, 88, 40, 1, BF),
    (1100, 64, 64, 16, 1, FP), (1537, 200, 136, 16, 3, BF), (1536, 136, 72, 24, 40, FP), (577, 128, 200, 64, 5, FP),
    (289, 72, 136, 128, 2, BF), (4000, 64, 64, 32, 4000, BF),
]


@pytest.mark.parametrize("T,H,N,r,n,dtype", CASES)
def test_lora_add(T, H, N, r, n, dtype):
    check(problem(T, H, N, r, n, dtype))


@pytest.mark.parametrize("T", [40, 700, 1300, 2500])
def test_runs_of_tokens_no_scales_and_strides(T):
    H, N, r, n = 128, 136, 16, 4
    ids = torch.tensor([-1, 2, 0, 3, 2]).repeat_interleave(-(-T // 5))[:T].to(torch.int32).cuda()
    a = problem(T, H, N, r, n, BF, ids)
    a["scales"] = None
    wide_x, wide_y = randn(T, H + 40, dtype=BF, seed=6), torch.full((T, N + 24), 7.0, dtype=BF).cuda()
    wide_y[:, 8:8 + N] = a["y"]
    b = {**a, "x": wide_x[:, 16:16 + H], "y": wide_y[:, 8:8 + N]}
    b["x"].copy_(a["x"])
    check(a)
    check(b)
    assert torch.equal(a["y"], b["y"]) and (wide_y[:, :8] == 7).all() and (wide_y[:, 8 + N:] == 7).all()


@pytest.mark.parametrize("T", [30, 600, 2300])
def test_tokens_without_an_adapter_stay_as_they_are(T):
    a = problem(T, 64, 64, 8, 3, BF, none=0.5)
    off = a["adapters"] < 0
    a["x"][off], a["y"][off] = math.nan, math.nan
    bits = a["y"][off].view(torch.int16).clone()
    wq.lora_add(**a)
    assert torch.equal(a["y"][off].view(torch.int16), bits) and a["y"][~off].isfinite().all()
    a["adapters"].fill_(-1)
    before = a["y"].clone()
    wq.lora_add(**a)
    assert torch.equal(a["y"].view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("T", [30, 600, 2300])
def test_bad_adapters_are_reported_and_skipped(T):
    a = problem(T, 64, 64, 8, 3, BF, none=0.0)
    a["adapters"][5], a["adapters"][T - 1] = 3, 10 ** 9
    b = {**a, "y": a["y"].clone(), "adapters": a["adapters"].clone()}
    b["adapters"][5] = b["adapters"][T - 1] = -1
    st = wq.new_status()
    wq.lora_add(**a, status=st)
    assert int(st) == -6
    check(b)
    assert torch.equal(a["y"], b["y"])


def test_a_row_does_not_depend_on_its_neighbours_or_the_run():
    a = problem(200, 512, 256, 16, 4, BF)
    y0 = a["y"].clone()
    wq.lora_add(**a)
    for _ in range(3):
        b = {**a, "y": y0.clone(), "adapters": a["adapters"].clone()}
        wq.lora_add(**b)
        assert torch.equal(a["y"], b["y"])
    b["y"], b["adapters"][:100] = y0.clone(), -1
    wq.lora_add(**b)
    assert torch.equal(b["y"][100:], a["y"][100:]) and torch.equal(b["y"][:100], y0[:100])
    c = problem(3000, 128, 128, 64, 5, BF)
    y0 = c["y"].clone()
    wq.lora_add(**c)
    for _ in range(3):
        b = {**c, "y": y0.clone()}
        wq.lora_add(**b)
        assert torch.equal(c["y"], b["y"])


@pytest.mark.parametrize("size", [1e4, 1e-4])
@pytest.mark.parametrize("T", [5, 1100, 2100])
def test_fp16_sums_past_its_range(size, T):
    """x A^T far past fp16's largest, and below its smallest, with B to match."""
    a = problem(T, 512, 64, 8, 2, FP)
    a["x"] = randn(T, 512, dtype=FP, seed=7, scale=max(size, 1.0))
    a["A"] = randn(2, 8, 512, dtype=FP, seed=8, scale=10.0 if size > 1 else size)
    a["B"] = randn(2, 64, 8, dtype=FP, seed=9, scale=1e-6 if size > 1 else 100.0)
    check(a)


@pytest.mark.parametrize("T", [9, 1100, 2100])
def test_nonfinite_values_stay_in_their_rows(T):
    a = problem(T, 64, 64, 8, 1, BF, torch.zeros(T, dtype=torch.int32).cuda())
    y0, x0 = a["y"].clone(), a["x"].clone()
    a["x"][3, 5], a["x"][4, 6], a["y"][6, 1] = math.nan, math.inf, math.inf
    wq.lora_add(**a)
    clean = {**a, "y": y0, "x": x0}
    wq.lora_add(**clean)
    assert a["y"][3].isnan().all() and not a["y"][4].isfinite().any() and a["y"][6, 1] == math.inf
    rest = torch.ones(T, dtype=torch.bool)
    rest[[3, 4, 6]] = False
    assert torch.equal(a["y"][rest], clean["y"][rest])


@pytest.mark.parametrize("T", [20, 500, 2200])
def test_replayed_in_a_graph_with_other_adapters(T):
    a = problem(T, 128, 128, 16, 6, BF)
    y0, ws = a["y"].clone(), wq.lora_add_workspace(a["y"], a["x"], a["A"])
    wq.lora_add(**a, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        wq.lora_add(**a, ws=ws)
    a["adapters"].copy_(ids_of(T, 6, seed=5, none=0.4))
    a["y"].copy_(y0)
    graph.replay()
    got = a["y"].clone()
    a["y"].copy_(y0)
    check(a, ws)
    assert torch.equal(got, a["y"])


def test_beside_the_int8_projection():
    """The run it belongs to: the shared W8A8 projection of a mixed batch, each
    request's adapter added to it."""
    T, H, N, r, n = 96, 512, 384, 16, 5
    a = problem(T, H, N, r, n, BF)
    W, sw = wq.quantize_weight(randn(N, H, dtype=BF, seed=11, scale=0.05), "channel")
    y = wq.linear_w8a8(a["x"], W, sw)
    a["y"] = y
    base = y.clone()
    check(a)
    off = a["adapters"] < 0
    assert torch.equal(y[off], base[off]) and not torch.equal(y[~off], base[~off])
