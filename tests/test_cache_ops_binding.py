"""What the torch binding of head norms, attention weights, eviction and adapters
refuses and passes on, with stand-ins for CUDA tensors and for the library: no
GPU is touched."""
import pytest
import torch

from test_serve_binding import Cuda, calls  # noqa: F401  (calls is a fixture)
from w8a8_int8_quantized_token_gb300 import binding as wq

BF, I32, I64, F32, U8 = torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.uint8


def head_args(**kw):
    a = dict(x=Cuda(4, 2, 64), weight=Cuda(64), positions=Cuda(4, dtype=I32), table=Cuda(9, 32, 2, dtype=F32),
             out=Cuda(4, 2, 64), status=Cuda(1, dtype=I32))
    return {**a, **kw}


def append_args(**kw):
    a = dict(k=Cuda(4, 2, 64), v=Cuda(4, 2, 32), positions=Cuda(4, dtype=I32), slots=Cuda(4, dtype=I64),
             table=Cuda(9, 32, 2, dtype=F32), k_cache=Cuda(8, 2, 16, 64), v_cache=Cuda(8, 2, 16, 32), k_weight=Cuda(64),
             q=Cuda(4, 6, 64), q_weight=Cuda(64), q_out=Cuda(4, 6, 64), status=Cuda(1, dtype=I32))
    return {**a, **kw}


def weight_args(**kw):
    a = dict(q=Cuda(4, 6, 64), k_cache=Cuda(8, 2, 16, 64), page_table=Cuda(3, 2, dtype=I32), key_len=Cuda(3, dtype=I32),
             max_len=30, lse=Cuda(4, 6, dtype=F32), weights=Cuda(3, 2, 32, dtype=F32), cu_q=Cuda(4, dtype=I32), max_q=2,
             ws=Cuda(1 << 20, dtype=U8), status=Cuda(1, dtype=I32))
    return {**a, **kw}


def evict_args(**kw):
    a = dict(weights=Cuda(3, 2, 32, dtype=F32), k_cache=Cuda(8, 2, 16, 64), v_cache=Cuda(8, 2, 16, 32),
             page_table=Cuda(3, 2, dtype=I32), key_len=Cuda(3, dtype=I32), max_len=30, budget=20, recent=4, first=2,
             out_table=Cuda(3, 2, dtype=I32), weights_out=Cuda(3, 2, 20, dtype=F32), new_len=Cuda(3, dtype=I32),
             kept=Cuda(3, 2, 20, dtype=I32), ws=Cuda(1 << 20, dtype=U8), status=Cuda(1, dtype=I32))
    return {**a, **kw}


def lora_args(**kw):
    a = dict(y=Cuda(4, 48), x=Cuda(4, 64), A=Cuda(3, 8, 64), B=Cuda(3, 48, 8), adapters=Cuda(4, dtype=I32),
             scales=Cuda(3, dtype=F32), ws=Cuda(1 << 20, dtype=U8), status=Cuda(1, dtype=I32))
    return {**a, **kw}


ENTRIES = [(wq.head_norm_rope, head_args), (wq.head_norm_rope_append_paged, append_args),
           (wq.attention_weights_paged, weight_args), (wq.evict_paged, evict_args), (wq.lora_add, lora_args)]
TENSORS = [(f, args, name) for f, args in ENTRIES for name, v in args().items()
           if isinstance(v, Cuda) and name not in ("status", "ws")]


@pytest.mark.parametrize("f,args", ENTRIES)
def test_good_arguments_reach_the_library(calls, f, args):  # noqa: F811
    f(**args())
    assert [name for name, _ in calls] == ["wq_" + f.__name__] and 77 in calls[0][1]
    assert len(calls[0][1]) == len(wq._SIGS["wq_" + f.__name__][1])


@pytest.mark.parametrize("f,args,name", TENSORS)
@pytest.mark.parametrize("bad", ["host", "device", "type"])
def test_every_tensor_is_checked(calls, f, args, name, bad):  # noqa: F811
    a = args()
    t = a[name]
    dtype = (I32 if t.dtype is BF else BF) if bad == "type" else t.dtype
    a[name] = Cuda(*t.shape, dtype=dtype, device={"host": -1, "device": 1, "type": 0}[bad])
    with pytest.raises(wq.WQError, match="CUDA|cuda" if bad != "type" else "must be"):
        f(**a)
    assert not calls


@pytest.mark.parametrize("f,args,name", TENSORS)
def test_every_shape_is_checked(calls, f, args, name):  # noqa: F811
    a = args()
    t = a[name]
    for dim in range(len(t.shape)):
        if name in ("x", "k_cache", "k", "q", "B") and dim in (0, 1):
            continue  # the sizes that the call goes by
        if (f, name, dim) == (wq.evict_paged, "k_cache", 3) or (name, dim) in (("k_cache", 2), ("A", 1), ("table", 0), ("table", 1), ("v_cache", 3)):
            continue
        shape = list(t.shape)
        shape[dim] -= 3 if (name, dim) == ("weights", 2) else 1
        with pytest.raises(wq.WQError):
            f(**{**a, name: Cuda(*shape, dtype=t.dtype)})
    with pytest.raises(wq.WQError):
        f(**{**a, name: Cuda(*t.shape, 1, dtype=t.dtype)})
    assert not calls


@pytest.mark.parametrize("f,args", ENTRIES)
def test_another_current_device_is_refused(calls, monkeypatch, f, args):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(wq.WQError, match="current device"):
        f(**args())
    assert not calls


@pytest.mark.parametrize("f,args,name,bad", [
    (f, args, name, bad) for f, args in ENTRIES for name in ("status", "ws") if name in args()
    for bad in [dict(device=-1), dict(device=1), dict(stride=(0,))] +
    ([dict(dtype=F32), dict(shape=(0,))] if name == "status" else [])])
def test_buffers_that_kernels_write_are_checked(calls, f, args, name, bad):  # noqa: F811
    a = args()
    kw = {**dict(shape=(4096,), dtype=a[name].dtype), **bad}
    a[name] = Cuda(*kw.pop("shape"), **kw)
    with pytest.raises(wq.WQError, match=name):
        f(**a)
    assert not calls


@pytest.mark.parametrize("f,kw,match", [
    (wq.head_norm_rope, head_args(positions=None), "positions"),
    (wq.head_norm_rope_append_paged, append_args(positions=None), "positions"),
    (wq.attention_weights_paged, weight_args(max_len=33), "max_len"),
    (wq.attention_weights_paged, weight_args(max_q=None), "max_q"),
    (wq.attention_weights_paged, weight_args(cu_q=None), "evenly"),
    (wq.evict_paged, evict_args(max_len=33), "page_table"),
    (wq.evict_paged, evict_args(out_table=Cuda(3, 1, dtype=I32)), "out_table"),
])
def test_what_does_not_fit_is_named(calls, f, kw, match):  # noqa: F811
    with pytest.raises(wq.WQError, match=match):
        f(**kw)
    assert not calls


def test_optional_tensors_may_be_left_out(calls):  # noqa: F811
    wq.head_norm_rope(**head_args(weight=None, table=None, positions=None, status=None))
    wq.head_norm_rope_append_paged(**append_args(q=None, q_weight=None, q_out=None, k_weight=None, table=None, positions=None))
    wq.evict_paged(**evict_args(out_table=None, weights_out=None))
    wq.lora_add(**lora_args(scales=None))
    assert len(calls) == 4


def test_strides_go_as_they_are(calls):  # noqa: F811
    wq.evict_paged(**evict_args(weights=Cuda(3, 2, 32, dtype=F32, stride=(900, 100, 1))))
    assert calls[0][1][1:3] == (900, 100)
    wq.lora_add(**lora_args(x=Cuda(4, 64, stride=(80, 1)), y=Cuda(4, 48, stride=(96, 1))))
    assert calls[1][1][1] == 80 and calls[1][1][13] == 96
    for name in ("A", "B"):
        t = lora_args()[name]
        with pytest.raises(wq.WQError, match=name):
            wq.lora_add(**lora_args(**{name: Cuda(*t.shape, stride=(2 * t.shape[1] * t.shape[2], t.shape[2], 1))}))
