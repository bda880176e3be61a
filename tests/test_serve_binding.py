"""What the torch binding of the serving operators refuses and passes on, with
stand-ins for CUDA tensors and for the library: no GPU is touched."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class Cuda:
    """As much of a CUDA tensor as the binding asks for."""

    def __init__(self, *shape, dtype=BF, stride=None, device=0):
        self.shape, self.dtype, self._device = torch.Size(shape), dtype, device
        self._stride = torch.empty(shape, device="meta").stride() if stride is None else stride

    is_cuda = property(lambda self: self._device >= 0)
    device = property(lambda self: torch.device("cuda", self._device) if self._device >= 0 else torch.device("cpu"))
    get_device = lambda self: self._device
    stride = lambda self, dim=None: self._stride if dim is None else self._stride[dim]
    dim = lambda self: len(self.shape)
    numel = lambda self: self.shape.numel()
    element_size = lambda self: torch.empty((), dtype=self.dtype).element_size()
    data_ptr = lambda self: 4096
    is_contiguous = lambda self: torch.empty_strided(self.shape, self._stride, device="meta").is_contiguous()


@pytest.fixture
def calls(monkeypatch):
    """The library calls made: (name, arguments)."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or 0

    monkeypatch.setattr(wq, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 77, raising=False)
    return made


def norm_args(**kw):
    a = dict(block=Cuda(4, 64), residual=Cuda(4, 64), gate=Cuda(64), post="layer", post_weight=Cuda(64),
             post_bias=Cuda(64), pre="layer", pre_weight=Cuda(64), pre_bias=Cuda(64), x_out=Cuda(4, 64), y=Cuda(4, 64))
    return {**a, **kw}


def rope_args(**kw):
    a = dict(x=Cuda(4, 2, 64), positions=Cuda(4, dtype=I32), table=Cuda(9, 32, 2, dtype=F32), out=Cuda(4, 2, 64),
             status=Cuda(1, dtype=I32))
    return {**a, **kw}


def append_args(**kw):
    a = dict(k=Cuda(4, 2, 64), v=Cuda(4, 2, 32), positions=Cuda(4, dtype=I32), slots=Cuda(4, dtype=I64),
             table=Cuda(9, 32, 2, dtype=F32), k_cache=Cuda(8, 2, 16, 64), v_cache=Cuda(8, 2, 16, 32), q=Cuda(4, 6, 64),
             q_out=Cuda(4, 6, 64), status=Cuda(1, dtype=I32))
    return {**a, **kw}


def attention_args(**kw):
    a = dict(q=Cuda(4, 6, 64), k_cache=Cuda(8, 2, 16, 64), v_cache=Cuda(8, 2, 16, 32), prefix_pages=Cuda(2, dtype=I32),
             prefix_len=20, page_table=Cuda(3, 2, dtype=I32), suffix_len=Cuda(3, dtype=I32), max_suffix=30,
             cu_q=Cuda(4, dtype=I32), max_q=2, out=Cuda(4, 6, 32), lse=Cuda(4, 6, dtype=F32),
             ws=Cuda(1 << 20, dtype=torch.uint8), status=Cuda(1, dtype=I32))
    return {**a, **kw}


ENTRIES = [(wq.block_norm, norm_args), (wq.rope, rope_args), (wq.rope_append_paged, append_args),
           (wq.attention_shared_prefix, attention_args)]
TENSORS = [(f, args, name) for f, args in ENTRIES for name, v in args().items()
           if isinstance(v, Cuda) and name not in ("status", "ws")]


@pytest.mark.parametrize("f,args", ENTRIES)
def test_good_arguments_reach_the_library(calls, f, args):
    f(**args())
    assert [name for name, _ in calls] == ["wq_" + f.__name__] and 77 in calls[0][1]


@pytest.mark.parametrize("f,args,name", TENSORS)
@pytest.mark.parametrize("device", [-1, 1])
def test_every_tensor_has_to_be_on_the_current_device(calls, f, args, name, device):
    a = args()
    t = a[name]
    a[name] = Cuda(*t.shape, dtype=t.dtype, device=device)
    with pytest.raises(wq.WQError, match="CUDA|cuda"):
        f(**a)
    assert not calls


BAD_BUFFERS = [(f, args, name, bad) for f, args in ENTRIES for name in ("status", "ws") if name in args()
               for bad in [dict(device=-1), dict(device=1), dict(stride=(0,))] +
               ([dict(dtype=F32), dict(shape=(0,))] if name == "status" else [])]


@pytest.mark.parametrize("f,args,name,bad", BAD_BUFFERS)
def test_buffers_that_kernels_write_are_checked(calls, f, args, name, bad):
    """A status in host memory or a workspace that repeats one byte would be
    written at an address, or to a length, that is not there."""
    a = args()
    kw = {**dict(shape=(4096,), dtype=a[name].dtype), **bad}
    a[name] = Cuda(*kw.pop("shape"), **kw)
    with pytest.raises(wq.WQError, match=name):
        f(**a)
    assert not calls


def test_a_workspace_counts_in_bytes(calls):
    wq.attention_shared_prefix(**attention_args(ws=Cuda(1234, dtype=F32)))
    assert calls[0][1][-3] == 4 * 1234


@pytest.mark.parametrize("f,args", ENTRIES)
def test_another_current_device_is_refused(calls, monkeypatch, f, args):
    """The library launches on the current device: tensors that agree with one
    another but not with it would be read from the wrong one."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(wq.WQError, match="current device"):
        f(**args())
    assert not calls


@pytest.mark.parametrize("f,args", ENTRIES[2:])
@pytest.mark.parametrize("shape", [(8, 2, 16, 32, 2), (8, 2, 16), (8, 2, 15, 32), (7, 2, 16, 32), (8, 3, 16, 32)])
def test_v_cache_has_the_pages_of_k_cache(calls, f, args, shape):
    """A fifth dimension would make the fourth one's elements lie apart."""
    with pytest.raises(wq.WQError, match="v_cache"):
        f(**args(v_cache=Cuda(*shape)))
    assert not calls


def passed(calls, f, **kw):
    del calls[:]
    f(**kw)
    return [a for a in calls[0][1] if isinstance(a, int)]


def test_dimensions_of_one_element_may_have_any_stride(calls):
    """As torch.empty(64, 1).t() has: the call is that with a contiguous tensor."""
    one = lambda **kw: norm_args(block=Cuda(1, 64), residual=Cuda(1, 64), x_out=Cuda(1, 64), y=Cuda(1, 64), **kw)
    want = passed(calls, wq.block_norm, **one())
    for name in ("block", "residual", "x_out", "y"):
        assert passed(calls, wq.block_norm, **{**one(), name: Cuda(1, 64, stride=(1, 1))}) == want
        assert passed(calls, wq.block_norm, **{**one(), name: Cuda(1, 64, stride=(0, 1))}) == want
    single = lambda **kw: attention_args(q=Cuda(1, 1, 64), k_cache=Cuda(8, 1, 16, 64), v_cache=Cuda(8, 1, 16, 32),
                                         page_table=Cuda(1, 2, dtype=I32), suffix_len=Cuda(1, dtype=I32),
                                         cu_q=Cuda(2, dtype=I32), out=Cuda(1, 1, 32), lse=None, **kw)
    want = passed(calls, wq.attention_shared_prefix, **single())
    for kw in (dict(page_table=Cuda(1, 2, dtype=I32, stride=(1, 1))), dict(q=Cuda(1, 1, 64, stride=(3, 5, 1))),
               dict(out=Cuda(1, 1, 32, stride=(0, 7, 1)))):
        assert passed(calls, wq.attention_shared_prefix, **{**single(), **kw}) == want


def test_other_strides_go_as_they_are(calls):
    wq.block_norm(**norm_args(block=Cuda(4, 64, stride=(80, 1))))
    assert calls[0][1][1] == 80
    del calls[:]
    wq.rope(**rope_args(x=Cuda(4, 2, 64, stride=(900, 200, 1))))
    assert calls[0][1][1:3] == (900, 200)
    del calls[:]
    wq.rope(**rope_args(x=Cuda(4, 1, 64, stride=(900, 7, 1)), out=Cuda(4, 1, 64)))
    assert calls[0][1][1:3] == (900, 64)


@pytest.mark.parametrize("f,args,name", [(wq.rope_append_paged, append_args, "positions"),
                                         (wq.attention_shared_prefix, attention_args, "prefix_pages")])
def test_a_missing_tensor_is_named(calls, f, args, name):
    with pytest.raises(wq.WQError, match=name):
        f(**args(**{name: None}))
    assert not calls
