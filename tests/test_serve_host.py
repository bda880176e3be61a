"""Host-side refusals of the serving entry points: no GPU is touched."""
import ctypes

import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding, build_lib

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
FAKE = 4096  # never dereferenced: argument checks fail first


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.lib()


def norm(lib, **kw):
    a = dict(block=FAKE, ldb=64, residual=FAKE, ldr=64, gate=None, ldg=0, scale=1.0, post=1, pw=FAKE, pb=None, pre=1,
             qw=FAKE, qb=None, eps=1e-6, T=4, H=64, dtype=0, x_out=FAKE, ldx=64, y=FAKE, ldy=64)
    a.update(kw)
    return lib.wq_block_norm(*a.values(), None)


def test_block_norm_refusals(lib):
    for kw in (dict(T=-1), dict(H=0), dict(dtype=3), dict(post=3), dict(pre=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(block=None), dict(x_out=None, y=None), dict(ldb=63), dict(ldr=1), dict(gate=FAKE, ldg=8),
               dict(ldx=0), dict(ldy=63)):
        assert norm(lib, **kw) == INVALID, kw
    assert norm(lib, H=32769, ldb=40000, ldr=40000, ldx=40000, ldy=40000) == UNSUPPORTED
    assert norm(lib, block=FAKE + 1) == UNSUPPORTED
    assert norm(lib, dtype=2, block=FAKE + 2) == UNSUPPORTED
    assert norm(lib, T=0, block=None, x_out=None, y=None) == 0


def test_rope_table_refusals(lib):
    ok = dict(table=FAKE, n=10, rot=64, base=1e4, scaling=0, factor=1.0, trained=0.0, fast=32.0, slow=1.0, m=0.0)
    call = lambda **kw: lib.wq_rope_table(*{**ok, **kw}.values(), None)
    for kw in (dict(n=-1), dict(rot=0), dict(rot=63), dict(base=1.0), dict(scaling=4), dict(factor=0.5), dict(m=-1.0),
               dict(table=None), dict(scaling=3, trained=0.0), dict(scaling=3, trained=9.0, slow=0.0),
               dict(scaling=3, trained=9.0, fast=0.5), dict(scaling=2, rot=2), dict(base=float("nan"))):
        assert call(**kw) == INVALID, kw
    assert call(rot=1026) == UNSUPPORTED
    assert call(n=0, table=None) == 0


def test_rope_refusals(lib):
    ok = dict(x=FAKE, xt=128, xh=64, pos=FAKE, table=FAKE, n=10, T=4, heads=2, D=64, rot=64, layout=0, inv=0, dtype=0,
              out=FAKE, ot=128, oh=64)
    call = lambda **kw: lib.wq_rope(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(heads=-1), dict(rot=66), dict(rot=7), dict(rot=0), dict(layout=2), dict(inv=2),
               dict(dtype=5), dict(x=None), dict(out=None), dict(pos=None), dict(table=None), dict(xt=-1), dict(oh=-8)):
        assert call(**kw) == INVALID, kw
    assert call(x=FAKE + 1) == UNSUPPORTED and call(table=FAKE + 4) == UNSUPPORTED
    assert call(T=0, x=None) == 0 and call(heads=0, x=None) == 0


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, k_page=2048, k_head=1024, k_token=64, v_page=2048, v_head=1024, v_token=64, num_pages=8,
             page_size=16, heads=2, dk=64, dv=64, dtype=0)
    c.update(kw)
    return ctypes.pointer(binding._PagedCache(*c.values()))


def test_append_refusals(lib):
    ok = dict(q=FAKE, qt=256, qh=64, nq=4, k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, pos=FAKE, slots=FAKE, table=FAKE,
              n=10, T=4, rot=64, layout=0, cache=cache(), qo=FAKE, qot=256, qoh=64)
    call = lambda **kw: lib.wq_rope_append_paged(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(rot=66), dict(rot=3), dict(layout=9), dict(cache=None), dict(k=None), dict(v=None),
               dict(slots=None), dict(pos=None), dict(table=None), dict(qo=None), dict(nq=0), dict(kt=-1),
               dict(cache=cache(dtype=2)), dict(cache=cache(page_size=0)), dict(cache=cache(k=None)),
               dict(cache=cache(num_pages=-1)), dict(cache=cache(heads=0))):
        assert call(**kw) == INVALID, kw
    assert call(k=FAKE + 1) == UNSUPPORTED
    assert call(T=0, k=None) == 0


def test_attention_refusals(lib):
    ok = dict(q=FAKE, qt=512, qh=64, T=4, B=2, cu=FAKE, max_q=2, nq=8, cache=cache(), pp=FAKE, P=100, pt=FAKE, ldt=4,
              sl=FAKE, S=64, scale=0.125, out=FAKE, ot=512, oh=64, lse=None, ws=FAKE, n=1 << 30)
    call = lambda **kw: lib.wq_attention_shared_prefix(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_q=0), dict(nq=0), dict(nq=7), dict(cache=None), dict(P=-1),
               dict(S=-1), dict(q=None), dict(out=None), dict(pp=None), dict(pt=None), dict(sl=None), dict(S=65),
               dict(cu=None, max_q=1), dict(B=0), dict(qt=-8), dict(ot=-2), dict(ldt=-1), dict(cache=cache(v=None))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(nq=258, cache=cache()), dict(cache=cache(dk=136)), dict(cache=cache(dv=60)), dict(cache=cache(k_token=65)),
               dict(qt=510), dict(oh=63), dict(q=FAKE + 8), dict(cache=cache(k=FAKE + 8)), dict(out=FAKE + 2), dict(qh=0), dict(ot=0),
               dict(T=1 << 24), dict(P=1 << 30)):
        assert call(**kw) == UNSUPPORTED, kw
    size = lambda **kw: lib.wq_attention_shared_prefix_workspace_size(
        *[{**ok, **kw}[k] for k in ("T", "B", "max_q", "nq", "cache", "P", "S")])
    need = size()
    assert need >= 2 * 4 * 8 * 65 * 4  # a part for the prefix and one for the suffixes, and their statistics
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE
    assert size(T=0) == 0 and size(nq=7) == 0
    assert call(T=0, q=None) == 0


def test_binding_refusals(lib):
    """Shapes, types and devices are checked before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(binding.WQError, match="CUDA"):
        binding.block_norm(x)
    with pytest.raises(binding.WQError, match="CUDA"):
        binding.rope(x.view(4, 1, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2))
    with pytest.raises(binding.WQError, match="CUDA"):
        binding.attention_shared_prefix(x.view(4, 1, 64), x.view(1, 1, 4, 64), x.view(1, 1, 4, 64), None, 0,
                                        torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 4)
