"""Host-side refusals of head norms, attention weights, eviction and adapters at
the C interface: no GPU is touched."""
import ctypes

import pytest

from w8a8_int8_quantized_token_gb300 import binding, build_lib

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5
FAKE = 1 << 20  # never dereferenced: argument checks fail first


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.lib()


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, k_page=2048, k_head=1024, k_token=64, v_page=2048, v_head=1024, v_token=64, num_pages=8,
             page_size=16, heads=2, dk=64, dv=64, dtype=0)
    c.update(kw)
    return ctypes.pointer(binding._PagedCache(*c.values()))


def test_head_norm_refusals(lib):
    ok = dict(x=FAKE, xt=128, xh=64, w=FAKE, eps=1e-6, pos=FAKE, table=FAKE, n=10, T=4, heads=2, D=64, rot=64, layout=0,
              dtype=0, out=FAKE, ot=128, oh=64)
    call = lambda **kw: lib.wq_head_norm_rope(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(heads=-1), dict(rot=66), dict(rot=7), dict(rot=-2), dict(D=0, rot=0), dict(layout=2),
               dict(dtype=5), dict(x=None), dict(out=None), dict(pos=None), dict(table=None), dict(xt=-1), dict(oh=-8),
               dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 1), dict(w=FAKE + 1), dict(out=FAKE + 1), dict(dtype=2, x=FAKE + 2), dict(table=FAKE + 4),
               dict(T=1 << 31), dict(D=16386, rot=64), dict(heads=65537)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, x=None) == 0 and call(heads=0, x=None) == 0


def test_head_norm_append_refusals(lib):
    ok = dict(q=FAKE, qt=256, qh=64, nq=4, qw=FAKE, k=FAKE, kt=128, kh=64, kw=FAKE, v=FAKE, vt=128, vh=64, eps=1e-6,
              pos=FAKE, slots=FAKE, table=FAKE, n=10, T=4, rot=64, layout=0, cache=cache(), qo=FAKE, qot=256, qoh=64)
    call = lambda **kw: lib.wq_head_norm_rope_append_paged(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(rot=66), dict(rot=3), dict(layout=9), dict(cache=None), dict(k=None), dict(v=None),
               dict(slots=None), dict(pos=None), dict(table=None), dict(qo=None), dict(nq=0), dict(kt=-1), dict(eps=-1.0),
               dict(cache=cache(dtype=2)), dict(cache=cache(page_size=0)), dict(cache=cache(k=None)),
               dict(cache=cache(num_pages=-1)), dict(cache=cache(heads=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(k=FAKE + 1), dict(qw=FAKE + 1), dict(kw=FAKE + 1), dict(table=FAKE + 4)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=0, k=None) == 0


def test_attention_weights_refusals(lib):
    ok = dict(q=FAKE, qt=512, qh=64, T=400, B=2, cu=FAKE, max_q=300, nq=8, cache=cache(), pt=FAKE, ldt=40, kl=FAKE, L=640,
              scale=0.125, lse=FAKE, decay=1.0, w=FAKE, ws_=2000, wh=640, ws=FAKE, n=1 << 30)
    call = lambda **kw: lib.wq_attention_weights_paged(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_q=0), dict(nq=0), dict(nq=7), dict(cache=None), dict(L=-1),
               dict(q=None), dict(lse=None), dict(w=None), dict(pt=None), dict(kl=None), dict(L=641), dict(cu=None),
               dict(qt=-8), dict(ldt=-1), dict(cache=cache(k=None)), dict(wh=639), dict(ws_=1279), dict(wh=1000, ws_=700),
               dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf")), dict(scale=0.0), dict(wh=-640)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(nq=258), dict(cache=cache(dk=136)), dict(cache=cache(dk=60)), dict(cache=cache(k_token=65)), dict(qt=510),
               dict(q=FAKE + 8), dict(cache=cache(k=FAKE + 8)), dict(qh=0), dict(qt=0), dict(T=1 << 24), dict(w=FAKE + 2),
               dict(lse=FAKE + 1)):
        assert call(**kw) == UNSUPPORTED, kw
    size = lambda **kw: lib.wq_attention_weights_paged_workspace_size(
        *[{**ok, **kw}[k] for k in ("T", "B", "max_q", "nq", "cache", "L")])
    assert size() >= 2 * 256 * 4 and size(max_q=1, T=2) == 0 and size(nq=7) == 0
    assert call(n=size() - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE
    assert call(B=0, kl=None) == 0 and call(L=0, pt=None) == 0


def test_evict_refusals(lib):
    ok = dict(w=FAKE, ws_=2000, wh=640, cache=cache(), B=2, pt=FAKE, ldt=40, kl=FAKE, L=640, budget=100, recent=10, first=4,
              ot=FAKE * 2, ldo=7, wo=FAKE * 3, os=400, oh=100, nl=FAKE * 4, kept=FAKE, ws=FAKE, n=1 << 30)
    call = lambda **kw: lib.wq_evict_paged(*{**ok, **kw}.values(), None, None)
    for kw in (dict(B=-1), dict(L=-1), dict(budget=0), dict(recent=-1), dict(first=-1), dict(recent=97), dict(cache=None),
               dict(cache=cache(v=None)), dict(w=None), dict(wo=None), dict(pt=None), dict(kl=None), dict(nl=None),
               dict(kept=None), dict(L=641), dict(ldo=6), dict(wh=639), dict(oh=99), dict(os=199), dict(ws_=-1),
               dict(wo=FAKE, os=2000, oh=700), dict(nl=FAKE), dict(nl=FAKE + 4), dict(kl=FAKE * 4 + 4), dict(ldt=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(cache=cache(dk=16386)), dict(cache=cache(k=FAKE + 1)), dict(w=FAKE + 2), dict(wo=FAKE * 3 + 2),
               dict(B=1 << 24, ws_=640, wh=640 * (1 << 24), os=100, oh=100 << 24, nl=FAKE << 10)):
        assert call(**kw) == UNSUPPORTED, kw
    need = lib.wq_evict_paged_workspace_size(2, 2, 100)
    assert need >= 2 * 2 * 100 * 8 and lib.wq_evict_paged_workspace_size(0, 2, 100) == 0
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE
    assert call(B=0, kl=None) == 0


def test_lora_refusals(lib):
    ok = dict(x=FAKE, ldx=64, T=400, H=64, A=FAKE, B=FAKE, s=FAKE, n=3, r=16, ids=FAKE, N=48, dtype=0, y=FAKE, ldy=48, ws=FAKE,
              nb=1 << 30)
    call = lambda **kw: lib.wq_lora_add(*{**ok, **kw}.values(), None, None)
    for kw in (dict(T=-1), dict(H=-8), dict(N=-8), dict(n=-1), dict(r=0), dict(dtype=2), dict(dtype=-1), dict(x=None),
               dict(A=None), dict(B=None), dict(ids=None), dict(y=None), dict(ldx=56), dict(ldy=40)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=60), dict(N=44), dict(r=12), dict(r=136), dict(ldx=68), dict(ldy=52), dict(n=8193), dict(x=FAKE + 2),
               dict(A=FAKE + 8), dict(B=FAKE + 8), dict(y=FAKE + 4), dict(s=FAKE + 2), dict(T=1 << 24)):
        assert call(**kw) == UNSUPPORTED, kw
    need = lib.wq_lora_add_workspace_size(400, 3, 16)
    assert need >= 400 * 4 and lib.wq_lora_add_workspace_size(4000, 3, 64) >= 4000 * 64 * 4 and lib.wq_lora_add_workspace_size(256, 3, 16) == 0
    assert lib.wq_lora_add_workspace_size(0, 3, 16) == 0
    assert call(nb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    for kw in (dict(T=0), dict(H=0), dict(N=0), dict(n=0)):
        assert call(**kw) == 0, kw
