"""Bad page ids in an eviction in place: told of wherever a key stays, also
where nothing moves; the other keys move as they would."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu


def evict(table, lens, **kw):
    g = torch.Generator().manual_seed(1)
    kc = torch.randn(8, 2, 16, 8, generator=g).bfloat16().cuda()
    vc, w = kc + 1, torch.rand(len(lens), 2, 64, generator=g).cuda()
    st = wq.new_status()
    wq.evict_paged(w, kc, vc, torch.tensor(table, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 64,
                   24, status=st, **kw)
    return int(st), kc, vc


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1])
@pytest.mark.parametrize("kw,page", [(dict(first=16, recent=8), 0),  # keys that stay at their place
                                     (dict(first=16), 1)])           # a page that keys go to
def test_in_a_sequence_that_is_cut(bad, kw, page):
    table = [[0, 1, 2, 3]]
    good = evict(table, [64], **kw)
    assert good[0] == 0
    table[0][page] = bad
    st, kc, vc = evict(table, [64], **kw)
    assert st == -6
    if page == 0:  # keys of page 0 stand: nothing else is lost
        assert torch.equal(kc, good[1]) and torch.equal(vc, good[2])
    else:  # neither read nor written
        start = evict(table, [0], **kw)
        assert torch.equal(kc, start[1]) and torch.equal(vc, start[2])


@pytest.mark.parametrize("lens,told", [([24, 20], True), ([16, 17], True), ([24, 16], False), ([64, 0], False)])
def test_in_a_sequence_that_keeps_all(lens, told):
    """Page 1 of the second sequence is bad: told of once it has a key there."""
    assert evict([[0, 1, 2, 3], [4, 8, 5, 6]], lens)[0] == (-6 if told else 0)
    assert evict([[0, 1, 2, 3], [4, 7, 5, 6]], lens)[0] == 0
