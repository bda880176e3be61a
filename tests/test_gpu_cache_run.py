"""The operators as a serving step runs them: projection and adapters, head norms
into the paged cache, attention, the keys' weights, eviction; called one after
the other, and recorded into one CUDA graph."""
import pytest
import torch

from w8a8_int8_quantized_token_gb300 import binding as wq

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Step:
    """One layer's attention half for B sequences with q new tokens each."""

    def __init__(self, B=5, q=1, start=(40, 3, 17, 33, 60), H=256, Hq=8, Hkv=2, D=64, page=16, most=96, budget=48):
        g = torch.Generator().manual_seed(0)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF).cuda()
        self.B, self.q, self.Hq, self.Hkv, self.D, self.page, self.most, self.budget = B, q, Hq, Hkv, D, page, most, budget
        N, pages = (Hq + 2 * Hkv) * D, -(-most // page)
        self.W = wq.quantize_weight(rand(N, H, scale=H ** -0.5), "channel")
        self.A, self.Bm = rand(3, 16, H, scale=H ** -0.5), rand(3, N, 16, scale=0.25)
        self.adapters = torch.tensor([b % 4 - 1 for b in range(B) for _ in range(q)], dtype=torch.int32).cuda()
        self.wq_, self.wk = rand(D) + 1, rand(D) + 1
        self.table = wq.rope_table(512, D)
        self.kc, self.vc = rand(B * pages, Hkv, page, D), rand(B * pages, Hkv, page, D)
        self.pt = torch.randperm(B * pages, generator=g).to(torch.int32).reshape(B, pages).cuda()
        self.len = torch.tensor(start, dtype=torch.int32).cuda()
        self.pos = self.len.clone()  # positions go on when keys have gone
        self.w = torch.zeros(B, Hkv, most, device="cuda")
        self.x = torch.empty(B * q, H, dtype=BF, device="cuda")
        self.out = torch.empty(B * q, Hq, D, dtype=BF, device="cuda")
        self.lse = torch.empty(B * q, Hq, device="cuda")
        self.new_len, self.kept = torch.empty_like(self.len), torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
        self.status = wq.new_status()
        self.flat = torch.arange(B, device="cuda")[:, None].expand(B, q).reshape(-1)
        self.ahead = torch.arange(q, dtype=torch.int32, device="cuda").repeat(B)

    def __call__(self):
        T = self.B * self.q
        y = wq.linear_w8a8(self.x, *self.W, status=self.status)
        wq.lora_add(y, self.x, self.A, self.Bm, self.adapters, status=self.status)
        q, k, v = y.view(T, -1, self.D).split([self.Hq, self.Hkv, self.Hkv], dim=1)
        at = self.len[self.flat] + self.ahead  # place in the sequence
        slots = self.pt[self.flat, (at // self.page).long()].long() * self.page + at % self.page
        q = wq.head_norm_rope_append_paged(k, v, self.pos[self.flat] + self.ahead, slots, self.table, self.kc, self.vc,
                                           k_weight=self.wk, q=q, q_weight=self.wq_, status=self.status)
        self.len += self.q
        self.pos += self.q
        wq.attention_shared_prefix(q, self.kc, self.vc, None, 0, self.pt, self.len, self.most, out=self.out, lse=self.lse,
                                   status=self.status)
        wq.attention_weights_paged(q, self.kc, self.pt, self.len, self.most, self.lse, self.w, status=self.status)
        wq.evict_paged(self.w, self.kc, self.vc, self.pt, self.len, self.most, self.budget, recent=8, first=2,
                       new_len=self.new_len, kept=self.kept, status=self.status)
        self.len.copy_(self.new_len)


def state(s):
    return [t.clone() for t in (s.out, s.lse, s.len, s.kept, s.kc, s.vc, s.w)]


@pytest.mark.parametrize("q", [1, 7])
def test_a_step_recorded_and_replayed_is_the_step(q):
    xs = [torch.randn(5 * q, 256, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in range(4)]
    eager, graphed = Step(q=q), Step(q=q)
    want = []
    for x in xs:
        eager.x.copy_(x)
        eager()
        want.append(state(eager))
    keep = [t.clone() for t in (graphed.kc, graphed.vc, graphed.len, graphed.pos)]
    graphed.x.copy_(xs[0])
    graphed()  # once outside, as torch asks
    for t, k in zip((graphed.kc, graphed.vc, graphed.len, graphed.pos), keep):
        t.copy_(k)
    graphed.w.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed()
    for x, w in zip(xs, want):
        graphed.x.copy_(x)
        graph.replay()
        got = state(graphed)
        for a, b in zip(got[:4], w[:4]):
            assert torch.equal(a, b)
        for c in (4, 5, 6):
            assert torch.equal(got[c], w[c])
    assert int(eager.status) == 0 and int(graphed.status) == 0
    assert int(eager.len.max()) == 48 and eager.len.min() == 3 + 4 * q  # some were cut, the short one was not


@pytest.mark.parametrize("q", [1, 7])
def test_without_eviction_the_weights_are_the_tokens(q):
    """A budget that no sequence reaches: every token has given each of its query
    heads' weight once, to the keys of its sequence."""
    s = Step(q=q, budget=96)
    for i in range(3):
        s.x.copy_(torch.randn(5 * q, 256, generator=torch.Generator().manual_seed(i)).to(BF))
        s()
    n = torch.arange(96, device="cuda") < s.len[:, None]
    total = (s.w * n[:, None]).sum(-1)
    # a step's sums drop the weights that its own keys' places held before (zeros here)
    assert ((total / (3 * q * s.Hq // s.Hkv)) - 1).abs().max() < 1e-4
    assert torch.equal(s.kept[0, 0, :int(s.len[0])].cpu(), torch.arange(int(s.len[0]), dtype=torch.int32))
    assert int(s.status) == 0


def test_calls_on_streams_of_their_own_are_the_calls_alone():
    """Adapters of many tokens twice, few tokens, weights and eviction side by
    side, each call with its own workspace."""
    g = torch.Generator().manual_seed(3)
    rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(BF).cuda()
    status = wq.new_status()
    x, A, Bm = rand(2300, 512), rand(4, 64, 512, scale=512 ** -0.5), rand(4, 1024, 64, scale=0.125)
    ids = torch.randint(-1, 4, (2300,), generator=g).to(torch.int32).cuda()
    pt = torch.randperm(4 * 32, generator=g).to(torch.int32).reshape(4, 32).cuda()
    q, kc, vc = rand(4 * 100, 8, 128), rand(4 * 32, 2, 64, 128), rand(4 * 32, 2, 64, 128)
    n, w0 = torch.tensor([2048, 1500, 100, 777], dtype=torch.int32).cuda(), torch.rand(4, 2, 2048, generator=g).cuda()
    lse = torch.full((400, 8), 4.0).cuda()

    def adapters(T):
        y0 = rand(T, 1024)
        def call():
            return [wq.lora_add(y0.clone(), x[:T], A, Bm, ids[:T], status=status)]
        return call

    def weights():
        return [wq.attention_weights_paged(q, kc, pt, n, 2048, lse, w0.clone(), status=status)]

    def evict():
        k, v, w = kc.clone(), vc.clone(), w0.clone()
        return [*wq.evict_paged(w, k, v, pt, n, 2048, 700, recent=30, first=2, status=status), k, v, w[..., :700].clone()]

    calls = [adapters(2300), weights, adapters(2000), evict, adapters(100)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i].append(c())
    torch.cuda.synchronize()
    for name, w, runs in zip("abcde", want, got):
        for run in runs:
            for a, b in zip(run, w):
                if a.dim() == 3 and a.shape[-1] == 700 and a.dtype == torch.float32:
                    rows = torch.arange(700, device="cuda") < n.clamp(max=700)[:, None, None]
                    a, b = a.where(rows, 0), b.where(rows, 0)
                assert torch.equal(a, b), name
    assert int(status) == 0
