"""The operators that a serving layer takes next to `perf/operators.py`'s, as
cases that can be timed and compared.

Keys on their way into the cache: the norm of each query and key head with the
rotary position in the same pass (`head`, `append`).  What the cache's keys are
worth and which of them stay: the accumulated attention weight of each key
(`weights`) and the eviction of the least attended ones (`evict`).  Beside a
shared projection: the low-rank adapters of many requests (`lora`).  Each case
is one call; `run` computes it in elementary float32 torch operations or, with
`own` set, through the library's entry points.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
MAX_POS = 65536  # rows of the rotary table a serving program keeps
EPS = 1e-6

# The most a drawn case may cost, from the largest listed ones.
MOST_ELEMS = 8191 * 56 * 128         # head, append: elements of all heads
MOST_SCORES = 64 * 4096 * 4096       # weights: query heads * tokens * keys, padded
MOST_KEYS = 64 * 8192 * 8 * 128      # weights: elements of the keys at their longest
MOST_CACHE = 64 * 2048 * 8 * 128     # evict: elements of the keys at their longest
MOST_TOKENS = 8192 * (7168 + 2 * 7168)  # lora: elements of x, and of y twice
MOST_RANKS = 512                     # lora: ranks of all adapters, where there are many tokens


def listed():
    return [
        # the 32 heads of 1021 tokens, in float32 (a model run at full precision), heads of 80 rotated in part
        dict(name="head odd", op="head", T=1021, heads=32, D=80, rot=32, layout="half", dtype="f32"),
        # a decode batch: queries and keys of one token a sequence, scattered over the pages
        dict(name="append decode", op="append", T=128, Hq=64, Hkv=8, D=128, rot=128, page=64, layout="half", dtype="bf16"),
        # a prompt of odd length
        dict(name="append prompt", op="append", T=8191, Hq=40, Hkv=8, D=128, rot=128, page=16, layout="inter", dtype="bf16"),
        # a decode batch of long ragged contexts: every step adds its weights
        dict(name="weights decode", op="weights", B=64, q=1, Hkv=8, G=8, D=128, L=8192, page=64, decay=1.0, shared=False, dtype="bf16"),
        # ragged prompt chunks behind a shared prompt, older weights fading
        dict(name="weights chunks", op="weights", B=6, q=501, Hkv=6, G=5, D=64, L=2047, page=16, decay=0.9, shared=True, dtype="f16"),
        # a prompt's tokens over the prompt itself
        dict(name="weights prompt", op="weights", B=1, q=4096, Hkv=8, G=8, D=128, L=4096, page=64, decay=1.0, shared=False, dtype="bf16"),
        # one long prompt cut down into pages of its own (its old pages stay with other requests)
        dict(name="evict prompt", op="evict", B=1, Hkv=8, D=128, L=32768, budget=4096, recent=256, first=4, page=64, inplace=False, dtype="bf16"),
        # a decode batch gives a page's worth of places back, in place, odd sizes
        dict(name="evict decode", op="evict", B=64, Hkv=8, D=128, L=2048, budget=1900, recent=100, first=4, page=32, inplace=True, dtype="bf16"),
        # one decode token with an adapter: latency
        dict(name="lora one", op="lora", T=1, H=7168, N=7168, r=16, n=8, dtype="bf16"),
        # a decode batch over 32 adapters at a fused query, key and value projection, some without one
        dict(name="lora decode", op="lora", T=128, H=7168, N=10240, r=16, n=32, dtype="bf16"),
        # a ragged middle size: an odd number of tokens and widths off the powers of two
        dict(name="lora ragged", op="lora", T=1021, H=4104, N=2056, r=24, n=5, dtype="f16"),
        # prompts with a few large adapters
        dict(name="lora prefill", op="lora", T=8192, H=7168, N=7168, r=64, n=8, dtype="bf16"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["head", "append", "weights", "weights", "evict", "evict", "lora", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    page = rng.choice([16, 32, 48, 64, 128])
    D = rng.choice([64, 80, 96, 128, 128])
    Hkv, G = rng.choice([1, 2, 4, 6, 8, 16]), rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    if op == "head":
        heads = rng.choice([1, 5, 8, 16, 32, 64])
        dtype = rng.choice([dtype, "f32"])
        return dict(op=op, T=_log(rng, 1, min(16384, MOST_ELEMS // (heads * D * SIZE[dtype] // 2))), heads=heads, D=D,
                    rot=rng.choice([D, D, D // 2, 32]), layout=rng.choice(["half", "inter"]), dtype=dtype)
    if op == "append":
        return dict(op=op, T=_log(rng, 1, min(16384, MOST_ELEMS // (Hkv * (G + 2) * D))), Hq=Hkv * G, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, 32]), page=page, layout=rng.choice(["half", "inter"]), dtype=dtype)
    if op == "weights":
        B, q = _log(rng, 1, 256), rng.choice([1, 1, 1, 3, _log(rng, 5, 2000)])
        L = max(q, _log(rng, 1, 16384))
        while B * Hkv * G * q * L > MOST_SCORES or B * L * Hkv * D > MOST_KEYS:
            if B > 1:
                B = (B + 1) // 2
            else:
                q, L = (q + 1) // 2, (L + 1) // 2
        return dict(op=op, B=B, q=q, Hkv=Hkv, G=G, D=D, L=L, page=page, decay=rng.choice([1.0, 1.0, 0.9]),
                    shared=rng.random() < 0.5, dtype=dtype)
    if op == "evict":
        B, L = _log(rng, 1, 128), _log(rng, 16, 32768)
        while B * L * Hkv * D > MOST_CACHE:
            B, L = (B + 1) // 2, L if B > 1 else L // 2
        budget = max(1, int(L * rng.choice([0.1, 0.25, 0.5, 0.9, 1.0])))
        recent = rng.randint(0, budget // 2)
        return dict(op=op, B=B, Hkv=Hkv, D=D, L=L, budget=budget, recent=recent, first=min(rng.choice([0, 1, 4]), budget - recent),
                    page=page, inplace=rng.random() < 0.5, dtype=dtype)
    H, N = 8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 1280)
    T = _log(rng, 1, min(16384, MOST_TOKENS // (H + 2 * N)))
    r = rng.choice([8, 16, 16, 24, 32, 64, 64])
    n = _log(rng, 1, 64)
    n = n if T <= 256 else max(1, min(n, MOST_RANKS // r))
    return dict(op=op, T=T, H=H, N=N, r=r, n=n, dtype=dtype)


# ---------------------------------------------------------------- inputs
def _lens(case):
    """Query tokens and keys of each sequence (the keys include the tokens' own): a decode batch has `q` tokens everywhere,
    chunks of more than 8 are ragged."""
    r = random.Random("%d %d %d" % (case["B"], case.get("q", 1), case["L"]))
    B, q, L = case["B"], case.get("q", 1), case["L"]
    ql = [q if q <= 8 or b == 0 else r.randint(1, q) for b in range(B)]
    kl = [L if b == 0 else r.randint(min(L, ql[b]), L) for b in range(B)]
    return ql, kl


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _table(rot):
    """cos and sin of pos * 10000^(-2i/rot), float32 from float64 angles: [MAX_POS, rot/2, 2]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * torch.exp(-math.log(10000.0) * 2 * i / rot)
    return torch.stack([a.cos(), a.sin()], -1).float()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case=dict(case), op=case["op"])
    if case["op"] == "head":
        T, n, D = case["T"], case["heads"], case["D"]
        s["x"] = _randn(g, (T, n, D), dt, 3.0)
        s["w"] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
        s["pos"] = torch.randint(0, MAX_POS, (T,), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = _table(case["rot"])
    elif case["op"] == "append":
        T, Hq, Hkv, D, page = (case[k] for k in ("T", "Hq", "Hkv", "D", "page"))
        qkv = _randn(g, (T, Hq + 2 * Hkv, D), dt, 3.0)  # one QKV linear's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        for k in ("w_q", "w_k"):
            s[k] = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(dt)
        s["pos"] = torch.randint(0, MAX_POS, (T,), device="cuda", generator=g, dtype=torch.int32)
        pages = T // page + 9
        slots = torch.randperm(pages * page, device="cuda", generator=g)[:T]
        slots[torch.rand(T, device="cuda", generator=g) < 0.02] = -1  # padding tokens
        s["slots"] = slots
        s["k_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["v_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["table"] = _table(case["rot"])
    elif case["op"] == "weights":
        B, Hkv, G, D, page, L = (case[k] for k in ("B", "Hkv", "G", "D", "page", "L"))
        ql, kl = _lens(case)
        T, ns = sum(ql), -(-L // page)
        order = torch.randperm(B * ns, device="cuda", generator=g).to(torch.int32)
        s["q"] = _randn(g, (T, Hkv * G, D), dt, 2.5)  # scores of a spread that trained heads have
        s["k_cache"] = _randn(g, (B * ns, Hkv, page, D), dt)
        s["page_table"] = order.reshape(B, ns).contiguous()
        s["key_len"] = _i32(kl)
        s["cu_q"] = _i32([sum(ql[:b]) for b in range(B + 1)])
        # where each token sits in its sequence, for the plain form
        s["seq"] = torch.tensor([b for b in range(B) for _ in range(ql[b])], dtype=torch.int64, device="cuda")
        s["idx"] = torch.tensor([i for b in range(B) for i in range(ql[b])], dtype=torch.int64, device="cuda")
        s["q_len"] = torch.tensor(ql, dtype=torch.int64, device="cuda")
        s["weights"] = torch.rand(B, Hkv, L, device="cuda", generator=g) * 2
        # what the attention over these keys gave the program, and over a shared prefix where there is one
        m, total = _sums(s)
        s["lse"] = (m + torch.log(total)).reshape(T, Hkv * G).contiguous()
        if case["shared"]:
            s["lse"] += torch.rand(s["lse"].shape, device="cuda", generator=g)
    elif case["op"] == "evict":
        B, Hkv, D, page, L = (case[k] for k in ("B", "Hkv", "D", "page", "L"))
        ns, no = -(-L // page), 0 if case["inplace"] else -(-case["budget"] // page)
        order = torch.randperm(B * (ns + no), device="cuda", generator=g).to(torch.int32)
        s["k_cache"] = _randn(g, (B * (ns + no), Hkv, page, D), dt)
        s["v_cache"] = _randn(g, (B * (ns + no), Hkv, page, D), dt)
        s["page_table"] = order[:B * ns].reshape(B, ns).contiguous()
        s["out_table"] = s["page_table"] if case["inplace"] else order[B * ns:].reshape(B, no).contiguous()
        s["key_len"] = _i32(_lens(case)[1])
        # few keys hold most of the weight, and some none at all
        s["weights"] = torch.exp(2 * torch.randn(B, Hkv, L, device="cuda", generator=g))
        s["weights"] *= torch.rand(B, Hkv, L, device="cuda", generator=g) > 0.03
        s["weights_out"] = torch.zeros(B, Hkv, case["budget"], device="cuda")
    else:
        T, H, N, r, n = (case[k] for k in ("T", "H", "N", "r", "n"))
        s["x"] = _randn(g, (T, H), dt)
        s["y"] = _randn(g, (T, N), dt)
        s["A"] = _randn(g, (n, r, H), dt, H ** -0.5)
        s["B"] = _randn(g, (n, N, r), dt, r ** -0.5)
        s["scales"] = 0.25 + 0.5 * torch.rand(n, device="cuda", generator=g)
        # a decode batch mixes its requests' adapters; prompts are runs of tokens; some have none
        ids = torch.randint(0, n, (T if T <= 256 else -(-T // 113),), device="cuda", generator=g, dtype=torch.int32)
        ids[torch.rand(ids.shape, device="cuda", generator=g) < (0.1 if T > 1 else 0.0)] = -1
        s["ids"] = (ids if T <= 256 else ids.repeat_interleave(113)[:T]).contiguous()
    return s


# ---------------------------------------------------------------- the plain forms
def _head_plain(x, w, pos, table, layout):
    """x [T, heads, D] -> float32: each head's norm, then the first rot of D rotated."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot = 2 * table.shape[1]
    c, s = table[pos.long()].unsqueeze(1).unbind(-1)
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * c - b * s, b * c + a * s
    r = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _scores(s):
    """Scores of the tokens, padded to the longest sequence: [B, Hkv, q, G, L], -inf where a token sees no key."""
    case = s["case"]
    B, Hkv, G, D, L, Q = (case[k] for k in ("B", "Hkv", "G", "D", "L", "q"))
    q = s["q"].float() / math.sqrt(D)
    k = s["k_cache"][s["page_table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    q = q.new_zeros(B, Q, Hkv, G, D).index_put((s["seq"], s["idx"]), q.view(-1, Hkv, G, D))
    x = (q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D) @ k.transpose(2, 3)).view(B, Hkv, Q, G, L)
    j = torch.arange(Q, device="cuda")
    last = s["key_len"].long()[:, None] - s["q_len"][:, None] + j  # [B, Q]
    hidden = (torch.arange(L, device="cuda") > last[..., None]) | (j >= s["q_len"][:, None])[..., None]
    return x.masked_fill_(hidden[:, None, :, None, :], float("-inf"))


def _sums(s):
    """Maximum and sum of exponentials of each (token, query head): [T, Hkv, G]."""
    x = _scores(s)
    m = x.amax(-1)
    total = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m)[..., None]).sum(-1)
    return m.transpose(1, 2)[s["seq"], s["idx"]], total.transpose(1, 2)[s["seq"], s["idx"]]


def _plain(s):
    case, op = s["case"], s["op"]
    dt = DT[case["dtype"]]
    if op == "head":
        return _head_plain(s["x"], s["w"], s["pos"], s["table"], case["layout"]).to(dt)
    if op == "append":
        keep = s["slots"] >= 0
        at = s["slots"][keep]
        page, off = at // case["page"], at % case["page"]
        s["k_cache"][page, :, off] = _head_plain(s["k"], s["w_k"], s["pos"], s["table"], case["layout"]).to(dt)[keep]
        s["v_cache"][page, :, off] = s["v"][keep]
        return _head_plain(s["q"], s["w_q"], s["pos"], s["table"], case["layout"]).to(dt), s["k_cache"], s["v_cache"]
    if op == "weights":
        B, Hkv, G, L, Q = (case[k] for k in ("B", "Hkv", "G", "L", "q"))
        lse = s["lse"].new_zeros(B, Q, Hkv, G).index_put((s["seq"], s["idx"]), s["lse"].view(-1, Hkv, G))
        add = torch.exp(_scores(s).sub_(lse.transpose(1, 2)[..., None])).sum((2, 3))  # [B, Hkv, L]
        i, n = torch.arange(L, device="cuda"), s["key_len"].long()
        old = torch.where((i < (n - s["q_len"])[:, None])[:, None], case["decay"] * s["weights"], 0.0)
        s["weights"].copy_(torch.where((i < n[:, None])[:, None], old + add, s["weights"]))
        return s["weights"]
    if op == "evict":
        Hkv, L, budget, page = (case[k] for k in ("Hkv", "L", "budget", "page"))
        i, n = torch.arange(L, device="cuda"), s["key_len"].long()
        key = s["weights"].masked_fill(((i < case["first"]) | (i >= (n - case["recent"])[:, None]))[:, None], float("inf"))
        key = key.masked_fill((i >= n[:, None])[:, None], float("-inf"))
        new = n.clamp(max=budget)
        j = torch.arange(budget, device="cuda")
        here = (j < new[:, None])[:, None]  # [B, 1, budget]
        kept = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]
        kept = torch.sort(kept.masked_fill(~here, L), dim=-1)[0]
        b, h, to = torch.nonzero(here.expand_as(kept), as_tuple=True)
        at = kept[b, h, to]
        src = (s["page_table"].long()[b, at // page], h, at % page)
        dst = (s["out_table"].long()[b, to // page], h, to % page)
        k, v = s["k_cache"][src], s["v_cache"][src]
        s["k_cache"][dst], s["v_cache"][dst] = k, v
        s["weights_out"][b, h, to] = s["weights"][b, h, at]
        kept = torch.where(here, kept, -1).to(torch.int32)
        return new.to(torch.int32), kept, s["weights_out"], s["k_cache"], s["v_cache"]
    n, r, H = s["A"].shape
    T = s["x"].shape[0]
    own_id = s["ids"][:, None] == torch.arange(n, device="cuda")  # [T, n]
    h = (s["x"].float() @ s["A"].float().view(n * r, H).t()).view(T, n, r) * (own_id * s["scales"])[..., None]
    s["y"].copy_(s["y"].float() + h.view(T, n * r) @ s["B"].float().transpose(1, 2).reshape(n * r, -1))
    return s["y"]


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from w8a8_int8_quantized_token_gb300 import binding as wq

    case, op = s["case"], s["op"]
    if op == "head":
        if "out" not in s:  # buffers a serving program keeps
            s["out"] = torch.empty_like(s["x"])
        return wq.head_norm_rope(s["x"], s["w"], s["pos"], s["table"], eps=EPS, layout=case["layout"], out=s["out"])
    if op == "append":
        if "q_out" not in s:
            s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        wq.head_norm_rope_append_paged(s["k"], s["v"], s["pos"], s["slots"], s["table"], s["k_cache"], s["v_cache"],
                                       k_weight=s["w_k"], q=s["q"], q_weight=s["w_q"], eps=EPS, layout=case["layout"],
                                       q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "weights":
        return wq.attention_weights_paged(s["q"], s["k_cache"], s["page_table"], s["key_len"], case["L"], s["lse"],
                                          s["weights"], cu_q=s["cu_q"], max_q=case["q"], decay=case["decay"])
    if op == "evict":
        if "ws" not in s:
            s["new_len"] = torch.empty_like(s["key_len"])
            s["kept"] = torch.empty(s["weights_out"].shape, dtype=torch.int32, device="cuda")
            s["ws"] = wq.evict_paged_workspace(s["weights"], case["L"], case["budget"])
        wq.evict_paged(s["weights"], s["k_cache"], s["v_cache"], s["page_table"], s["key_len"], case["L"], case["budget"],
                       recent=case["recent"], first=case["first"], out_table=None if case["inplace"] else s["out_table"],
                       weights_out=s["weights_out"], new_len=s["new_len"], kept=s["kept"], ws=s["ws"])
        return s["new_len"], s["kept"], s["weights_out"], s["k_cache"], s["v_cache"]
    if "ws" not in s:
        s["ws"] = wq.lora_add_workspace(s["y"], s["x"], s["A"])
    return wq.lora_add(s["y"], s["x"], s["A"], s["B"], s["ids"], scales=s["scales"], ws=s["ws"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- cost
def work(case):
    z = SIZE[case["dtype"]]
    if case["op"] == "head":
        n = case["T"] * case["heads"]
        return {"bytes": 2 * z * n * case["D"] + case["T"] * (4 + 4 * case["rot"]), "flops": n * (4 * case["D"] + 3 * case["rot"])}
    if case["op"] == "append":
        T, D, heads = case["T"], case["D"], case["Hq"] + case["Hkv"]
        return {"bytes": 2 * z * T * (heads + case["Hkv"]) * D + T * (12 + 4 * case["rot"]),
                "flops": T * heads * (4 * D + 3 * case["rot"])}
    if case["op"] == "weights":
        ql, kl = _lens(case)
        Hkv, D = case["Hkv"], case["D"]
        seen = sum(q * n - q * (q - 1) // 2 for q, n in zip(ql, kl)) * Hkv * case["G"]
        return {"bytes": sum(ql) * Hkv * case["G"] * (z * D + 4) + sum(kl) * Hkv * (z * D + 8), "flops": (2 * D + 3) * seen}
    if case["op"] == "evict":
        kl = _lens(case)[1]
        kept = sum(min(n, case["budget"]) for n in kl)
        return {"bytes": case["Hkv"] * (4 * sum(kl) + kept * (4 * z * case["D"] + 8)), "flops": case["Hkv"] * sum(kl)}
    T, H, N, r = (case[k] for k in ("T", "H", "N", "r"))
    return {"bytes": z * (T * (H + 2 * N) + min(T, case["n"]) * r * (H + N)), "flops": 2 * T * r * (H + N)}


# ---------------------------------------------------------------- the definition in 64 bits
def _head_exact(x, w, pos, rot, layout):
    """The norm as a division by the root, the rotation as a product of complex numbers, angles in 64 bits."""
    y = x.double()
    y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
    i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device), 2 * i / rot)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "head":
        return _head_exact(s["x"], s["w"], s["pos"], case["rot"], case["layout"])
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = _head_exact(s["k"], s["w_k"], s["pos"], case["rot"], case["layout"])
        t = torch.nonzero(s["slots"] >= 0).flatten()
        flat = s["slots"][t]
        for h in range(case["Hkv"]):
            kc[flat // case["page"], h, flat % case["page"]] = k[t, h]
            vc[flat // case["page"], h, flat % case["page"]] = s["v"][t, h].double()
        return _head_exact(s["q"], s["w_q"], s["pos"], case["rot"], case["layout"]), kc, vc
    if case["op"] == "weights":
        ql, kl = _lens(case)
        w, t0 = s["weights"].double(), 0
        for b in range(case["B"]):
            n, m = ql[b], kl[b]
            seen = torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n)
            for h in range(case["Hkv"]):
                heads = slice(h * case["G"], (h + 1) * case["G"])
                k = s["k_cache"][s["page_table"][b].long(), h].reshape(-1, case["D"])[:m].double()
                x = torch.einsum("tgd,kd->gtk", s["q"][t0:t0 + n, heads].double(), k) * case["D"] ** -0.5
                p = torch.exp(x - s["lse"][t0:t0 + n, heads].double().t()[..., None]) * seen
                w[b, h, :m - n] *= case["decay"]
                w[b, h, m - n:m] = 0
                w[b, h, :m] += p.sum((0, 1))
            t0 += n
        return w
    if case["op"] == "evict":
        kl, page, budget = _lens(case)[1], case["page"], case["budget"]
        kc, vc, wo = s["k_cache"].double(), s["v_cache"].double(), s["weights_out"].double()
        kept = torch.full(wo.shape, -1, dtype=torch.int32, device="cuda")
        for b in range(case["B"]):
            n = kl[b]
            new = min(n, budget)
            lo, hi = min(case["first"], n), max(n - case["recent"], min(case["first"], n))
            pages, out = s["page_table"][b].long(), s["out_table"][b].long()
            j = torch.arange(new, device="cuda")
            for h in range(case["Hkv"]):
                at = torch.arange(n, device="cuda")
                if n > budget:
                    # the middle keys in falling order of weight, earlier ones first among equals
                    mid = torch.argsort(-s["weights"][b, h, lo:hi].double(), stable=True)[:budget - lo - (n - hi)] + lo
                    at = torch.cat([at[:lo], mid.sort()[0], at[hi:]])
                kept[b, h, :new] = at.to(torch.int32)
                wo[b, h, :new] = s["weights"][b, h, at].double()
                for c, was in ((kc, s["k_cache"]), (vc, s["v_cache"])):
                    c[out[j // page], h, j % page] = was[pages[at // page], h, at % page].double()
        return s["key_len"].clamp(max=budget), kept, wo, kc, vc
    y = s["y"].double()
    for a in range(case["n"]):
        t = torch.nonzero(s["ids"] == a).flatten()
        y[t] += (s["x"][t].double() @ s["A"][a].double().t()) @ s["B"][a].double().t() * s["scales"][a].double()
    return y
