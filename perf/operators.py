"""The serving operators around the MoE layer, as cases that can be timed and compared.

Four operators make the attention half of a decoder layer: the norms around a
block (`block_norm`), rotary positions (`rope`), the rotated append to a paged
cache (`append`) and attention for a batch that shares a prefix (`attention`).
Each case is one call; `run` computes it in elementary float32 torch operations
or, with `own` set, through the library's entry points.
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
MOST_SCORES = 256 * 64 * (32768 + 256)  # attention: rows * keys
MOST_SUFFIX = 64 * 8192 * 8 * 128       # attention: elements of K in all suffixes at their longest
MOST_ELEMS = 8192 * 7168                # the others: elements of the main tensor


def listed():
    return [
        # one decode token through the norms between two halves of a layer of hidden size 7168
        dict(name="norm one token", op="norm", T=1, H=7168, dtype="bf16", post="none", pre="rms", gate="none", scale=1.0),
        # the 8192 tokens of a prefill step: norm after the block, residual, norm before the next
        dict(name="norm prefill", op="norm", T=8192, H=7168, dtype="bf16", post="rms", pre="rms", gate="none", scale=1.0),
        # layer norms with a gate per token and a residual scale, at an odd width
        dict(name="norm gated odd", op="norm", T=1021, H=4099, dtype="f16", post="layer", pre="layer", gate="token", scale=0.5),
        # the query heads of a decode batch
        dict(name="rope decode", op="rope", T=128, heads=64, D=128, rot=128, lead=0, layout="half", dtype="bf16", inverse=False),
        # the rotary 64 of 192 elements of 128 heads, a strided view, in a prefill chunk
        dict(name="rope slice prefill", op="rope", T=4096, heads=128, D=64, rot=64, lead=128, layout="inter", dtype="bf16", inverse=False),
        # a decode batch: one token a sequence, scattered over the pages
        dict(name="append decode", op="append", T=128, Hq=64, Hkv=8, D=128, rot=128, page=64, layout="half", dtype="bf16"),
        # a prefill chunk with odd counts, heads of 80 rotated in part
        dict(name="append prefill", op="append", T=8191, Hq=28, Hkv=7, D=80, rot=32, page=16, layout="half", dtype="f16"),
        # one sequence, a short prompt and a few tokens: latency
        dict(name="attend one", op="attention", B=1, q=1, Hkv=8, G=4, D=128, P=1000, L=17, page=16, dtype="bf16"),
        # a decode batch behind a system prompt
        dict(name="attend decode", op="attention", B=64, q=1, Hkv=8, G=8, D=128, P=8192, L=1024, page=64, dtype="bf16"),
        # a large batch that shares one long document
        dict(name="attend long prefix", op="attention", B=256, q=1, Hkv=8, G=8, D=128, P=32768, L=256, page=64, dtype="bf16"),
        # a batch that shares nothing, with long ragged contexts
        dict(name="attend no prefix", op="attention", B=64, q=1, Hkv=8, G=4, D=128, P=0, L=8192, page=32, dtype="bf16"),
        # ragged prompt chunks behind a shared prompt of odd length
        dict(name="attend chunks", op="attention", B=6, q=501, Hkv=6, G=5, D=64, P=3001, L=2047, page=16, dtype="f16"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "append", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        H = rng.choice([128 * _log(rng, 1, 64), _log(rng, 100, 8192)])
        T = _log(rng, 1, max(1, min(65536, MOST_ELEMS // H)))
        return dict(op=op, T=T, H=H, dtype=rng.choice([dtype, "f32"]) if T * H <= MOST_ELEMS // 2 else dtype,
                    post=rng.choice(["none", "rms", "layer"]), pre=rng.choice(["rms", "rms", "layer"]),
                    gate=rng.choice(["none", "shared", "token"]) if T * H * 5 <= MOST_ELEMS * 4 else "none",
                    scale=rng.choice([1.0, 0.5, 0.22]))
    D = rng.choice([64, 80, 96, 128, 128])
    if op == "rope":
        heads = rng.choice([1, 5, 8, 16, 32, 64, 128])
        lead = rng.choice([0, 0, 64, 128])
        return dict(op=op, T=_log(rng, 1, min(16384, MOST_ELEMS // (heads * (D + lead)))), heads=heads, D=D,
                    rot=rng.choice([D, D, D // 2, 32]), lead=lead, layout=rng.choice(["half", "inter"]),
                    dtype=rng.choice([dtype, "f32"]) if heads <= 32 else dtype, inverse=rng.random() < 0.25)
    if op == "append":
        Hkv, G = rng.choice([1, 2, 4, 7, 8, 16]), rng.choice([1, 2, 4, 7, 8])
        return dict(op=op, T=_log(rng, 1, min(16384, MOST_ELEMS // (Hkv * (G + 2) * D))), Hq=Hkv * G, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, 32]), page=rng.choice([16, 32, 48, 64, 128]), layout=rng.choice(["half", "inter"]), dtype=dtype)
    Hkv = rng.choice([1, 2, 4, 6, 8, 16])
    G = rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
    B = _log(rng, 1, 256)
    q = rng.choice([1, 1, 1, 2, 4, _log(rng, 5, 600)])
    P = rng.choice([0, _log(rng, 1, 65536), _log(rng, 256, 65536)])
    L = max(q, _log(rng, 1, 8192))
    while B * q * Hkv * G * (P + L) > MOST_SCORES or B * L * Hkv * D > MOST_SUFFIX:
        if B > 1:
            B = (B + 1) // 2
        else:
            P, L = P // 2, max(q, L // 2)
    return dict(op=op, B=B, q=q, Hkv=Hkv, G=G, D=D, P=P, L=L, page=rng.choice([16, 32, 48, 64, 128]), dtype=dtype)


# ---------------------------------------------------------------- inputs
def _lens(case):
    """Query tokens and suffix lengths of each sequence (the suffix includes the query tokens): a decode batch has `q` tokens
    everywhere, chunks of more than 8 are ragged."""
    r = random.Random("%d %d %d" % (case["B"], case["q"], case["L"]))
    B, q, L = case["B"], case["q"], case["L"]
    ql = [q if q <= 8 or b == 0 else r.randint(1, q) for b in range(B)]
    sl = [L if b == 0 else r.randint(min(L, ql[b]), L) for b in range(B)]
    return ql, sl


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _table(rot):
    """cos and sin of pos * 10000^(-2i/rot), float32 from float64 angles: [MAX_POS, rot/2, 2]."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * torch.exp(-math.log(10000.0) * 2 * i / rot)
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case=dict(case), op=case["op"])
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # activations with 1% outlier channels, as the layer's own inputs have
        out = 1 + 19 * (torch.rand(H, device="cuda", generator=g) < 0.01).float()
        s["block"] = (torch.randn(T, H, device="cuda", generator=g) * out).to(dt)
        s["residual"] = (torch.randn(T, H, device="cuda", generator=g) * out * 4).to(dt)
        s["gate"] = None if case["gate"] == "none" else _randn(g, (H,) if case["gate"] == "shared" else (T, H), dt)
        for k in ("post", "pre"):
            s["w_" + k] = None if case[k] == "none" else (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(dt)
            s["b_" + k] = _randn(g, (H,), dt, 0.1) if case[k] == "layer" else None
    elif case["op"] == "rope":
        T, n, D = case["T"], case["heads"], case["D"]
        s["x"] = _randn(g, (T, n, case["lead"] + D), dt)[:, :, case["lead"]:]
        s["pos"] = torch.randint(0, MAX_POS, (T,), device="cuda", generator=g, dtype=torch.int32)
        s["table"] = _table(case["rot"])
    elif case["op"] == "append":
        T, Hq, Hkv, D, page = (case[k] for k in ("T", "Hq", "Hkv", "D", "page"))
        qkv = _randn(g, (T, Hq + 2 * Hkv, D), dt)  # one QKV linear's output
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["pos"] = torch.randint(0, MAX_POS, (T,), device="cuda", generator=g, dtype=torch.int32)
        pages = T // page + 9
        slots = torch.randperm(pages * page, device="cuda", generator=g)[:T]
        slots[torch.rand(T, device="cuda", generator=g) < 0.02] = -1  # padding tokens
        s["slots"] = slots
        s["k_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["v_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["table"] = _table(case["rot"])
    else:
        B, Hkv, G, D, P, page = (case[k] for k in ("B", "Hkv", "G", "D", "P", "page"))
        ql, sl = _lens(case)
        T = sum(ql)
        np_, ns = -(-P // page), -(-case["L"] // page)
        pages = np_ + B * ns
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        s["q"] = _randn(g, (T, Hkv * G, D), dt, 2.5)  # scores of a spread that trained heads have
        s["k_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["v_cache"] = _randn(g, (pages, Hkv, page, D), dt)
        s["prefix_pages"] = order[:np_].contiguous()
        s["page_table"] = order[np_:].reshape(B, ns).contiguous()
        s["suffix_len"] = torch.tensor(sl, dtype=torch.int32, device="cuda")
        s["cu_q"] = torch.tensor([sum(ql[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        # where each token sits in its sequence, for the plain form
        s["seq"] = torch.tensor([b for b in range(B) for _ in range(ql[b])], dtype=torch.int64, device="cuda")
        s["idx"] = torch.tensor([i for b in range(B) for i in range(ql[b])], dtype=torch.int64, device="cuda")
        s["q_len"] = torch.tensor(ql, dtype=torch.int64, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms
def _norm_plain(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()
    return v + b.float() if b is not None else v


def _rope_plain(x, pos, table, layout, inverse=False):
    """x [T, heads, D] -> float32, the first rot of D rotated."""
    x = x.float()
    rot = 2 * table.shape[1]
    c, s = table[pos.long()].unsqueeze(1).unbind(-1)
    s = -s if inverse else s
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * c - b * s, b * c + a * s
    r = torch.cat([u, v], -1) if layout == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain(s):
    case, op = s["case"], s["op"]
    dt = DT[case["dtype"]]
    if op == "norm":
        n = _norm_plain(s["block"].float(), case["post"], s["w_post"], s["b_post"])
        n = n * s["gate"].float() if s["gate"] is not None else n
        h = s["residual"].float() + case["scale"] * n
        return h.to(dt), _norm_plain(h, case["pre"], s["w_pre"], s["b_pre"]).to(dt)
    if op == "rope":
        return _rope_plain(s["x"], s["pos"], s["table"], case["layout"], case["inverse"]).to(dt)
    if op == "append":
        at = s["slots"][s["slots"] >= 0]
        page, off = at // case["page"], at % case["page"]
        keep = s["slots"] >= 0
        s["k_cache"][page, :, off] = _rope_plain(s["k"], s["pos"], s["table"], case["layout"]).to(dt)[keep]
        s["v_cache"][page, :, off] = s["v"][keep]
        return _rope_plain(s["q"], s["pos"], s["table"], case["layout"]).to(dt), s["k_cache"], s["v_cache"]
    B, Hkv, G, D, P, L = (case[k] for k in ("B", "Hkv", "G", "D", "P", "L"))
    T, Q = s["q"].shape[0], int(case["q"])
    q = s["q"].float() / math.sqrt(D)
    # prefix: every token against the shared keys, [Hkv, T*G, P]
    kp = s["k_cache"][s["prefix_pages"].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :P].float()
    vp = s["v_cache"][s["prefix_pages"].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :P].float()
    sp = (q.view(T, Hkv, G, D).transpose(0, 1).reshape(Hkv, T * G, D) @ kp.transpose(1, 2))
    sp = sp.view(Hkv, T, G, P).transpose(0, 1)
    # suffixes: sequences padded to Q tokens and L keys
    ks = s["k_cache"][s["page_table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    vs = s["v_cache"][s["page_table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L].float()
    qs = q.new_zeros(B, Q, Hkv, G, D).index_put((s["seq"], s["idx"]), q.view(T, Hkv, G, D))
    ss = qs.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, D) @ ks.transpose(2, 3)
    ss = ss.view(B, Hkv, Q, G, L).transpose(1, 2)[s["seq"], s["idx"]]  # [T, Hkv, G, L]
    last = s["suffix_len"].long()[s["seq"]] - s["q_len"][s["seq"]] + s["idx"]
    ss = ss.masked_fill((torch.arange(L, device="cuda") > last[:, None])[:, None, None, :], float("-inf"))
    m = torch.maximum(sp.amax(-1), ss.amax(-1)) if P else ss.amax(-1)
    ep, es = torch.exp(sp - m[..., None]), torch.exp(ss - m[..., None])
    total = ep.sum(-1) + es.sum(-1)
    op_ = (ep.transpose(0, 1).reshape(Hkv, T * G, P) @ vp).view(Hkv, T, G, D).transpose(0, 1)
    es = q.new_zeros(B, Q, Hkv, G, L).index_put((s["seq"], s["idx"]), es)
    os_ = es.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * G, L) @ vs
    os_ = os_.view(B, Hkv, Q, G, D).transpose(1, 2)[s["seq"], s["idx"]]
    return ((op_ + os_) / total[..., None]).reshape(T, Hkv * G, D).to(dt), (m + torch.log(total)).reshape(T, Hkv * G)


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from w8a8_int8_quantized_token_gb300 import binding as wq

    case, op = s["case"], s["op"]
    if op == "norm":
        if "x_out" not in s:  # buffers a serving program keeps
            s["x_out"], s["y"] = torch.empty_like(s["block"]), torch.empty_like(s["block"])
        return wq.block_norm(s["block"], residual=s["residual"], gate=s["gate"], scale=case["scale"],
                             post=case["post"], post_weight=s["w_post"], post_bias=s["b_post"],
                             pre=case["pre"], pre_weight=s["w_pre"], pre_bias=s["b_pre"], eps=EPS,
                             x_out=s["x_out"], y=s["y"])
    if op == "rope":
        if "out" not in s:
            s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")
        return wq.rope(s["x"], s["pos"], s["table"], layout=case["layout"], inverse=case["inverse"], out=s["out"])
    if op == "append":
        if "q_out" not in s:
            s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        wq.rope_append_paged(s["k"], s["v"], s["pos"], s["slots"], s["table"], s["k_cache"], s["v_cache"],
                             layout=case["layout"], q=s["q"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if "out" not in s:
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        s["ws"] = wq.attention_shared_prefix_workspace(s["q"], s["k_cache"], s["v_cache"], case["B"], case["P"],
                                                       case["L"], case["q"])
    wq.attention_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], case["P"], s["page_table"],
                               s["suffix_len"], case["L"], cu_q=s["cu_q"], max_q=case["q"], out=s["out"],
                               lse=s["lse"], ws=s["ws"])
    return s["out"], s["lse"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- cost
def work(case):
    z = SIZE[case["dtype"]]
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        gate = {"none": 0, "shared": H, "token": T * H}[case["gate"]]
        weights = H * sum({"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("post", "pre"))
        return {"bytes": z * (4 * T * H + gate + weights), "flops": 10 * T * H}
    if case["op"] == "rope":
        n = case["T"] * case["heads"]
        return {"bytes": 2 * z * n * case["D"] + case["T"] * (4 + 4 * case["rot"]), "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        T, D = case["T"], case["D"]
        return {"bytes": 2 * z * T * (case["Hq"] + 2 * case["Hkv"]) * D + T * (12 + 4 * case["rot"]),
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    ql, sl = _lens(case)
    Hq, D = case["Hkv"] * case["G"], case["D"]
    seen = sum(q * case["P"] + q * n - q * (q - 1) // 2 for q, n in zip(ql, sl))
    keys = case["P"] + sum(sl)
    return {"bytes": 2 * z * sum(ql) * Hq * D + 4 * sum(ql) * Hq + 2 * z * keys * case["Hkv"] * D,
            "flops": 4 * D * Hq * seen}


# ---------------------------------------------------------------- the definition in 64 bits
def _norm_exact(v, kind, w, b):
    if kind == "none":
        return v
    mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else 0.0
    d = v - mean
    r = d / torch.sqrt((d ** 2).sum(1, keepdim=True) / v.shape[1] + EPS) * w.double()
    return r if b is None else r + b.double()


def _rope_exact(x, pos, rot, layout, inverse=False):
    """The rotation as a product of complex numbers, angles in 64 bits."""
    y = x.double().clone()
    i = torch.arange(rot // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[:, None] / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device), 2 * i / rot)
    turn = torch.polar(torch.ones_like(angle), -angle if inverse else angle)[:, None, :]
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        n = _norm_exact(s["block"].double(), case["post"], s["w_post"], s["b_post"]) * case["scale"]
        h = s["residual"].double() + (n if s["gate"] is None else n * s["gate"].double())
        return h, _norm_exact(h, case["pre"], s["w_pre"], s["b_pre"])
    if case["op"] == "rope":
        return _rope_exact(s["x"], s["pos"], case["rot"], case["layout"], case["inverse"])
    if case["op"] == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = _rope_exact(s["k"], s["pos"], case["rot"], case["layout"])
        t = torch.nonzero(s["slots"] >= 0).flatten()
        flat = s["slots"][t]
        for h in range(case["Hkv"]):
            kc[flat // case["page"], h, flat % case["page"]] = k[t, h]
            vc[flat // case["page"], h, flat % case["page"]] = s["v"][t, h].double()
        return _rope_exact(s["q"], s["pos"], case["rot"], case["layout"]), kc, vc
    Hkv, G, D, P = (case[k] for k in ("Hkv", "G", "D", "P"))
    ql, sl = _lens(case)
    T = sum(ql)
    o = torch.zeros(T, Hkv * G, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, Hkv * G, dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        kp = s["k_cache"][s["prefix_pages"].long(), h].reshape(-1, D)[:P].double()
        vp = s["v_cache"][s["prefix_pages"].long(), h].reshape(-1, D)[:P].double()
        t0 = 0
        for b in range(case["B"]):
            n = ql[b]
            ks = s["k_cache"][s["page_table"][b].long(), h].reshape(-1, D)[:sl[b]].double()
            vs = s["v_cache"][s["page_table"][b].long(), h].reshape(-1, D)[:sl[b]].double()
            k, v = torch.cat([kp, ks]), torch.cat([vp, vs])
            heads = slice(h * G, (h + 1) * G)
            x = torch.einsum("tgd,kd->tgk", s["q"][t0:t0 + n, heads].double(), k) * D ** -0.5
            hidden = torch.ones(n, P + sl[b], dtype=torch.bool, device="cuda").tril(P + sl[b] - n).logical_not()
            x = x.masked_fill(hidden[:, None, :], -math.inf)
            lse[t0:t0 + n, heads] = torch.logsumexp(x, -1)
            o[t0:t0 + n, heads] = torch.softmax(x, -1) @ v
            t0 += n
    return o, lse
