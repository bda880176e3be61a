"""One decoder layer as a server runs it, with every part from the library.

A prompt that all sequences share is computed once into a paged key/value
cache; then each sequence takes tokens of its own behind it:

    y        = RMS(h)                                     block_norm
    q, k, v  = y Wqkv                                     linear_w8a8
    cache   <- rope(k), v;  q = rope(q)                   rope_append_paged
    o        = attention(q, shared prompt, own tokens)    attention_shared_prefix
    h, y     = h + RMS(o Wo), RMS(h)                      linear_w8a8, block_norm
    h, y     = h + s * RMS(moe(y)), RMS(h)                moe_forward, block_norm

    python examples/serve_layer.py

runs the sequences' tokens once as ragged chunks and once token by token and
compares the two (the weights and inputs are random).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w8a8_int8_quantized_token_gb300 import binding as wq  # noqa: E402


class Layer:
    """Weights, rotary table and paged cache of one layer."""

    def __init__(self, H=256, q_heads=8, kv_heads=2, D=64, I=128, E=8, k=2, pages=64, page=16,
                 trained=64, device="cuda"):
        g = torch.Generator(device=device).manual_seed(0)
        rand = lambda *shape: (torch.randn(*shape, device=device, generator=g) * 0.05).bfloat16()
        self.H, self.q_heads, self.kv_heads, self.D, self.k, self.page = H, q_heads, kv_heads, D, k, page
        self.qkv = wq.quantize_weight(rand((q_heads + 2 * kv_heads) * D, H), "channel")
        self.o = wq.quantize_weight(rand(H, q_heads * D), "channel")
        w13, w2 = zip(*((wq.quantize_weight(rand(2 * I, H), "channel"), wq.quantize_weight(rand(H, I), "channel"))
                        for _ in range(E)))
        self.w13, self.s13 = (torch.stack(t) for t in zip(*w13))
        self.w2, self.s2 = (torch.stack(t) for t in zip(*w2))
        self.router = rand(E, H).float()
        self.norms = [1 + rand(H) for _ in range(5)]
        # positions past the trained context: YaRN, four times as long
        self.table = wq.rope_table(4 * trained, D, scaling="yarn", factor=4.0, trained=trained)
        self.k_cache = torch.zeros(pages, kv_heads, page, D, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)

    def step(self, x, positions, slots, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, cu_q, max_q,
             status):
        """x bf16 [T, H]: the tokens' residual stream -> the layer's output."""
        T, D, n = x.shape[0], self.D, self.norms
        h, y = wq.block_norm(x, pre="rms", pre_weight=n[0])
        qkv = wq.linear_w8a8(y, *self.qkv).view(T, -1, D)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        q = wq.rope_append_paged(k, v, positions, slots, self.table, self.k_cache, self.v_cache, q=q, status=status)
        o = wq.attention_shared_prefix(q, self.k_cache, self.v_cache, prefix_pages, prefix_len, page_table,
                                       suffix_len, max_suffix, cu_q=cu_q, max_q=max_q, status=status)
        a = wq.linear_w8a8(o.view(T, -1), *self.o)
        h, y = wq.block_norm(a, residual=h, post="rms", post_weight=n[1], pre="rms", pre_weight=n[2])
        m = wq.moe_forward(y, y.float() @ self.router.T, self.w13, self.s13, self.w2, self.s2, self.k)
        return wq.block_norm(m, residual=h, scale=0.5, post="rms", post_weight=n[3], pre="rms", pre_weight=n[4])[1]


def run(prompt=37, lengths=(5, 1, 20), device="cuda"):
    """Outputs of the sequences' tokens, as chunks and token by token, and the
    largest error of the prompt's cached keys turned back to position 0."""
    B, T = len(lengths), sum(lengths)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)
    outs = []
    status = wq.new_status(device)
    for chunks in (True, False):
        layer = Layer(device=device)
        page = layer.page
        g = torch.Generator(device=device).manual_seed(1)
        x0 = torch.randn(prompt, layer.H, device=device, generator=g).bfloat16()
        xs = [torch.randn(n, layer.H, device=device, generator=g).bfloat16() for n in lengths]
        npx, ns = -(-prompt // page), -(-max(lengths) // page)
        order = torch.randperm(layer.k_cache.shape[0], generator=torch.Generator().manual_seed(2)).tolist()
        prefix, own = order[:npx], [order[npx + b * ns:npx + (b + 1) * ns] for b in range(B)]
        slot = lambda pages, t: pages[t // page] * page + t % page
        # the shared prompt: one sequence without a prefix
        layer.step(x0, torch.arange(prompt, dtype=torch.int32, device=device),
                   torch.tensor([slot(prefix, t) for t in range(prompt)], device=device), None, 0, i32([prefix]),
                   i32([prompt]), prompt, i32([0, prompt]), prompt, status)
        # the sequences behind it: all their tokens at once, or one each at a time
        out = [[] for _ in range(B)]
        for first, last in ([(0, max(lengths))] if chunks else [(t, t + 1) for t in range(max(lengths))]):
            took = [range(first, min(last, n)) for n in lengths]
            n = [len(t) for t in took]
            cu = [sum(n[:b]) for b in range(B + 1)]
            x = torch.cat([xs[b][t.start:t.stop] for b, t in enumerate(took)])
            y = layer.step(x, i32([prompt + t for b in range(B) for t in took[b]]),
                           torch.tensor([slot(own[b], t) for b in range(B) for t in took[b]], device=device),
                           i32(prefix), prompt, i32(own), i32([t.stop if len(t) else 0 for t in took]), max(lengths),
                           i32(cu), max(n), status)
            for b in range(B):
                out[b].append(y[cu[b]:cu[b + 1]])
        outs.append(torch.cat([torch.cat(o) for o in out]))
    # the cached keys of the prompt, turned back, are the keys as they came
    keys = torch.stack([layer.k_cache[slot(prefix, t) // page, :, slot(prefix, t) % page] for t in range(prompt)])
    back = wq.rope(keys, torch.arange(prompt, dtype=torch.int32, device=device), layer.table, inverse=True,
                   status=status)
    y = wq.block_norm(x0, pre="rms", pre_weight=layer.norms[0])[1]
    k = wq.linear_w8a8(y, *layer.qkv).view(prompt, -1, layer.D)[:, layer.q_heads:layer.q_heads + layer.kv_heads]
    m2 = float(layer.table[0, 0, 0]) ** 2  # YaRN scales cos and sin by m, so turning back gives m^2 k
    if int(status) != 0:
        raise RuntimeError(f"status {int(status)}")
    return outs[0], outs[1], float((back.float() / m2 - k.float()).abs().max() / k.float().abs().max())


def main():
    chunk, single, key_error = run()
    diff = float((chunk.float() - single.float()).norm() / chunk.float().norm())
    print(f"{chunk.shape[0]} tokens: chunks against token by token {diff:.2e}, keys turned back {key_error:.2e}")
    return chunk, single, key_error


if __name__ == "__main__":
    main()
