"""Plain float64 definitions of the serving operators (norms around a block,
rotary positions, rotated append, attention behind a shared prefix), on the
CPU, with the error bounds that go with the library's float32 arithmetic."""
import math

import torch

# unit roundoff of a type: half the spacing at 1
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
E = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, want, tol, what):
    """|got - want| <= tol element by element (both may be inf or -inf alike)."""
    g, w = f64(got), want
    assert g.shape == w.shape, (what, g.shape, w.shape)
    same = (g == w) & torch.isinf(w)
    bad = ~(((g - w).abs() <= tol) | same)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {g.numel()} off, first at {i}: got {g[i]}, "
                             f"want {w[i]}, tolerance {torch.as_tensor(tol).expand_as(w)[i]}")


def norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    v = v if w is None else v * w
    return v + b if kind == "layer" and b is not None else v


def block_norm(block, residual, gate, scale, post, pw, pb, pre, qw, qb, eps):
    """(h, N_pre(h)) and for each the magnitude its float32 error scales with:
    a row's largest |term| (a subtracted mean and a cancelling residual leave
    errors of the size of their operands), spread over the row by the second
    norm, whose factor is 1/rms."""
    block, residual, gate, pw, pb, qw, qb = map(f64, (block, residual, gate, pw, pb, qw, qb))
    n = norm(block, post, pw, pb, eps)
    gate = 1.0 if gate is None else gate
    term = scale * gate * n
    h = term + (0.0 if residual is None else residual)
    wmax = 1.0 if pw is None else pw.abs()
    spread = (block - (block.mean(1, keepdim=True) if post == "layer" else 0)).pow(2).mean(1, keepdim=True)
    # the mean's own float32 error is relative to |block|, scaled by 1/rms
    mag_n = n.abs() + (block.abs().amax(1, keepdim=True) / torch.sqrt(spread + eps) * wmax
                       if post == "layer" else 0.0) + (0 if pb is None else pb.abs())
    mag_h = abs(scale) * (gate if isinstance(gate, float) else gate.abs()) * mag_n + \
        (0 if residual is None else residual.abs())
    y = norm(h, pre, qw, qb, eps)
    if pre == "none":
        return h, y, mag_h, mag_h
    c = h - (h.mean(1, keepdim=True) if pre == "layer" else 0)
    r = 1 / torch.sqrt(c.pow(2).mean(1, keepdim=True) + eps)
    wy = torch.ones_like(y) if qw is None else qw.abs().expand_as(y)
    # y = c * r * w: error of c (mag_h, and of its mean), and of r relative to
    # itself: the root mean square of the errors of c times r, at most the
    # largest mag_h times r
    worst = mag_h.amax(1, keepdim=True)
    mag_y = (mag_h + worst) * r * wy + c.abs() * r * wy * (1 + worst * r) + (0 if qb is None else qb.abs())
    return h, y, mag_h, mag_y


def rotate(x, pos, table, layout, inverse=False):
    """x [T, heads, D] in float64, table the float32 one; also |a| + |b| of each pair."""
    x, t = f64(x), f64(table)
    rot = 2 * t.shape[1]
    c, s = t[pos.cpu().long()].unsqueeze(1).unbind(-1)
    s = -s if inverse else s
    ia = list(range(rot // 2)) if layout == "half" else list(range(0, rot, 2))
    ib = list(range(rot // 2, rot)) if layout == "half" else list(range(1, rot, 2))
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * (c.abs() + s.abs())
    return y, mag


def rope_tol(y, mag, dtype):
    """Two products and a sum in float32 (three roundings of at most the
    pair's magnitude each, the subtraction one more), one rounding to dtype."""
    return U[dtype] * y.abs() + 4 * E * mag + TINY[dtype]


def table(max_pos, rot, base, scaling="none", factor=1.0, trained=0, beta_fast=32.0, beta_slow=1.0, mscale=0.0):
    i = torch.arange(rot // 2, dtype=torch.float64)
    m = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        d = lambda n: rot * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))
        lo, hi = max(math.floor(d(beta_fast)), 0), min(math.ceil(d(beta_slow)), rot - 1)
        hi = hi + 0.001 if hi == lo else hi
        u = 1 - ((i - lo) / (hi - lo)).clamp(0, 1)
        f = f * (u + (1 - u) / factor)
        m = mscale if mscale else (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return m * torch.stack([a.cos(), a.sin()], -1)


def keys_of(cache, pages, n, head):
    """The first n keys of a page list, [n, D] float64."""
    return f64(cache[pages.long(), head]).reshape(-1, cache.shape[-1])[:n]


def attention(q, k_cache, v_cache, prefix_pages, P, page_table, suffix_len, cu_q, scale, dtype):
    """out, lse, and their tolerances.

    The library's weights are rounded to dtype (u each), so out is off by at
    most u * sum p |v| plus its own rounding u |out|.  In float32: a score
    takes dk products, off by at most dk E times the sum of |q k| scale, plus
    the exponential's 2^-22 and its argument's rounding (|score| E in base 2,
    with the running maximum subtracted: 4 E times the largest |score| covers
    both); the sums over n keys of non-negative weights are off by at most
    n E (as many additions) relative."""
    q, kc, vc = q.cpu(), k_cache.cpu(), v_cache.cpu()
    pt, sl, cu = page_table.cpu(), suffix_len.cpu().tolist(), cu_q.cpu().tolist()
    T, Hq, dk = q.shape
    Hkv, dv = kc.shape[1], vc.shape[3]
    G, u = Hq // Hkv, U[dtype]
    out, tol = torch.zeros(T, Hq, dv, dtype=torch.float64), torch.zeros(T, Hq, dv, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    ltol = torch.zeros(T, Hq, dtype=torch.float64)
    for h in range(Hkv):
        kp, vp = (keys_of(c, prefix_pages.cpu(), P, h) if P else torch.zeros(0, c.shape[-1], dtype=torch.float64)
                  for c in (kc, vc))
        for b in range(len(sl)):
            n = cu[b + 1] - cu[b]
            ks, vs = keys_of(kc, pt[b], sl[b], h), keys_of(vc, pt[b], sl[b], h)
            k, v = torch.cat([kp, ks]), torch.cat([vp, vs])
            if n == 0 or not len(k):
                continue
            rows, heads = slice(cu[b], cu[b] + n), slice(h * G, (h + 1) * G)
            qf = f64(q[rows, heads])  # [n, G, dk]
            last = P - 1 + (sl[b] - n + 1 + torch.arange(n)).clamp(min=0)
            seen = (torch.arange(len(k)) <= last[:, None])[:, None, :]  # [n, 1, keys]
            count = seen.sum(-1).double()  # [n, 1]
            x = (qf @ k.T * scale).masked_fill(~seen, -math.inf)
            mag = (qf.abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(-1)  # [n, G]
            some = (count > 0).expand(n, G)
            p = torch.where(some[..., None], torch.softmax(x, -1), torch.zeros_like(x))
            e = dk * E * mag + 2.0 ** -22 + 4 * E * x.masked_fill(~seen, 0).abs().amax(-1) + count * E
            o, spread = p @ v, p @ v.abs()
            under = count[..., None] * TINY[dtype] * v.abs().amax(0)  # weights below dtype's normal range
            out[rows, heads] = o
            tol[rows, heads] = torch.where(some[..., None], u * (o.abs() + spread) + 4 * e[..., None] * spread +
                                           under + TINY[dtype], torch.zeros_like(o))
            z = torch.logsumexp(x, -1)
            lse[rows, heads] = z
            ltol[rows, heads] = torch.where(some, 2 * e + 4 * E * (1 + z.abs()), torch.zeros_like(z))
    return out, lse, tol, ltol


def head_norm_rotate(x, w, pos, tab, layout, eps):
    """rope(RMS(x) w) of x [T, heads, D] in float64, and its magnitudes as rotate gives them; tab None: the norm alone."""
    x = f64(x)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (1.0 if w is None else f64(w))
    if tab is None:
        return y, y.abs()
    z, mag = rotate(y, pos, tab, layout)
    rot = 2 * tab.shape[1]
    mag[..., rot:] = y[..., rot:].abs()
    return z, mag


def head_norm_tol(y, mag, dtype, D):
    """The sum of squares: chains of at most max(16, D / 32) fused steps in a
    lane, five levels of a tree, the mean's product: relative to itself, halved
    by the root; the root's reciprocal (2 ulp, 4 E), two products: 16 + D / 32 +
    8 units at most.  The rotation 4 E, one rounding to dtype."""
    return U[dtype] * y.abs() + (28 + D / 32) * E * mag + TINY[dtype]


def attention_weights(q, k_cache, page_table, key_len, cu_q, lse, weights, scale, decay):
    """The new weights in float64 and their tolerance.

    A score takes dk products in float32, off by at most dk E times the sum of
    |q k| scale; the factor scale log2(e), the product with it and the sum with
    the log-sum-exp (itself times log2(e)) round at most four times, each E times
    |score| + |lse|; the exponential is off by 2^-22 and its argument's base
    change by as much.  Rows are added in chains of at most 64 within a tile (any
    page size: all rows over 8 warps), tile by tile and part by part.  A weight
    below float32's normal range, 2^-126, may count as zero."""
    pt, kl, cu = page_table.cpu().long(), key_len.cpu().tolist(), cu_q.cpu().tolist()
    B, Hkv = weights.shape[:2]
    G = q.shape[1] // Hkv
    q, kc, lse, w = f64(q), k_cache.cpu(), f64(lse), f64(weights)
    tol = torch.zeros_like(w)
    for b in range(B):
        n, m = cu[b + 1] - cu[b], kl[b]
        old = max(0, m - n)
        w[b, :, :old] *= decay
        w[b, :, old:m] = 0
        tol[b, :, :m] = 2 * E * w[b, :, :m].abs()
        if n == 0 or m == 0:
            continue
        seen = torch.arange(m) <= (m - n + torch.arange(n))[:, None]
        for h in range(Hkv):
            k = keys_of(kc, pt[b], m, h)
            rows, heads = slice(cu[b], cu[b] + n), slice(h * G, (h + 1) * G)
            x = (q[rows, heads] @ k.T) * scale  # [n, G, m]
            mag = (q[rows, heads].abs() @ k.abs().T) * scale
            z = lse[rows, heads][..., None]
            p = torch.where(seen[:, None] & (z > -math.inf), torch.exp(x - z), torch.zeros(()).double())
            e = q.shape[2] * E * mag + 2.0 ** -21 + 4 * E * (x.abs() + z.abs().nan_to_num(posinf=0.0))
            chain = 64 + n * G / 8 + 2 * 152
            add = p.sum((0, 1))
            w[b, h, :m] += add
            tol[b, h, :m] += (p * e * 1.01).sum((0, 1)) + chain * E * add + E * w[b, h, :m].abs() + n * G * 2.0 ** -126
    return w, tol


def lora(y, x, A, B, ids, scales, dtype):
    """y plus each token's adapter in float64, and the tolerance: H products and
    at most 16 sums more in float32 for a sum of the first product, two 16-bit
    operands that leave 2 U^2 of it (fp16: relative to the row's largest), r
    products of both operands for a sum of the second, the scale, y's rounding."""
    y, x, A, B, s = map(f64, (y, x, A, B, scales))
    out, tol = y.clone(), torch.zeros_like(y)
    for t, a in enumerate(ids.tolist()):
        if 0 <= a < A.shape[0]:
            h, hm = A[a] @ x[t], A[a].abs() @ x[t].abs()
            f = 1.0 if s is None else float(s[a])
            d = f * (B[a] @ h)
            top = h.abs().max() if dtype == torch.float16 else 0.0
            eh = (A.shape[2] + 16) * E * hm + 2 * U[dtype] ** 2 * (h.abs() + top) + TINY[torch.float32]
            out[t] += d
            tol[t] = abs(f) * (B[a].abs() @ (eh + (2 * A.shape[1] + 4) * E * h.abs())) + 4 * E * (d.abs() + y[t].abs()) + \
                U[dtype] * out[t].abs() + TINY[dtype]
    return out, tol
