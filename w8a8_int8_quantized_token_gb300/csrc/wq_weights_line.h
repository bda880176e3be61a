// How the blocks of the attention-weights kernel share its work, and which of
// their parts its second kernel adds.  Plain integer arithmetic for host and
// device: the tests drive this file on the CPU.
//
// A unit is a (sequence, key head, pair of key tiles, query tile); those in which
// no token sees a key are left out.  All units lie on one line, in that order, and
// block c of n takes those from total * c / n on.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define WQ_HD __host__ __device__ __forceinline__
#else
#define WQ_HD inline
#endif

namespace wq {

constexpr int kWeightsPair = 256;  // keys of a pair of key tiles

struct WeightsLine {
  int T, B, max_q, heads, max_len;
  const int32_t *cu_q;     // [B + 1], nullptr: max_q tokens each
  const int32_t *key_len;  // [B]
  int tpt;                 // tokens of a query tile
  int shift;               // log2 of the tokens that its cost goes by, at most tpt
};

template <class N>
WQ_HD N least(N a, N b) {
  return a < b ? a : b;
}
template <class N>
WQ_HD N most(N a, N b) {
  return a > b ? a : b;
}

// A sequence: its tokens, keys, and the cost of its pairs of key tiles.  A pair
// costs 1 where all tokens are one query tile.  Else it costs its query tiles,
// as many as there would be of 2^shift tokens each, which add up without a
// loop; the tiles themselves have tpt >= 2^shift tokens, and a part of a pair's
// cost is that part of them.
struct Seq {
  int t0, n, len;
  int old;       // keys that were there before the tokens' own (negative: tokens with no key)
  int pairs, tiles, costs;
  int p1, d1;    // first pair whose keys not all tokens see, and how far it starts past `old`

  // query tiles of 2^shift tokens that see nothing of pair p, at the front of the sequence's
  WQ_HD int unseen(int p, int shift) const { return most(0, (p * kWeightsPair - old) >> shift); }
  WQ_HD int cost(int p, int shift) const { return tiles <= 1 ? 1 : costs - unseen(p, shift); }
  // cost of the pairs before p, of one key head
  WQ_HD int64_t before(int p, int shift) const {
    if (tiles <= 1) return p;
    const int64_t m = most(0, p - p1);
    return int64_t(p) * costs - (m * (d1 >> shift) + int64_t(kWeightsPair >> shift) * (m * (m - 1) / 2));
  }
};

WQ_HD Seq seq_of(const WeightsLine &a, int c0, int c1, int l) {
  Seq s;
  s.t0 = least(most(c0, 0), a.T);
  s.n = least(most(c1 - s.t0, 0), least(a.max_q, a.T - s.t0));
  s.len = least(most(l, 0), a.max_len);
  s.old = s.len - s.n;
  s.pairs = (s.len + kWeightsPair - 1) / kWeightsPair;
  s.tiles = (s.n + a.tpt - 1) / a.tpt;
  s.costs = (s.n + (1 << a.shift) - 1) >> a.shift;
  s.p1 = s.old <= 0 ? 0 : (s.old + kWeightsPair - 1) / kWeightsPair;
  s.d1 = s.p1 * kWeightsPair - s.old;
  return s;
}
WQ_HD bool in_range(const WeightsLine &a, const Seq &s, int c0, int c1, int l) {
  return s.t0 == c0 && s.t0 + s.n == c1 && s.len == l;
}
WQ_HD int first_of(const WeightsLine &a, int b) {
  return a.cu_q ? a.cu_q[b] : b * a.max_q;
}

// A place on the line: its sequence and the offset in it, the line's length
struct Place {
  int b;
  int64_t off, total, at;
};
// Where block c of n begins
WQ_HD int64_t first_unit(int64_t total, int64_t c, int64_t n) { return total * c / n; }

// Query tiles [qa, qb) of a sequence against a pair of key tiles; with one
// query tile in all, against `pairs` pairs one after the other
struct Piece {
  int b, h, k0, pairs, qa, qb;
  Seq s;
  bool whole;  // all query tiles of the pair
  int slot;    // else: where its sums go
};

// The pieces of a block, one after the other
struct Walk {
  int b, h, p;
  int64_t u, left;  // units of the pair that are done; units of the block to come
  int n0, n1, nl;   // the next sequence, read ahead
  Seq s;

  WQ_HD void ahead(const WeightsLine &a) {
    const bool some = b + 1 < a.B;
    n0 = some ? first_of(a, b + 1) : 0;
    n1 = some ? first_of(a, b + 2) : 0;
    nl = some ? a.key_len[b + 1] : 0;
  }
  WQ_HD void begin(const WeightsLine &a, const Place &at, int64_t units) {
    b = at.b;
    left = units;
    u = 0;
    h = p = 0;
    if (units <= 0) return;
    s = seq_of(a, first_of(a, b), first_of(a, b + 1), a.key_len[b]);
    ahead(a);
    const int64_t head = s.before(s.pairs, a.shift);
    h = int(at.off / head);
    const int64_t rest = at.off - h * head;
    int lo = 0, hi = s.pairs - 1;  // the last pair that starts at or before `rest`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s.before(mid, a.shift) <= rest) lo = mid;
      else hi = mid - 1;
    }
    p = lo;
    u = rest - s.before(p, a.shift);
  }
  WQ_HD bool next(const WeightsLine &a, Piece &o) {
    if (left <= 0) return false;
    while (p >= s.pairs) {  // the next head, or sequence with keys
      p = 0;
      if (s.pairs > 0 && ++h < a.heads) break;
      h = 0;
      ++b;
      s = seq_of(a, n0, n1, nl);
      ahead(a);
    }
    o.b = b;
    o.h = h;
    o.k0 = p * kWeightsPair;
    o.s = s;
    if (s.tiles <= 1) {  // a unit a pair
      const int take = int(least<int64_t>(s.pairs - p, left));
      o.pairs = take;
      o.qa = 0;
      o.qb = s.tiles;
      o.whole = true;
      o.slot = 0;
      left -= take;
      p += take;
      return true;
    }
    const int first = most(0, (p * kWeightsPair - s.old) / a.tpt), cost = s.cost(p, a.shift);
    const int64_t tiles = s.tiles - first, take = least<int64_t>(cost - u, left);
    o.pairs = 1;
    o.qa = first + int(u * tiles / cost);
    o.qb = first + int((u + take) * tiles / cost);
    o.whole = take == cost;
    o.slot = u == 0 ? 1 : 0;
    left -= take;
    u += take;
    if (u == cost) u = 0, ++p;
    return true;
  }
};

// Whether block c of n begins a pair that it leaves to blocks after it, whose
// first unit is at `at`: that pair in w, the end of its units in `end`
WQ_HD bool left_to_others(const WeightsLine &a, const Place &at, int64_t c, int64_t n, Walk &w, int64_t &end) {
  if (at.at >= at.total) return false;
  w.begin(a, at, 1);
  const int64_t start = at.at - w.u;
  end = start + w.s.cost(w.p, a.shift);
  return w.u > 0 && start >= first_unit(at.total, c, n);
}
// The blocks after c that have a part of that pair, in the order of the line
template <class F>
WQ_HD void parts_after(int64_t total, int64_t c, int64_t n, int64_t end, F &&f) {
  int64_t lo = first_unit(total, c + 1, n);
  for (int64_t k = c + 1; k < n && lo < end; ++k) {
    const int64_t hi = first_unit(total, k + 1, n);
    if (lo < hi) f(k);  // not a block without units
    lo = hi;
  }
}

}  // namespace wq
