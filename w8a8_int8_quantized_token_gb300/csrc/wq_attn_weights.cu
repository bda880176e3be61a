// Accumulated attention weight of the keys of a paged cache (tcgen05, sm_103a).
//
//   w[b][h][i] = decay w[b][h][i] + sum_{rows r that see key i} exp(c q_r.k_i - lse_r)
//
// over the new tokens' rows r = (token, query head of group h) of sequence b,
// whose log-sum-exp the attention over the same keys has left.
//
// The scores are taken as S^T = K Q^T: 128 keys are the rows of a tensor-memory
// tile and up to 128 query rows its columns.  So a thread owns a key and sums
// along its columns: no sum crosses threads, a masked or unwritten key spoils
// nothing but its own row, and nothing has to be cleared.  Two key tiles share
// every query tile that is loaded.
//   warps 0-3, 4-7  weights of key tile 0, 1 of a pair: a thread owns a key
//   warp 8          TMA: key tiles page by page, query tiles
//   warps 9, 10     MMA issue for key tile 0, 1: a thread each, whose waits (over
//                   100 cycles, even for nothing) then pass in the other's
//                   products; warp 9 owns the tensor memory
// Tensor memory: two score buffers of 128 columns for each key tile.
//
// A unit is a (sequence, key head, pair of key tiles, query tile); those in
// which no token sees a key are left out.  All units lie on one line, which the
// blocks cut into equal pieces (wq_weights_line.h), so that ragged lengths and the
// triangle of a prompt cost no idle SMs.  Where the cut falls between the query tiles of a
// pair, the parts of its sums go to the workspace and a second kernel adds them
// in the order of the line.  One query tile a sequence (decode) is never cut.
//
// Few rows: bound by HBM, every key read once; 64 sequences of up to 8192 keys (8
// heads of 128, one token each) take 103 us, 6.1 TB/s.  What let it get there:
// instructions a pair, since every role walks the pairs with one warp a
// scheduler, which takes about six cycles for each (135 us with the sequence, the
// pages and the log-sum-exps looked up pair by pair).
// Many rows: a step of 128 rows against a pair takes 1.3 us (a prompt of 4096
// tokens, 64 heads, 171 us).  Its products alone take 122 us, where their operands
// from shared memory let them, and the chain of waits, loads from tensor memory
// and sums without any exponential 158.  Shorter code helped (191 us with the loops
// over a tile's columns unrolled, 168 so); fewer ex2 (a part of them as polynomials,
// 179 us), 16 warps that weigh (179) and loads ahead (185) did not.
//
// Every wait on a memory barrier is bounded (1 s); on expiry the kernel records WQ_ERR_TIMEOUT,
// waits (bounded) for its own copies and MMAs, frees tensor memory and exits.
#include <algorithm>
#include <type_traits>

#include "wq_attn.cuh"
#include "wq_tc.cuh"

namespace wq {
namespace {

using namespace tc;
using attn::start_next_kernel;
using attn::wait_last_kernel;

constexpr int BK = 128, BR = 128;  // keys, query rows of a tile
constexpr int PAIR = kWeightsPair; // keys of a pair of tiles
static_assert(PAIR == 2 * BK, "a pair of key tiles");
constexpr int NTHREADS = 352;
constexpr int WARP_TMA = 8, WARP_MMA = 9;  // MMA: two warps
constexpr int MAX_BLOCKS = 152;    // one block an SM
constexpr int BATCH = 4;           // query tiles whose log-sum-exps are staged together

// Shared memory: a sequence of one query tile takes two of as many rows as they
// have (a decode step's have 16), and as many key tiles as fit beside them; one
// of many takes the keys of one pair and as many query tiles as fit, since they
// come one a step and from L2 (two of them: 1.42 us a step without a
// single exponential).
template <int D>
struct Plan {
  static constexpr int CH = D / 64;              // 128-byte column chunks
  static constexpr int KB = BK * D * 2;          // bytes of a key tile
  static constexpr int NK = 8, NQ = 8;           // key and query tiles in flight, at most
  static constexpr int B_K_FULL = 0, B_K_EMPTY = NK, B_Q_FULL = 2 * NK, B_Q_EMPTY = B_Q_FULL + NQ,
                       B_S_FULL = B_Q_EMPTY + NQ,  // [key tile][buffer]
                       B_S_EMPTY = B_S_FULL + 4, B_DONE = B_S_EMPTY + 4, NBAR = B_DONE + 2;
  static constexpr int OFF_LSE = 0;              // [2 key tiles][2][BATCH][BR] float
  static constexpr int OFF_BAR = OFF_LSE + 2 * 2 * BATCH * BR * 4;
  static constexpr int OFF_START = OFF_BAR + (NBAR + 1) / 2 * 16;  // sequence and offset of the block's first unit
  static constexpr int OFF_SCAN = OFF_START + 16;                  // sums of the warps
  static constexpr int OFF_TMEM = OFF_SCAN + (NTHREADS / 32) * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int OFF_Q = 9216;
  static_assert(OFF_ABORT + 4 <= OFF_Q && OFF_Q % 1024 == 0, "shared memory plan");
  static constexpr int MOST = 232448 - 1024;     // the rest aligns the tiles
  static __host__ __device__ constexpr int query_bytes(int cols) { return cols * D * 2; }
  static __host__ __device__ int query_tiles(int cols, bool many) {
    const int n = (MOST - OFF_Q - 2 * KB) / query_bytes(cols);
    return many ? (n < NQ ? n : NQ) : 2;
  }
  static __host__ __device__ int key_tiles(int cols, bool many) {
    const int n = (MOST - OFF_Q - query_tiles(cols, many) * query_bytes(cols)) / KB;
    return n < NK ? n : NK;
  }
  static int smem(int cols, bool many) {
    return OFF_Q + query_tiles(cols, many) * query_bytes(cols) + key_tiles(cols, many) * KB + 1024;
  }
};

// Place at = f(length of the line), found by the whole block.  The sequences out
// of range are told of.
template <class F>
__device__ __forceinline__ Place locate(const WeightArgs &a, int64_t *scan, int64_t *out, bool tell,
                                        F &&f) {
  const int threads = int(blockDim.x), per = (a.B + threads - 1) / threads, b0 = threadIdx.x * per;
  auto cost = [&](int b, bool say) {
    const int c0 = first_of(a, b), c1 = first_of(a, b + 1), l = a.key_len[b];
    const Seq s = seq_of(a, c0, c1, l);
    if (say && !in_range(a, s, c0, c1, l)) set_status(a.status, WQ_ERR_INDEX);
    return s.before(s.pairs, a.shift) * a.heads;
  };
  int64_t own = 0;
  for (int b = b0; b < min(b0 + per, a.B); ++b) own += cost(b, tell);
  int64_t sum = own;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) scan[warp] = sum;
  __syncthreads();
  int64_t total = 0, base = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
  const int64_t at = f(total);
  sum += base;
  if (at >= sum - own && at < sum) {
    int64_t left = at - (sum - own);
    int b = b0;
    for (int64_t c; left >= (c = cost(b, false)); ++b) left -= c;
    out[0] = b;
    out[1] = left;
  }
  __syncthreads();
  Place p{int(out[0]), out[1], total, at};
  return p;
}

template <class DT>
constexpr uint32_t kTypes = std::is_same<DT, Bf16>::value ? (1u << 7) | (1u << 10) : 0u;

// -lse in base 2, to be added to scores in base 2.  A row that saw no key
// (lse = -inf) gives no weight, as one of lse = inf does.
__device__ __forceinline__ float neg_lse2(float l) {
  constexpr float hi = 1.44269502162933349609375f, lo = 1.92596299112661746887e-8f;  // log2(e) in two parts
  if (fabsf(l) == INFINITY) return -INFINITY;
  return __fmaf_rn(-l, hi, __fmul_rn(-l, lo));
}

// The weight of key i
__device__ __forceinline__ float *weight_at(const WeightArgs &a, int b, int h, int i) {
  return a.w + b * a.w_seq + h * a.w_head + i;
}

template <class DT, int D, bool MANY>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmK, const WeightArgs a) {
  using P = Plan<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::OFF_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + P::OFF_TMEM);
  auto bar = [&](int i) { return base + P::OFF_BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  start_next_kernel();
  if (threadIdx.x == 0) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    *abort_flag = 0;
    for (int i = 0; i < P::NBAR; ++i) mbar_init(bar(i), i >= P::B_S_EMPTY && i < P::B_DONE   ? 4   // warps of a key tile
                        : (i >= P::B_K_EMPTY && i < P::B_Q_FULL) || (i >= P::B_Q_EMPTY && i < P::B_S_FULL) ? 2  // MMA warps
                                                               : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  const Place at = locate(a, reinterpret_cast<int64_t *>(sm + P::OFF_SCAN),
                          reinterpret_cast<int64_t *>(sm + P::OFF_START), blockIdx.x == 0,
                          [](int64_t total) { return first_unit(total, blockIdx.x, gridDim.x); });
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk;
  walk.begin(a, at, first_unit(at.total, blockIdx.x + 1, gridDim.x) - at.at);
  const int tpt = a.tpt;
  const uint32_t nk = uint32_t(P::key_tiles(a.cols, MANY)), nq = uint32_t(P::query_tiles(a.cols, MANY));
  const uint32_t qbytes = uint32_t(P::query_bytes(a.cols)), off_k = P::OFF_Q + nq * qbytes;
  bool ok = true;                // this role's waits all ended in time

  if (warp == WARP_TMA) {
    // -------------------------------------------------------------- copies
    const bool leader = elect_one();
    uint32_t kt = 0, qt = 0;  // key and query tiles so far
    uint32_t ks = 0, kp = 1, qs = 0, qp = 1;  // their slots and the parities of the slots' releases
    const int nbox = BK / a.box;
    bool bad = false;  // a page id outside the cache
    // Lane L looks up box L of a pair, one pair ahead of its copies, and starts
    // them
    const int mine = lane < nbox ? 0 : 1;  // its key tile
    const uint32_t box_at = uint32_t((lane - mine * nbox) * a.box * 128);
    Piece p, nx;
    bool more = walk.next(a, p);
    int pi = 0, place = 0;  // of this lane's box
    auto begin = [&](const Piece &q) {
      const int key = q.k0 + lane * a.box;
      pi = key / a.page_size;
      place = key - pi * a.page_size;
      return lane < 2 * nbox && key < q.s.len ? a.page_table[q.b * a.ld_table + pi] : 0;
    };
    int page = more ? begin(p) : 0;
    while (more && ok) {
      const bool again = walk.next(a, nx);
      const int32_t *pages = a.page_table + p.b * a.ld_table;
#pragma unroll 1
      for (int k = 0; k < p.pairs && ok; ++k) {
        const int k0 = p.k0 + k * PAIR, y = place;
        int w = page;
        if (unsigned(w) >= unsigned(a.num_pages)) {  // read outside the tensor: zeros
          w = int(a.num_pages);
          bad = true;
        }
        if (k + 1 < p.pairs) {
          pi += a.step_pages;
          place += a.step_place;
          if (place >= a.page_size) place -= a.page_size, ++pi;
          page = lane < 2 * nbox && k0 + PAIR + lane * a.box < p.s.len ? pages[pi] : 0;
        } else if (again) {
          page = begin(nx);
        }
        if (p.qb == p.qa) continue;  // no token: nothing to multiply
        const bool on = lane < 2 * nbox && k0 + lane * a.box < p.s.len;
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {
          const int boxes = min(nbox, (p.s.len - k0 - g * BK + a.box - 1) / a.box);
          if (boxes <= 0) break;
          if (!(ok = wait_warp(bar(P::B_K_EMPTY) + 8 * ks, kp, abort_flag))) break;
          const uint32_t full = bar(P::B_K_FULL) + 8 * ks, dst = base + off_k + ks * P::KB + box_at;
          if (leader) mbar_expect_tx(full, uint32_t(boxes * a.box * P::CH * 128));
          __syncwarp();
          if (on && mine == g) {
#pragma unroll
            for (int ch = 0; ch < P::CH; ++ch) tma_load_4d(dst + ch * BK * 128, &tmK, ch * 64, y, p.h, w, full);
          }
          if (++ks == nk) ks = 0, kp ^= 1;
          ++kt;
        }
        if (k > 0) continue;  // the query tile is there
#pragma unroll 1
        for (int q = p.qa; q < p.qb && ok; ++q) {
          if (!(ok = wait_warp(bar(P::B_Q_EMPTY) + 8 * qs, qp, abort_flag))) break;
          if (leader) {
            const uint32_t full = bar(P::B_Q_FULL) + 8 * qs;
            mbar_expect_tx(full, uint32_t(P::CH * tpt * a.G * 128));
#pragma unroll
            for (int ch = 0; ch < P::CH; ++ch)
              tma_load_3d(base + P::OFF_Q + qs * qbytes + ch * a.cols * 128, &tmQ, ch * 64, p.h * a.G,
                          p.s.t0 + q * tpt, full);
          }
          if (++qs == nq) qs = 0, qp ^= 1;
          ++qt;
        }
      }
      p = nx;
      more = again;
    }
    if (bad) set_status(a.status, WQ_ERR_INDEX);
    if (!ok) {  // let copies already in flight land before the block goes away
      *abort_flag = 1;
      for (uint32_t i = kt > nk ? kt - nk : 0; i < kt; ++i)
        mbar_wait_bounded(bar(P::B_K_FULL + int(i % nk)), (i / nk) & 1);
      for (uint32_t i = qt > nq ? qt - nq : 0; i < qt; ++i)
        mbar_wait_bounded(bar(P::B_Q_FULL + int(i % nq)), (i / nq) & 1);
    }
  } else if (warp >= WARP_MMA) {
    // -------------------------------------------------------------- products
    const int g = warp - WARP_MMA;  // key tile
    if (elect_one()) {
      const uint32_t idesc = idesc_f16(BK, a.cols) | kTypes<DT>;
      const int steps = (a.dk + 15) / 16;
      const uint64_t dq0 = sdesc(base + P::OFF_Q), dk0 = sdesc(base + off_k);
      const uint32_t dq1 = uint32_t(a.cols * 128) >> 4;  // to a query tile's next 64 columns
      uint32_t ks = 0, kp = 0, qs = 0, qp = 0, st = 0;
      auto wait = [&](uint32_t b, uint32_t parity) {
        if (ok) ok = wait_one(b, parity, abort_flag);
      };
      Piece p;
      while (ok && walk.next(a, p)) {
        if (p.qb == p.qa) continue;
#pragma unroll 1
        for (int k = 0; k < p.pairs && ok; ++k) {
          const bool two = p.k0 + k * PAIR + BK < p.s.len, tile = g == 0 || two;
          // Both warps wait for both key tiles and for every query tile, and
          // both release them, with work for them or without: a wait by parity
          // cannot tell a phase from the one two before it, so none may be
          // passed over, and no slot may be filled again before both have seen it.
          const uint32_t k1 = ks + 1 == nk ? 0 : ks + 1, kp1 = k1 == 0 ? kp ^ 1 : kp;
          wait(bar(P::B_K_FULL) + 8 * ks, kp);
          if (two) wait(bar(P::B_K_FULL) + 8 * k1, kp1);
          const uint32_t kg = g ? k1 : ks, other = g ? ks : k1;
          if (ok && (g || two)) mbar_arrive(bar(P::B_K_EMPTY) + 8 * other);
          const uint64_t dk = dk0 + kg * uint32_t(P::KB >> 4);
#pragma unroll 1
          for (int q = p.qa; q < p.qb; ++q) {
            const bool done = k + 1 == p.pairs;  // with the query tile
            if (k == 0) wait(bar(P::B_Q_FULL) + 8 * qs, qp);
            if (tile) {
              const uint32_t buf = st & 1;
              wait(bar(P::B_S_EMPTY + 2 * g) + 8 * buf, ((st >> 1) & 1) ^ 1);
              tc_fence_after();
              if (ok) {
                const uint64_t dq = dq0 + qs * (qbytes >> 4);
                const uint32_t to = tmem + g * 256 + buf * 128;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  if (i >= steps) break;
                  mma_f16(to, dk + (((i / 4) * (BK * 128) + (i % 4) * 32) >> 4),
                          dq + (i / 4) * dq1 + ((i % 4) * 32 >> 4), idesc, i ? 1u : 0u);
                }
                if (q + 1 == p.qb) mma_commit(bar(P::B_K_EMPTY) + 8 * kg);
                if (done) mma_commit(bar(P::B_Q_EMPTY) + 8 * qs);
                mma_commit(bar(P::B_S_FULL + 2 * g) + 8 * buf);
              }
              ++st;
            } else if (done && ok) {
              mma_commit(bar(P::B_Q_EMPTY) + 8 * qs);  // products of the pairs before may still read it
            }
            if (done && ++qs == nq) qs = 0, qp ^= 1;
          }
          ks = two ? k1 : ks;
          kp = two ? kp1 : kp;
          if (++ks == nk) ks = 0, kp ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
      mma_commit(bar(P::B_DONE + g));
      mbar_wait_bounded(bar(P::B_DONE + g), 0);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- weights
    const int g = warp >> 2, tid = threadIdx.x & 127, col = g * BK + tid;
    const uint32_t ts = tmem + (uint32_t((warp & 3) * 32) << 16) + g * 256;
    float *ls = reinterpret_cast<float *>(sm + P::OFF_LSE) + g * 2 * BATCH * BR;
    const int tok = tid / a.G, hd = tid - tok * a.G;  // the column whose lse this thread brings
    const float c = a.scale_log2;
    constexpr int LB = MANY ? BATCH : 1;
    uint32_t st = 0, ql = 0;  // score tiles, and batches of query tiles' log-sum-exps so far
    float l[LB];
    auto lse_of = [&](const Piece &q, int tile) {
#pragma unroll
      for (int e = 0; e < LB; ++e) {
        const int j = (tile + e) * tpt + tok;
        l[e] = tok < tpt && j < q.s.n ? a.lse[int64_t(q.s.t0 + j) * a.Hq + q.h * a.G + hd] : INFINITY;
      }
    };
    // what a key had before
    auto look = [&](const Piece &q, int k0) {
      return q.whole && k0 + col < q.s.old ? *weight_at(a, q.b, q.h, k0 + col) : 0.0f;
    };
    // Adds the weights of the columns of a score tile in v; lb: their rows'
    // log-sum-exps.  All of them, or those in [lo, hi).
    Pair s0, s1;
    auto weigh = [&](auto &v, const float *lb) {
      const Pair cc = pair(c, c);
      float x, y;
#pragma unroll
      for (int e = 0; e < int(sizeof(v) / 4); e += 4) {
        const float4 n = *reinterpret_cast<const float4 *>(lb + e);
        split(fma_p(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), cc, pair(n.x, n.y)), x, y);
        s0 = add_p(s0, pair(ex2(x), ex2(y)));
        split(fma_p(pair(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), cc, pair(n.z, n.w)), x, y);
        s1 = add_p(s1, pair(ex2(x), ex2(y)));
      }
    };
    auto weigh_some = [&](auto &v, const float *lb, int lo, int hi) {
#pragma unroll
      for (int e = 0; e < int(sizeof(v) / 4); e += 2) {
        const float x = ex2(__fmaf_rn(__uint_as_float(v[e]), c, lb[e]));
        const float y = ex2(__fmaf_rn(__uint_as_float(v[e + 1]), c, lb[e + 1]));
        s0 = add_p(s0, pair(e >= lo && e < hi ? x : 0.0f, e + 1 >= lo && e + 1 < hi ? y : 0.0f));
      }
    };
    Piece p, nx;
    bool more = walk.next(a, p);
    float old = more ? look(p, p.k0) : 0.0f;
    if (more) lse_of(p, p.qa);
    // A warp whose wait ran out goes on to the next barrier of its key tile's
    // warps, without work, and they leave together: none is left there by one
    // that saw the scores in time or did not.
    bool go = true;
    while (more && go) {
      const bool again = walk.next(a, nx);
      float *to = weight_at(a, p.b, p.h, p.k0 + col);
#pragma unroll 1
      for (int k = 0; k < p.pairs && go; ++k) {
        const int k0 = p.k0 + k * PAIR, i = k0 + col;
        const float was = old;
        if (k + 1 < p.pairs) old = look(p, k0 + PAIR);
        else if (again) old = look(nx, nx.k0);
        const bool tile = k0 + g * BK < p.s.len;
        float sum = 0.0f;
#pragma unroll 1
        for (int q = p.qa; q < p.qb; ++q) {
          const int batch = LB > 1 ? (q - p.qa) % LB : 0;
          if (k == 0 && batch == 0) {  // the rows' log-sum-exps, the next batch's ahead
            ++ql;
#pragma unroll
            for (int e = 0; e < LB; ++e) ls[((ql & 1) * LB + e) * BR + tid] = neg_lse2(l[e]);
            if (q + LB < p.qb) lse_of(p, q + LB);
            else if (again) lse_of(nx, nx.qa);
            // two batches on, all have read what was here
            if (!(go = named_sync_and(1 + g, 128, ok))) break;
          }
          if (!tile || !ok) continue;
          const float *lb = ls + ((ql & 1) * LB + batch) * BR;
          const uint32_t buf = st & 1, at = ts + buf * 128;
          if (!(ok = wait_warp(bar(P::B_S_FULL + 2 * g) + 8 * buf, (st >> 1) & 1, abort_flag))) {
            *abort_flag = 1;
            continue;
          }
          tc_fence_after();
          // columns of the tile that count: its tokens', from the first that sees
          // this key on (those that no row fills hold whatever was there)
          const int hi = min(tpt, p.s.n - q * tpt) * a.G;
          const int lo = min(max(0, i - p.s.old - q * tpt), tpt) * a.G;
          const bool seen = __all_sync(0xffffffffu, lo == 0);  // by all tokens, all keys of the warp
          s0 = s1 = pair(0.0f, 0.0f);
          // Loops of little code: unrolled, with the next columns' loads ahead,
          // they take longer (prompt of 4096: 174 -> 208 us).
          if (hi <= 8) {
            uint32_t v[8];
            tmem_ld8(at, v);
            tmem_wait_ld(v);
            if (seen && hi == 8) weigh(v, lb);
            else weigh_some(v, lb, lo, hi);
          } else {
            int e = 0;
            if (seen) {
#pragma unroll 1
              for (; e + 32 <= hi; e += 32) {
                uint32_t v[32];
                tmem_ld32(at + e, v);
                wait_ld32(v);
                weigh(v, lb + e);
              }
            }
#pragma unroll 1
            for (; e < hi; e += 32) {
              uint32_t v[32];
              tmem_ld32(at + e, v);
              wait_ld32(v);
              weigh_some(v, lb + e, lo - e, hi - e);
            }
          }
          float x, y;
          split(add_p(s0, s1), x, y);
          sum += x + y;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(P::B_S_EMPTY + 2 * g) + 8 * buf);
          ++st;
        }
        if (go && ok && i < p.s.len) {
          if (!p.whole) a.part[(int64_t(blockIdx.x) * 2 + p.slot) * PAIR + col] = sum;
          else to[k * PAIR] = __fmaf_rn(a.decay, was, sum);
        }
      }
      if (p.qa == p.qb && again) lse_of(nx, nx.qa);  // no token here
      p = nx;
      more = again;
    }
  }
  if (!ok) {
    *abort_flag = 1;
    set_status(a.status, WQ_ERR_TIMEOUT);
  }
  __syncthreads();  // the products are over
  if (warp == WARP_MMA) tmem_dealloc(tmem, 512);
}

// Adds the parts of the pair that block c of the first kernel began and left
// to the blocks after it, in their order: a thread a key.
__global__ void __launch_bounds__(PAIR) attn_weights_join_kernel(const WeightArgs a) {
  __shared__ int64_t scan[PAIR / 32], out[2];
  const int64_t blocks = gridDim.x + 1, c = blockIdx.x;
  const Place at = locate(a, scan, out, false, [&](int64_t total) { return first_unit(total, c + 1, blocks); });
  wait_last_kernel();  // in every block: what follows the join may then rely on both
  Walk w;
  int64_t end;
  if (!left_to_others(a, at, c, blocks, w, end)) return;
  const int i = w.p * PAIR + threadIdx.x;
  if (i >= w.s.len) return;
  float sum = a.part[(c * 2 + 1) * PAIR + threadIdx.x];
  parts_after(at.total, c, blocks, end, [&](int64_t k) { sum += a.part[k * 2 * PAIR + threadIdx.x]; });
  float *to = weight_at(a, w.b, w.h, i);
  *to = __fmaf_rn(a.decay, i < w.s.old ? *to : 0.0f, sum);
}

// Any page size and pitch: a block takes 32 keys of one head, a lane a key; the
// warps share the rows, and add their sums in the order of the warps.  Bound by two
// shared-memory reads a product: 16 sequences of 4096 keys, 8 key heads of 8 and 128
// elements, 160 us with pages of one key, where the kernel above takes 35 with 16.
template <class DT>
__global__ void __launch_bounds__(256) attn_weights_any_kernel(const WeightArgs a) {
  constexpr int KT = 32, NW = 8;
  __shared__ float ks[KT][129];
  __shared__ float qs[NW][128];
  __shared__ float part[NW][KT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = (a.max_len + KT - 1) / KT;
  const int tile = int(blockIdx.x % unsigned(tiles)), bh = int(blockIdx.x / unsigned(tiles));
  const int b = bh / a.heads, h = bh - b * a.heads;
  const int c0 = first_of(a, b), c1 = first_of(a, b + 1), l = a.key_len[b];
  const Seq s = seq_of(a, c0, c1, l);
  if (tile == 0 && h == 0 && threadIdx.x == 0 && !in_range(a, s, c0, c1, l)) set_status(a.status, WQ_ERR_INDEX);
  const int k0 = tile * KT, i = k0 + lane;
  if (k0 >= s.len) return;
  for (int r = warp; r < KT; r += NW) {
    const int key = k0 + r;
    int page = key < s.len ? a.page_table[b * a.ld_table + key / a.page_size] : 0;
    const bool good = key < s.len && unsigned(page) < unsigned(a.num_pages);
    if (key < s.len && !good) {
      set_status(a.status, WQ_ERR_INDEX);
      page = 0;
    }
    const uint16_t *k = a.k + page * a.k_page + h * a.k_head + key % a.page_size * a.k_token;
    for (int d = lane; d < a.dk; d += 32) ks[r][d] = good ? DT::to_f(k[d]) : 0.0f;
  }
  __syncthreads();
  float sum = 0.0f;
  const int64_t rows = int64_t(s.n) * a.G;
  for (int64_t r = warp; r < rows; r += NW) {
    const int j = int(r / a.G), hd = h * a.G + int(r - int64_t(j) * a.G);
    if (s.old + j < k0) continue;  // sees none of these keys
    const uint16_t *q = a.q + (s.t0 + j) * a.q_token + hd * a.q_head;
    __syncwarp();
    for (int d = lane; d < a.dk; d += 32) qs[warp][d] = DT::to_f(q[d]);
    __syncwarp();
    float x = 0.0f;
    for (int d = 0; d < a.dk; ++d) x = __fmaf_rn(qs[warp][d], ks[lane][d], x);
    x = ex2(__fmaf_rn(x, a.scale_log2, neg_lse2(a.lse[int64_t(s.t0 + j) * a.Hq + hd])));
    if (i <= s.old + j) sum += x;
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && i < s.len) {
    sum = 0.0f;
    for (int w = 0; w < NW; ++w) sum += part[w][lane];
    float *to = weight_at(a, b, h, i);
    *to = __fmaf_rn(a.decay, i < s.old ? *to : 0.0f, sum);
  }
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <class DT, int D, bool MANY>
int launch_tiles(const WeightArgs &a, cudaStream_t st) {
  auto *k = attn_weights_kernel<DT, D, MANY>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, Plan<D>::MOST + 1024)) return WQ_ERR_LAUNCH;
  CUtensorMap mq, mk;
  auto pitch = [](int64_t extent, int64_t stride) { return extent == 1 && stride == 0 ? 8 : stride; };
  const int64_t qd[3] = {a.dk, a.Hq, a.T};
  const int64_t qs[2] = {pitch(a.Hq, a.q_head), pitch(a.T, a.q_token)};
  const int qb[3] = {64, a.G, a.tpt};
  const int box[4] = {64, a.box, 1, 1};
  const int64_t kd[4] = {a.dk, a.page_size, a.heads, a.num_pages};
  const int64_t ks[3] = {pitch(a.page_size, a.k_token), pitch(a.heads, a.k_head), pitch(a.num_pages, a.k_page)};
  if (!make_tma_nd_b16_sw128(&mq, a.q, 3, qd, qs, qb) || !make_tma_nd_b16_sw128(&mk, a.k, 4, kd, ks, box))
    return WQ_ERR_UNSUPPORTED;
  k<<<unsigned(a.blocks), NTHREADS, Plan<D>::smem(a.cols, MANY), st>>>(mq, mk, a);
  int rc = launched(1);
  if (rc == WQ_OK && MANY && a.blocks > 1)
    rc = attn::launch_chained(attn_weights_join_kernel, unsigned(a.blocks - 1), PAIR, 0, true, st, a);
  return rc;
}

template <class DT>
int launch_t(const WeightArgs &a, cudaStream_t st) {
  if (a.tiles && a.split) return a.dk > 64 ? launch_tiles<DT, 128, true>(a, st) : launch_tiles<DT, 64, true>(a, st);
  if (a.tiles) return a.dk > 64 ? launch_tiles<DT, 128, false>(a, st) : launch_tiles<DT, 64, false>(a, st);
  const int64_t blocks = int64_t(a.B) * a.heads * ((a.max_len + 31) / 32);
  if (blocks >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  attn_weights_any_kernel<DT><<<unsigned(blocks), 256, 0, st>>>(a);
  return launched(1);
}

}  // namespace

// Query tiles of as many tokens as fill 128 rows, no more than a sequence may
// have (a decode step's tile is 16 columns wide, not 128).
void plan_weights(WeightArgs &a) {
  a.tpt = std::max(1, std::min(BR / a.G, a.max_q));
  a.shift = 0;
  while ((2 << a.shift) <= a.tpt) ++a.shift;
  a.cols = (a.tpt * a.G + 15) / 16 * 16;
  a.box = gcd(a.page_size, BK);
  a.step_pages = PAIR / a.page_size;
  a.step_place = PAIR % a.page_size;
  const bool pitches = (a.k_token || a.page_size == 1) && (a.k_head || a.heads == 1) &&
                       (a.k_page || a.num_pages <= 1);
  // TMA boxes of 8 keys or more, a lane for each box of a pair; pitches other
  // than zero; waits that end after 1 s, which 2^25 keys do not reach
  a.tiles = a.T > 0 && a.page_size % 8 == 0 && a.num_pages > 0 && pitches && a.max_len <= (1 << 25);
  const int64_t most = int64_t(a.B) * a.heads * ((a.max_len + PAIR - 1) / PAIR) *
                       std::max(1, (a.max_q + a.tpt - 1) / a.tpt);
  a.blocks = int(std::max<int64_t>(1, std::min<int64_t>(MAX_BLOCKS, most)));
  a.split = a.tiles && a.max_q > a.tpt;
}

size_t weights_ws_bytes(const WeightArgs &a) {
  return a.split ? size_t(a.blocks) * 2 * PAIR * sizeof(float) : 0;
}

int launch_weights(const WeightArgs &a, int dtype, cudaStream_t st) {
  return dtype == WQ_DT_BF16 ? launch_t<Bf16>(a, st) : launch_t<F16>(a, st);
}

}  // namespace wq
