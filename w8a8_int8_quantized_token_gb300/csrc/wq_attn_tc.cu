// Attention over a paged cache for many query rows (tcgen05, sm_103a): two
// tiles of 128 rows of one key head share every key and value tile.
//
//   S = Q K^T (128 x 128, float32 in tensor memory),  P = exp2(c S - c m),
//   O += P V,  l += row sums of P,  at the end O / l and its log-sum-exp.
//
// Rows are (token, query head of the group) pairs, so that every query head
// of a group uses the keys that are loaded once.  Tiles of the two row tiles
// alternate on the tensor cores: while one tile's scores are exponentiated,
// the other's products run.
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread owns one row
//   warp 8          tensor memory and MMA issue (one thread)
//   warp 9          TMA: queries, and keys and values page by page
//   warps 10, 11    none (the third warpgroup gives its registers to the others)
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D each).  P takes the
// place of its S (64 columns, 16-bit pairs) as the A operand of the second
// product.  O is rescaled only when a row's maximum has grown by more than
// 2^8 over the one in use: until then the weights are at most 2^8, their sum
// stays exact in the same sense, and the final division removes the factor.
//
// The range is cut two ways.  The prefix is the same for all tokens: its
// (key head, row tile pair) items times 128-key tiles form one line of equal
// units, which the blocks cut into equal pieces, so a piece may end inside an
// item and begin the next; each piece leaves a partial result.  Suffixes: a
// block per (range, sequence, key head, row tile pair).
//
// Values past the end of a range may be anything (a page is shared with
// unwritten places), and 0 * NaN is NaN: the last tile's tail is cleared in
// shared memory before its product.
//
// Every wait is bounded (1 s); on expiry the kernel records WQ_ERR_TIMEOUT,
// waits (bounded) for its own copies and MMAs, frees tensor memory and exits.
#include <algorithm>
#include <type_traits>

#include "wq_attn.cuh"
#include "wq_tc.cuh"

namespace wq {
namespace {

using namespace tc;
using namespace attn;

constexpr int BM = 128, BN = 128;  // rows of a tile, keys of a tile
constexpr int NTHREADS = 384;
constexpr int WARP_MMA = 8, WARP_TMA = 9;  // of the third warpgroup; its other two warps idle
// Registers a thread: 3 x 168 at launch (the most for 384 threads), shared out
// as 2 x 216 for the softmax, which holds a row of 128 scores, and 72
constexpr int REGS_SOFTMAX = 216, REGS_OTHER = 72;
static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * 168, "a larger sum would wait forever");

template <int D>
struct Plan {
  static constexpr int CH = D / 64;              // 128-byte column chunks
  static constexpr int QB = BM * D * 2;          // bytes of one query tile
  static constexpr int KVB = BN * D * 2;         // bytes of a key or value tile
  static constexpr int NS = D == 128 ? 5 : 8;    // ring depth: keys and values in turn
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * QB;
  static constexpr int OFF_BAR = OFF_KV + NS * KVB;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_Q_FULL = 2 * NS, B_Q_EMPTY = B_Q_FULL + 1,
                       B_S = B_Q_EMPTY + 1,      // [2] scores of a row tile are in
      B_P = B_S + 2,                             // [2][2] half a tile of weights is in
      B_O = B_P + 4,                             // [2] a value product is done
      B_TAIL = B_O + 2,                          // a last value tile's tail is cleared
      B_DONE = B_TAIL + 1, NBAR = B_DONE + 1;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static_assert(SMEM <= 232448, "shared memory plan too large");
  static constexpr uint32_t T_O = 2 * BN;        // tensor-memory column of O0
  static_assert(2 * BN + 2 * D <= 512, "tensor memory plan");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// shared-memory matrix descriptor of the values: the columns (N) are
// contiguous, 64 of them in a 128-byte swizzled row; the next 64 columns lie
// one chunk (16 KB) on, the next 8 keys 1024 bytes on
__device__ __forceinline__ uint64_t sdesc_n(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(BN * 128 >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
template <class DT>
constexpr uint32_t kTypes = std::is_same<DT, Bf16>::value ? (1u << 7) | (1u << 10) : 0u;
constexpr uint32_t kBTransposed = 1u << 16;

template <class DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<DT, Bf16>::value) return bf16x2_rn(lo, hi);
  else return f16x2_rn(lo, hi);
}
__device__ __forceinline__ void fma2(float &a0, float &a1, float m, float c) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mov.b64 d, {%3, %3};\n"
      " fma.rn.f32x2 a, a, b, d;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(m), "f"(c));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// How the launch is cut (host values)
struct Cut {
  int tpt;            // tokens of a row tile: 128 / G
  int pairs_p;        // row tile pairs of the prefix (0: no prefix here)
  int units_p;        // 128-key tiles of the prefix
  int blocks_p;       // blocks that share the prefix's line of units
  int pairs_s;        // row tile pairs of a suffix (0: no suffixes here)
  int box;            // cache rows of one TMA box
  bool out16;         // out rows take 16-byte stores
};

// One piece of work: row tiles of a source against a key range
struct Piece {
  Source s;
  int head, tok0;     // key head; first token (of the source) of row tile 0
  int k0, k1;         // keys
  int slot, last;     // partial-result slot; slots (slot, last) stay empty
};

__device__ __forceinline__ Piece prefix_piece(const AttnArgs &a, const Cut &c, int64_t u0,
                                              int64_t u1, int block) {
  const int64_t total = int64_t(a.Hkv) * c.pairs_p * c.units_p;
  const int item = int(u0 / c.units_p);
  const int64_t start = int64_t(item) * c.units_p;
  Piece p;
  p.s = source_of(a, -1);
  p.head = item / c.pairs_p;
  p.tok0 = (item % c.pairs_p) * 2 * c.tpt;
  p.k0 = int(u0 - start) * BN;
  const int64_t e = u1 - start;
  p.k1 = e >= c.units_p ? a.P : int(e) * BN;
  // ordinal of this block among those that share the item
  const int first = int(((start + 1) * c.blocks_p - 1) / total);
  p.slot = block - first;
  p.last = p.k1 == a.P ? a.sp : p.slot + 1;
  return p;
}

__device__ __forceinline__ Piece suffix_piece(const AttnArgs &a, const Cut &c, int64_t it) {
  Piece p;
  const int pair = int(it % c.pairs_s);
  it /= c.pairs_s;
  p.head = int(it % a.Hkv);
  it /= a.Hkv;
  p.s = source_of(a, int(it % a.B));
  const int split = int(it / a.B);
  p.tok0 = pair * 2 * c.tpt;
  p.k0 = split * a.s_chunk;
  const int lastj = min(p.s.n, p.tok0 + 2 * c.tpt) - 1;
  p.k1 = min(min(p.s.len, visible(p.s, lastj)), p.k0 + a.s_chunk);
  p.slot = p.s.slot0 + split;
  p.last = p.slot + 1;
  return p;
}

template <class DT, int D>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttnArgs a, const Cut c) {
  using P = Plan<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::OFF_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + P::OFF_TMEM);
  auto bar = [&](int i) { return base + P::OFF_BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < P::NBAR; ++i) mbar_init(bar(i), i >= P::B_P && i < P::B_O ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    *abort_flag = 1;
    set_status(a.status, WQ_ERR_TIMEOUT);
  };

  // ---- this block's pieces, the same list for every role
  const bool line = int(blockIdx.x) < c.blocks_p;
  const int64_t total = int64_t(a.Hkv) * c.pairs_p * c.units_p;
  const int64_t u_begin = line ? int64_t(blockIdx.x) * total / c.blocks_p : 0;
  const int64_t u_end = line ? int64_t(blockIdx.x + 1) * total / c.blocks_p : 1;
  // calls f(piece, key tiles, row tiles in use); stops when f returns false
  auto pieces = [&](auto &&f) {
    for (int64_t u = u_begin; u < u_end;) {
      Piece p;
      if (line) {
        const int64_t stop = min((u / c.units_p + 1) * c.units_p, u_end);
        p = prefix_piece(a, c, u, stop, int(blockIdx.x));
        u = stop;
      } else {
        p = suffix_piece(a, c, int64_t(blockIdx.x) - c.blocks_p);
        u = u_end;
      }
      if (p.tok0 >= p.s.n) return;
      const int n = p.k1 > p.k0 ? (p.k1 - p.k0 + BN - 1) / BN : 0;
      if (!f(p, n, p.tok0 + c.tpt < p.s.n ? 2 : 1)) return;
    }
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == WARP_TMA) {
      // ------------------------------------------------------------ copies
      int g = 0;       // ring stages issued
      int q = 0;       // pieces with keys
      int tails = 0;
      bool ok = true;
      const int nbox = BN / c.box;
      auto wait = [&](int b, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_wait<200>(bar(b), parity, abort_flag))) return true;
        fail();
        ok = false;
        return false;
      };
      pieces([&](const Piece &p, int n, int tiles) {
        if (n == 0) return true;
        if (!wait(P::B_Q_EMPTY, (q & 1) ^ 1)) return false;
        if (lane == 0) {
          mbar_expect_tx(bar(P::B_Q_FULL), uint32_t(tiles * P::CH * c.tpt * a.G * 128));
          for (int t = 0; t < tiles; ++t)
            for (int ch = 0; ch < P::CH; ++ch)
              tma_load_3d(base + P::OFF_Q + t * P::QB + ch * BM * 128, &tmQ, ch * 64, p.head * a.G,
                          p.s.t0 + p.tok0 + t * c.tpt, bar(P::B_Q_FULL));
        }
        ++q;
        for (int j = 0; j < n; ++j) {
          const int kb = p.k0 + j * BN;
          const int boxes = min(nbox, (p.k1 - kb + c.box - 1) / c.box);  // with a key in range
          // lane b looks box b up; a bad page is read outside the tensor: zeros
          int page = int(a.num_pages), place = 0;
          if (lane < boxes) {
            const int key = kb + lane * c.box, pi = key / a.page_size;
            place = key - pi * a.page_size;
            page = p.s.pages[pi];
            if (page < 0 || page >= a.num_pages) {
              set_status(a.status, WQ_ERR_INDEX);
              page = int(a.num_pages);
            }
          }
          for (int kv = 0; kv < 2; ++kv, ++g) {
            const int s = g % P::NS;
            if (!wait(P::B_EMPTY + s, ((g / P::NS) & 1) ^ 1)) return false;
            const uint32_t dst = base + P::OFF_KV + uint32_t(s * P::KVB);
            if (lane == 0) mbar_expect_tx(bar(P::B_FULL + s), uint32_t(boxes * c.box * P::CH * 128));
            __syncwarp();
            if (lane < boxes) {
  #pragma unroll
              for (int ch = 0; ch < P::CH; ++ch)
                tma_load_4d(dst + uint32_t(ch * BN + lane * c.box) * 128, kv ? &tmV : &tmK, ch * 64,
                            place, p.head, page, bar(P::B_FULL + s));
            }
            __syncwarp();
            if (kv && kb + BN > p.k1) {
              // clear the values past the range, once the copies are in
              if (!wait(P::B_FULL + s, (g / P::NS) & 1)) {
                ++g;
                return false;
              }
              uint8_t *v = sm + P::OFF_KV + s * P::KVB;
              const int r0 = p.k1 - kb;
              for (int i = lane; i < (BN - r0) * 8 * P::CH; i += 32) {
                const int row = i / (8 * P::CH), ch = i % (8 * P::CH);
                *reinterpret_cast<uint4 *>(v + ((ch / 8) * BN + r0 + row) * 128 + (ch % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
              fence_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(P::B_TAIL));
              ++tails;
            }
          }
        }
        return true;
      });
      if (!ok) {  // let copies already in flight land before the block goes away
        if (q > 0) mbar_wait_bounded(bar(P::B_Q_FULL), (q - 1) & 1);
        for (int i = g > P::NS ? g - P::NS : 0; i < g; ++i)
          mbar_wait_bounded(bar(P::B_FULL + i % P::NS), (i / P::NS) & 1);
      }
    } else if (warp == WARP_MMA) {
      // ------------------------------------------------------------ products
      if (lane == 0) {
        constexpr uint32_t id_s = idesc_f16(BM, BN) | kTypes<DT>;
        constexpr uint32_t id_o = idesc_f16(BM, D) | kTypes<DT> | kBTransposed;
        int g = 0, q = 0, tails = 0;
        int done[2] = {0, 0};  // key tiles each row tile has worked on
        auto wait = [&](int b, uint32_t parity) {
          if (mbar_wait(bar(b), parity, abort_flag)) return true;
          fail();
          return false;
        };
        auto scores = [&](int t, int stage) {
          const uint32_t qa = base + P::OFF_Q + t * P::QB, ka = base + P::OFF_KV + uint32_t(stage * P::KVB);
  #pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = uint32_t(k / 4) * (BM * 128) + uint32_t(k % 4) * 32;
            mma_f16(tmem + t * BN, sdesc(qa + o), sdesc(ka + o), id_s, k ? 1u : 0u);
          }
          mma_commit(bar(P::B_S + t));
        };
        pieces([&](const Piece &p, int n, int tiles) {
          if (n == 0) return true;
          if (!wait(P::B_Q_FULL, q & 1)) return false;
          ++q;
          if (!wait(P::B_FULL + g % P::NS, (g / P::NS) & 1)) return false;
          tc_fence_after();
          for (int t = 0; t < tiles; ++t) scores(t, g % P::NS);
          mma_commit(bar(P::B_EMPTY + g % P::NS));
          ++g;
          for (int j = 0; j < n; ++j) {
            const int sv = g % P::NS, sk = (g + 1) % P::NS;
            if (!wait(P::B_FULL + sv, (g / P::NS) & 1)) return false;
            if (p.k0 + (j + 1) * BN > p.k1) {
              if (!wait(P::B_TAIL, tails & 1)) return false;
              ++tails;
            }
            const uint32_t va = base + P::OFF_KV + uint32_t(sv * P::KVB);
            for (int t = 0; t < tiles; ++t) {
              const uint32_t ph = done[t] & 1;
  #pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (!wait(P::B_P + 2 * t + h, ph)) return false;
                tc_fence_after();
  #pragma unroll
                for (int k = 4 * h; k < 4 * h + 4; ++k)
                  mma_f16_ts(tmem + P::T_O + t * D, tmem + t * BN + 8 * k, sdesc_n(va + 2048 * k), id_o,
                             (j | k) ? 1u : 0u);
              }
              mma_commit(bar(P::B_O + t));
              ++done[t];
              if (j + 1 < n) {
                if (!wait(P::B_FULL + sk, ((g + 1) / P::NS) & 1)) return false;
                tc_fence_after();
                scores(t, sk);
              }
            }
            mma_commit(bar(P::B_EMPTY + sv));
            if (j + 1 < n) mma_commit(bar(P::B_EMPTY + sk));
            g += j + 1 < n ? 2 : 1;
          }
          mma_commit(bar(P::B_Q_EMPTY));
          return true;
        });
        mma_commit(bar(P::B_DONE));
        mbar_wait_bounded(bar(P::B_DONE), 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * BN, to = tmem + lanes + P::T_O + t * D;
    const float sl2 = a.scale_log2;
    int done = 0;  // key tiles so far
    pieces([&](const Piece &p, int n, int tiles) {
      if (t >= tiles) return true;
      const int tok = row / a.G, j0 = p.tok0 + t * c.tpt + tok;
      const bool mine = tok < c.tpt && j0 < p.s.n;
      const int lim = mine ? min(p.k1, visible(p.s, j0)) : 0;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < n; ++j, ++done) {
        const int kb = p.k0 + j * BN;
        if (!__all_sync(0xffffffffu, mbar_wait(bar(P::B_S + t), done & 1, abort_flag))) {
          fail();
          return false;
        }
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, v[i]);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, kb + BN > lim)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kb + 32 * i + e >= lim) v[i][e] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mx[i] = __uint_as_float(v[i][0]);
#pragma unroll
          for (int e = 1; e + 1 < 32; e += 2)
            mx[i] = max3(mx[i], __uint_as_float(v[i][e]), __uint_as_float(v[i][e + 1]));
          mx[i] = fmaxf(mx[i], __uint_as_float(v[i][31]));
        }
        const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        const bool grow = m != -INFINITY && (top - m) * sl2 > 8.0f;
        if (__any_sync(0xffffffffu, grow)) {
          // the product of the tile before has to be in before O is scaled
          if (j > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(P::B_O + t), (done - 1) & 1, abort_flag))) {
            fail();
            return false;
          }
          tc_fence_after();
          const float f = grow ? ex2((m - top) * sl2) : 1.0f;
          l *= f;
          if (grow) m = top;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(to + 32 * i, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + 32 * i, o);
          }
          tmem_wait_st();
        }
        if (m == -INFINITY) m = top;
        const float neg = m == -INFINITY ? 0.0f : -m * sl2;
        float sum[4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x = __uint_as_float(v[2 * h + e / 32][e % 32]);
            float y = __uint_as_float(v[2 * h + e / 32][e % 32 + 1]);
            fma2(x, y, sl2, neg);
            x = ex2(x);
            y = ex2(y);
            add2(sum[(e & 2)], sum[(e & 2) + 1], x, y);
            w[e / 2] = pack2<DT>(x, y);
          }
          tmem_st32(ts + 32 * h, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(P::B_P + 2 * t + h));
        }
        l += (sum[0] + sum[2]) + (sum[1] + sum[3]);
      }
      // ---- the row's result
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(P::B_O + t), (done - 1) & 1, abort_flag))) {
          fail();
          return false;
        }
        tc_fence_after();
      }
      const bool none = l == 0.0f;
      const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (none ? 0.0f : l);
      const float lse = none ? -INFINITY : (m * sl2 + log2f(l)) * 0.6931471805599453f;
      const int64_t tg = p.s.t0 + j0, qh = int64_t(p.head) * a.G + (row - tok * a.G);
      if (mine) {
        if (a.o_part) {
          float *lp = a.lse_part + (tg * a.Hq + qh) * a.slots;
          lp[p.slot] = lse;
          for (int s = p.slot + 1; s < p.last; ++s) lp[s] = -INFINITY;
        } else if (a.lse) {
          a.lse[tg * a.Hq + qh] = lse;
        }
      }
      float *op = a.o_part ? a.o_part + ((tg * a.Hq + qh) * a.slots + p.slot) * a.dv : nullptr;
      uint16_t *o16 = a.out + tg * a.o_token + qh * a.o_head;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
        if (!mine) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (32 * i + e >= a.dv) continue;
          if (op) {
            if (none) continue;  // the join skips an empty part
            *reinterpret_cast<uint4 *>(op + 32 * i + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            *reinterpret_cast<uint4 *>(op + 32 * i + e + 4) =
                make_uint4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
          } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack2<DT>(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
            uint32_t *d = reinterpret_cast<uint32_t *>(o16 + 32 * i + e);
            if (c.out16) {
              *reinterpret_cast<uint4 *>(d) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) d[k] = w[k];
            }
          }
        }
      }
      tc_fence_before();  // O is read before the next piece's first product (through B_P)
      return true;
    });
  }
  __syncthreads();
  if (warp == WARP_MMA) tmem_dealloc(tmem, 512);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <class DT, int D>
int launch_one(const AttnArgs &a, Cut c, int64_t blocks, cudaStream_t st) {
  auto *k = attn_tile_kernel<DT, D>;
  static bool sized = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           Plan<D>::SMEM) == cudaSuccess;
  if (!sized) return WQ_ERR_LAUNCH;
  CUtensorMap mq, mk, mv;
  auto pitch = [](int64_t extent, int64_t stride) { return extent == 1 && stride == 0 ? 8 : stride; };
  const int64_t qd[3] = {a.dk, a.Hq, a.T};
  const int64_t qs[2] = {pitch(a.Hq, a.q_head), pitch(a.T, a.q_token)};
  const int qb[3] = {64, a.G, c.tpt};
  const int box[4] = {64, c.box, 1, 1};
  const int64_t kd[4] = {a.dk, a.page_size, a.Hkv, a.num_pages};
  const int64_t ks[3] = {pitch(a.page_size, a.k_token), pitch(a.Hkv, a.k_head), pitch(a.num_pages, a.k_page)};
  const int64_t vd[4] = {a.dv, a.page_size, a.Hkv, a.num_pages};
  const int64_t vs[3] = {pitch(a.page_size, a.v_token), pitch(a.Hkv, a.v_head), pitch(a.num_pages, a.v_page)};
  if (!make_tma_nd_b16_sw128(&mq, a.q, 3, qd, qs, qb) ||
      !make_tma_nd_b16_sw128(&mk, a.k, 4, kd, ks, box) ||
      !make_tma_nd_b16_sw128(&mv, a.v, 4, vd, vs, box))
    return WQ_ERR_UNSUPPORTED;
  k<<<unsigned(blocks), NTHREADS, Plan<D>::SMEM, st>>>(mq, mk, mv, a, c);
  return launched(1);
}

}  // namespace

int launch_attention_tiles(const AttnArgs &a, int dtype, cudaStream_t st) {
  Cut c{};
  c.tpt = BM / a.G;
  c.box = gcd(a.page_size, BN);
  c.out16 = a.o_token % 8 == 0 && a.o_head % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
  int64_t blocks = 0;
  if (a.tc_prefix) {
    c.pairs_p = (a.T + 2 * c.tpt - 1) / (2 * c.tpt);
    c.units_p = (a.P + BN - 1) / BN;
    c.blocks_p = a.p_blocks;
    blocks = c.blocks_p;
  }
  if (a.tc_suffix) {
    c.pairs_s = (a.max_q + 2 * c.tpt - 1) / (2 * c.tpt);
    blocks += int64_t(a.ss) * a.B * a.Hkv * c.pairs_s;
  }
  if (blocks == 0) return WQ_OK;
  if (blocks >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  const bool wide = a.dk > 64 || a.dv > 64;
  if (dtype == WQ_DT_BF16)
    return wide ? launch_one<Bf16, 128>(a, c, blocks, st) : launch_one<Bf16, 64>(a, c, blocks, st);
  return wide ? launch_one<F16, 128>(a, c, blocks, st) : launch_one<F16, 64>(a, c, blocks, st);
}

// Blocks that share the prefix's units, and the most blocks that meet in one
// item (its partial results)
void plan_prefix_tiles(AttnArgs &a) {
  const int tpt = BM / a.G;
  const int64_t items = int64_t(a.Hkv) * ((a.T + 2 * tpt - 1) / (2 * tpt));
  const int64_t units = (a.P + BN - 1) / BN, total = items * units;
  const int64_t sms = 152;
  // whole items where their waves are full to nine tenths, else equal pieces
  // of at least two units
  const int64_t waves = (items + sms - 1) / sms;
  int64_t blocks = items;
  if (items * 10 < waves * sms * 9) blocks = std::max<int64_t>(std::min(sms, total / 2), 1);
  a.p_blocks = int(blocks);
  a.sp = 1;
  if (blocks != items) {
    a.sp = 0;
    for (int64_t i = 0; i < items; ++i) {  // fewer than 152 * waves of them
      const int64_t f = ((i * units + 1) * blocks - 1) / total, l = ((i + 1) * units * blocks - 1) / total;
      a.sp = std::max(a.sp, int(l - f + 1));
    }
  }
}

}  // namespace wq
