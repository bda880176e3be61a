// Attention over a paged cache for many query rows (tcgen05, sm_103a): two
// tiles of 128 rows of one key head share every key and value tile.
//
//   S = Q K^T (128 x 128, float32 in tensor memory),  P = exp2(c S - c m),
//   O += P V,  l += row sums of P,  at the end O / l and its log-sum-exp.
//
// Rows are (token, query head of the group) pairs, so that every query head
// of a group uses the keys that are loaded once.  Two row tiles alternate on
// the tensor cores: while one tile's scores are exponentiated, the other's
// products run.  With heads of up to 64 a third score buffer lets the next
// scores be ready when a softmax ends.
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread owns one row
//   warps 8, 9      MMA issue, in turns; warp 8 owns the tensor memory
//   warp 10         TMA: queries, and keys and values page by page
//   warp 11         none (the third warpgroup gives its registers to the others)
// Tensor memory: two score buffers of 128 columns (three for D = 64), O0, O1
// (D each).  P takes the place of its S (64 columns, 16-bit pairs) as the A
// operand of the second product.  O is rescaled only when a row's maximum has
// grown by more than 2^8 over the one in use: until then the weights are at most
// 2^8, and the final division removes the factor.  P is rounded to 16 bits as the
// operand that it is; l sums the weights as they were.  A second sum, of the rounded ones, would
// divide the result better (error against 64 bits 0.0021 -> 0.0020 in bf16) but
// makes a call 17% longer at D = 64 (142 -> 166 us) and 5% at D = 128 (244 -> 257).
//
// The range is cut two ways.  The prefix is the same for all tokens.  A gang
// of blocks, one per row tile pair, walks the same keys at the same time, so
// that a tile of keys comes from HBM once and from L2 for the other members
// (blocks that walk apart read a prefix larger than L2 once each: 160 us of
// HBM time where 24 are needed, at 256 sequences behind 32768 keys of 8
// heads).  (key head, group of pairs) items times 128-key tiles form one line
// of equal units that the gangs cut into equal pieces: a piece may end inside
// an item and begin the next, and each leaves a partial result.  Suffixes: a
// block per (range, sequence, key head, row tile pair).
//
// Measured (bf16): a step of 256 rows x 128 keys takes 1.66 us at D = 128,
// 1.54 PFLOP/s over 152 SMs (0.79 of the measured cuBLAS burst), bound by the
// products and the hand-overs between the roles: without the exponentials it
// takes as long.  At D = 64 it takes 1.14 us (0.58 of burst), bound by the chain
// of loads, maximum, weights and stores of each softmax warp (without the
// exponentials 0.2 us less); with two score buffers it took 1.45 us.  An end of a
// range costs about 8 us (first loads 3, last product and results 4).
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
constexpr int WARP_MMA = 8, WARP_TMA = 10, WARP_IDLE = 11;  // MMA: two warps
// Registers a thread: 3 x 168 at launch (the most for 384 threads), shared out
// as 2 x 208 for the softmax, which holds a row of 128 scores, and 88
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 88;
static_assert(2 * REGS_SOFTMAX + REGS_OTHER <= 3 * 168, "a larger sum would wait forever");

template <int D>
struct Plan {
  static constexpr int CH = D / 64;              // 128-byte column chunks
  static constexpr int QB = BM * D * 2;          // bytes of one query tile
  static constexpr int KVB = BN * D * 2;         // bytes of a key or value tile
  static constexpr int NS = D == 128 ? 5 : 8;    // ring depth: keys and values in turn
  static constexpr int NB = D == 128 ? 2 : 3;    // score buffers in tensor memory
  // A wait by parity cannot tell a phase from the one two before it: whoever
  // waits has to know that all phases before are over.  Within a piece each
  // step's barrier (used in turn) is waited on by one row tile's warps alone,
  // which have seen every phase.  Between pieces, one of which may leave row
  // tile 1 without work, every softmax and product warp waits for the queries,
  // which come after all of the piece before, and takes part in their release.
  static constexpr int NSB = NB % 2 ? 2 * NB : NB;
  // Signals of a row tile's value products, two in turn.  Not all are waited on.
  // When the scores of key tile j are in, the products up to j - NB are over, so
  // the one of j - 1 may be waited for, and the one of j only after that.  (With
  // four in turn a piece's end needs one wait, but a step of heads of 64 takes
  // 1.22 us instead of 1.14.)
  static constexpr int NO = 2;
  static constexpr int Q_EMPTY_COUNT = 8 + 2;  // softmax and product warps
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = 2 * QB;
  static constexpr int OFF_BAR = OFF_KV + NS * KVB;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_Q_FULL = 2 * NS, B_Q_EMPTY = B_Q_FULL + 1,
                       B_S = B_Q_EMPTY + 1,      // [NSB] a step's scores are in
                       B_P = B_S + NSB,          // [NSB][2] half of its weights are in
                       B_O = B_P + 2 * NSB,      // [2][NO] a value product of a row tile is done
                       B_TAIL = B_O + 2 * NO,    // [2] in turn: a last value tile's tail is cleared
                       B_DONE = B_TAIL + 2, NBAR = B_DONE + 2;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static_assert(SMEM <= 232448, "shared memory plan too large");
  static constexpr uint32_t T_O = NB * BN;       // tensor-memory column of O0
  static_assert(NB * BN + 2 * D <= 512, "tensor memory plan");
  // keys NB tiles ahead of the values at hand, and those between
  static_assert(NS >= 2 * NB, "ring too shallow");
};

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
  int gang, gangs;    // row tile pairs that walk together; gangs on the prefix's line of units
  int groups;         // gangs' worths of pairs: ceil(pairs_p / gang)
  int stretch;        // units of a gang (the last may have fewer)
  int pairs_s;        // row tile pairs of a suffix (0: no suffixes here)
  int box;            // cache rows of one TMA box
  int step_pages, step_place;  // 128 keys on: pages, and places beyond them
  bool out16;         // out rows take 16-byte stores
};

// Whether every value product signals its end.  With as many score buffers as
// row tiles a tile's next scores are issued after it by the same thread and
// say so themselves; then only a result's last product signals.
template <int NB>
__device__ __forceinline__ bool signal_each(int tiles) {
  return NB > tiles;
}

// One piece of work: row tiles of a source against a key range
struct Piece {
  Source s;
  int head, tok0;     // key head; first token (of the source) of row tile 0
  int k0, k1;         // keys
  int slot, last;     // partial-result slot; slots (slot, last) stay empty
  bool open, close;   // the rows' sums begin, end with this piece
};

// units u0 .. u1 of one item, for member `member` of gang `gang`
__device__ __forceinline__ Piece prefix_piece(const AttnArgs &a, const Cut &c, int u0, int u1,
                                              int gang, int member) {
  const int item = u0 / c.units_p, start = item * c.units_p;
  Piece p;
  p.s = source_of(a, -1);
  p.head = item / c.groups;
  p.tok0 = ((item - p.head * c.groups) * c.gang + member) * 2 * c.tpt;
  p.k0 = (u0 - start) * BN;
  p.k1 = u1 - start >= c.units_p ? a.P : (u1 - start) * BN;
  p.slot = gang - start / c.stretch;  // ordinal of this gang among those that share the item
  p.last = p.k1 == a.P ? a.sp : p.slot + 1;
  p.open = p.close = true;
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
  p.open = p.close = true;
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

  attn::start_next_kernel();
  if (threadIdx.x == 0) {
    prefetch_map(&tmQ);
    prefetch_map(&tmK);
    prefetch_map(&tmV);
    *abort_flag = 0;
    for (int i = 0; i < P::NBAR; ++i)
      mbar_init(bar(i), i == P::B_Q_EMPTY                      ? P::Q_EMPTY_COUNT
                        : i >= P::B_P && i < P::B_O            ? 4   // warps of a row tile
                        : i >= P::B_EMPTY && i < P::B_Q_FULL   ? 2   // row tiles
                                                               : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  bool ok = true;  // this role's waits all ended in time

  // ---- this block's pieces, the same list for every role
  const int gang = int(blockIdx.x) / max(c.gang, 1), member = int(blockIdx.x) - gang * c.gang;
  const bool line = gang < c.gangs;
  const int u_begin = line ? gang * c.stretch : 0;
  const int u_end = line ? min(u_begin + c.stretch, a.Hkv * c.groups * c.units_p) : 1;
  // calls f(piece, key tiles, row tiles in use); stops when f returns false
  auto pieces = [&](auto &&f) {
    auto take = [&](const Piece &p) {
      const int n = p.k1 > p.k0 ? (p.k1 - p.k0 + BN - 1) / BN : 0;
      return f(p, n, p.tok0 + c.tpt < p.s.n ? 2 : 1);
    };
    for (int u = u_begin, part = 0; u < u_end;) {
      Piece p;
      if (line) {
        const int stop = min((u / c.units_p + 1) * c.units_p, u_end);
        p = prefix_piece(a, c, u, stop, gang, member);
        u = stop;
      } else {
        p = suffix_piece(a, c, int64_t(blockIdx.x) - int64_t(c.gang) * c.gangs);
        if (a.whole && a.P > 0) {  // the prefix, then the suffix, under the same sums
          p.open = part == 0;
          if (part == 0) {
            part = p.k1 > p.k0 ? 1 : 2;
            p.close = part == 2;
            p.s.pages = a.prefix_pages;
            p.s.len = p.k1 = a.P;
            p.s.causal = false;
          } else {
            part = 2;
          }
        }
        if (!a.whole || a.P == 0 || part == 2) u = u_end;
      }
      if (p.tok0 >= p.s.n) continue;  // a gang's last group, a short sequence
      if (!take(p)) return;
    }
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == WARP_TMA) {
      // ------------------------------------------------------------ copies
      int s = 0, g = 0, q = 0;  // ring stage; stages issued; pieces with keys
      uint32_t ph = 1;          // parity of the ring's releases
      int tails = 0;            // cleared tails
      bool bad = false;         // a page id outside the cache
      const int nbox = BN / c.box;
      const bool leader = elect_one();
      pieces([&](const Piece &p, int n, int tiles) {
        if (n == 0) return true;
        if (p.open && !(ok = wait_warp(bar(P::B_Q_EMPTY), (q & 1) ^ 1, abort_flag))) return false;
        if (leader && p.open) {
          mbar_expect_tx(bar(P::B_Q_FULL), uint32_t(tiles * P::CH * c.tpt * a.G * 128));
#pragma unroll 1
          for (int t = 0; t < tiles; ++t)
            for (int ch = 0; ch < P::CH; ++ch)
              tma_load_3d(base + P::OFF_Q + t * P::QB + ch * BM * 128, &tmQ, ch * 64, p.head * a.G,
                          p.s.t0 + p.tok0 + t * c.tpt, bar(P::B_Q_FULL));
        }
        q += p.open;
        // lane b looks up box b of a tile, one tile ahead of its copies; a bad
        // page is read outside the tensor: zeros
        const int key0 = p.k0 + lane * c.box;
        int pi = key0 / a.page_size, place = key0 - pi * a.page_size;
        int left = lane < nbox ? p.k1 - key0 : 0;  // keys from this lane's box on
        int page = left > 0 ? p.s.pages[pi] : 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          int y = place, w = page;
          if (left > 0 && unsigned(w) >= unsigned(a.num_pages)) {
            w = int(a.num_pages);
            bad = true;
          }
          const int boxes = __popc(__ballot_sync(0xffffffffu, left > 0));  // with a key in range
          pi += c.step_pages;
          place += c.step_place;
          if (place >= a.page_size) place -= a.page_size, ++pi;
          left -= BN;
          if (left > 0) page = p.s.pages[pi];
          auto stage = [&](const CUtensorMap *map) {
            ok = wait_warp(bar(P::B_EMPTY + s), ph, abort_flag);
            if (!ok) return false;
            const uint32_t full = bar(P::B_FULL + s);
            uint32_t dst = base + P::OFF_KV + uint32_t(s * P::KVB);
            if (leader) mbar_expect_tx(full, uint32_t(boxes * c.box * P::CH * 128));
#pragma unroll 1
            for (int b = 0; b < boxes; ++b) {
              const int by = __shfl_sync(0xffffffffu, y, b), bw = __shfl_sync(0xffffffffu, w, b);
              if (leader) {
#pragma unroll
                for (int ch = 0; ch < P::CH; ++ch)
                  tma_load_4d(dst + ch * BN * 128, map, ch * 64, by, p.head, bw, full);
              }
              dst += uint32_t(c.box * 128);
            }
            if (++s == P::NS) s = 0, ph ^= 1;
            ++g;
            return true;
          };
          if (!stage(&tmK) || !stage(&tmV)) return false;
        }
        const int r0 = (p.k1 - p.k0) % BN;
        if (r0) {
          // clear the values past the range, once the last copies are in
          const int sv = (g - 1) % P::NS;
          if (!(ok = wait_warp(bar(P::B_FULL + sv), ((g - 1) / P::NS) & 1, abort_flag))) return false;
          uint8_t *v = sm + P::OFF_KV + sv * P::KVB;
#pragma unroll 1
          for (int i = lane; i < (BN - r0) * 8 * P::CH; i += 32) {
            const int row = i / (8 * P::CH), ch = i % (8 * P::CH);
            *reinterpret_cast<uint4 *>(v + ((ch / 8) * BN + r0 + row) * 128 + (ch % 8) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
          __syncwarp();
          // Two barriers in turn: the prefix's tail and the suffix's may both be
          // ahead of the products, and a barrier holds one phase
          if (lane == 0) mbar_arrive(bar(P::B_TAIL + (tails & 1)));
          ++tails;
        }
        return true;
      });
      if (bad) set_status(a.status, WQ_ERR_INDEX);
      if (!ok) {  // let copies already in flight land before the block goes away
        *abort_flag = 1;
        if (q > 0) mbar_wait_bounded(bar(P::B_Q_FULL), (q - 1) & 1);
        for (int i = g > P::NS ? g - P::NS : 0; i < g; ++i)
          mbar_wait_bounded(bar(P::B_FULL + i % P::NS), (i / P::NS) & 1);
      }
    } else if (warp != WARP_IDLE) {
      // ------------------------------------------------------------ products
      // A piece's steps k = (key tile, row tile) use the score buffers in turn:
      // QK(k) fills one, its weights take its place, PV(k) empties it, and
      // QK(k + NB) fills it again.  A step here is PV(k), then QK(k + NB), from
      // k = -NB on.  With two row tiles two warps take alternate steps (a wait
      // takes over 100 cycles even when there is nothing to wait for, and one
      // warp's waits pass in the other's step); with one, one warp takes all.
      // With two buffers the two warps take turns, which keeps the row tiles
      // half a step apart: warp 0 begins a piece and warp 1 ends it, so that a
      // turn is never given twice, and after a wait that ran out a warp still
      // takes its turns, so that the other ends.
      const int t = warp - WARP_MMA;
      const bool leader = elect_one();
      constexpr uint32_t id_s = idesc_f16(BM, BN) | kTypes<DT>;
      constexpr uint32_t id_o = idesc_f16(BM, D) | kTypes<DT> | kBTransposed;
      constexpr int NB = P::NB;
      uint32_t g = 0, kk = 0;    // ring stages and steps of the pieces before
      int q = 0, tails = 0;      // pieces; cleared tails
      uint32_t ends0 = 0, ends1 = 0;  // signals on each row tile's products so far
      auto wait = [&](int b, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, wait_one(bar(b), parity, abort_flag));
        if (!ok) *abort_flag = 1;
      };
      // both row tiles release a stage; where there is one, it counts twice
      auto release = [&](uint32_t stage, int tiles) {
        mma_commit(bar(P::B_EMPTY + stage));
        if (tiles == 1) mbar_arrive(bar(P::B_EMPTY + stage));
      };
      pieces([&](const Piece &p, int n, int tiles) {
        if (n == 0) return true;
        const bool tail = (p.k1 - p.k0) % BN != 0, two = tiles == 2;
        const int steps = n * tiles;
        const bool each = signal_each<NB>(tiles);
        const bool turns = NB == 2 && two;
        auto pass = [&]() { asm volatile("bar.arrive %0, 64;" ::"r"(2 - t) : "memory"); };
        if (turns && t == 1) pass();
        if (p.open) {  // by both warps, even where one has no rows
          wait(P::B_Q_FULL, q & 1);
          if (ok && lane == 0) mbar_arrive(bar(P::B_Q_EMPTY));
        }
        q += p.open;
        if (turns) {
          // The common case written out: warp t keeps to row tile t and one
          // buffer, and what a step needs is counted on by one.  (Through the
          // general loop below a step of 256 rows x 128 keys takes 1.71 us
          // instead of 1.67: these warps are bound by what they issue.)
          const uint32_t buf = (kk + uint32_t(t)) & 1, ts = tmem + buf * BN, to = tmem + P::T_O + t * D;
          const uint64_t dq = sdesc(base + P::OFF_Q + t * P::QB);
          uint32_t s = g % P::NS, ph = (g / P::NS) & 1, pp = ((kk + uint32_t(t)) >> 1) & 1;
          auto next = [&]() {
            if (++s == P::NS) s = 0, ph ^= 1;
          };
          auto scores = [&](uint32_t stage) {
            const uint64_t dk = sdesc(base + P::OFF_KV + stage * P::KVB);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t at = ((i / 4) * (BM * 128) + (i % 4) * 32) >> 4;
              mma_f16(ts, dq + at, dk + at, id_s, i ? 1u : 0u);
            }
            mma_commit(bar(P::B_S + buf));
          };
          wait(P::B_FULL + s, ph);
          named_sync(1 + t, 64);
          tc_fence_after();
          if (leader && ok) {
            scores(s);
            release(s, 2);
          }
          pass();
          next();
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const uint32_t sv = s;
            const bool more = j + 1 < n;
            wait(P::B_FULL + sv, ph);
            next();
            if (more) wait(P::B_FULL + s, ph);
            else if (tail) wait(P::B_TAIL + (tails & 1), (tails >> 1) & 1);
            const uint64_t dv = sdesc_n(base + P::OFF_KV + sv * P::KVB);
            wait(P::B_P + 2 * buf, pp);
            named_sync(1 + t, 64);
            tc_fence_after();
            if (leader && ok) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_f16_ts(to, ts + 8 * i, dv + ((2048 * i) >> 4), id_o, j | i || !p.open ? 1u : 0u);
            }
            wait(P::B_P + 2 * buf + 1, pp);
            pp ^= 1;
            tc_fence_after();
            if (leader && ok) {
#pragma unroll
              for (int i = 4; i < 8; ++i) mma_f16_ts(to, ts + 8 * i, dv + ((2048 * i) >> 4), id_o, 1u);
              if (more) scores(s);
              else if (p.close) mma_commit(bar(P::B_O + P::NO * t + ((t ? ends1 : ends0) % P::NO)));
            }
            if (t == 0 || more) pass();  // the last turn is nobody's to wait for
            if (leader && ok) {
              release(sv, 2);
              if (more) release(s, 2);
            }
            if (more) next();
          }
        } else {
          int k = two ? -NB + ((t - NB) & 1) : t == 0 ? -NB : steps;
          // Where step k is: ring stage and parity of PV(k)'s values and of
          // QK(k + NB)'s keys (two stages on from step to step), barrier and
          // parity of its weights, barrier of those scores, and their buffer.
          // Counted on, since the divisions stand in the way of the issue.
          const int j0 = two ? k >> 1 : k, jn0 = two ? (k + NB) >> 1 : k + NB;
          const uint32_t v0 = g + uint32_t(2 * j0 + 1 + 2 * P::NS), c0 = g + uint32_t(2 * jn0);
          const uint32_t p0 = kk + uint32_t(k + 2 * P::NSB), s0 = kk + uint32_t(k + NB);
          uint32_t sv = v0 % P::NS, pv = (v0 / P::NS) & 1, sk = c0 % P::NS, pk = (c0 / P::NS) & 1;
          uint32_t pb = p0 % P::NSB, pp = (p0 / P::NSB) & 1, sb = s0 % P::NSB, buf = s0 % NB;
          const int o = two ? t : 0, on = two ? (t + NB) & 1 : 0;  // row tiles of PV(k), of QK(k + NB)
          const uint32_t to = tmem + P::T_O + o * D;
          const uint64_t dq = sdesc(base + P::OFF_Q + on * P::QB);
          auto on_by = [](uint32_t &x, uint32_t by, uint32_t of) {
            x += by;
            const bool wrap = x >= of;
            x -= wrap ? of : 0;
            return uint32_t(wrap);
          };
#pragma unroll 1
          for (int j = j0; k < steps; k += tiles, ++j) {
            const bool more = k + NB < steps;
            // operands and barriers, ready ahead of the waits
            uint32_t ts = tmem + buf * BN, acc = j > 0 || !p.open;
            uint32_t bar_o = bar(P::B_O + P::NO * o) + 8 * (((o ? ends1 : ends0) + (each ? uint32_t(j) : 0u)) % P::NO);
            uint32_t bar_s = bar(P::B_S + sb);
            const bool signal = each || (j + 1 == n && p.close);
            uint64_t dv = sdesc_n(base + P::OFF_KV + sv * P::KVB), dk = sdesc(base + P::OFF_KV + sk * P::KVB);
            asm volatile("" : "+r"(ts), "+r"(acc), "+r"(bar_o), "+r"(bar_s), "+l"(dv), "+l"(dk));
            if (k >= 0) {
              wait(P::B_FULL + sv, pv);
              if (tail && j + 1 == n) wait(P::B_TAIL + (tails & 1), (tails >> 1) & 1);
            }
            if (more) wait(P::B_FULL + sk, pk);
            if (k >= 0) wait(P::B_P + 2 * pb, pp);
            tc_fence_after();
            auto scores = [&]() {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t at = ((i / 4) * (BM * 128) + (i % 4) * 32) >> 4;
                mma_f16(ts, dq + at, dk + at, id_s, i ? 1u : 0u);
              }
              mma_commit(bar_s);
            };
            if (k >= 0) {
              if (leader && ok) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mma_f16_ts(to, ts + 8 * i, dv + ((2048 * i) >> 4), id_o, i ? 1u : acc);
              }
              wait(P::B_P + 2 * pb + 1, pp);
              tc_fence_after();
              if (leader && ok) {
#pragma unroll
                for (int i = 4; i < 8; ++i) mma_f16_ts(to, ts + 8 * i, dv + ((2048 * i) >> 4), id_o, 1u);
                if (signal) mma_commit(bar_o);
                if (more) scores();
              }
            } else if (more && leader && ok) {
              scores();
            }
            if (leader && ok) {
              if (k >= 0) release(sv, tiles);
              if (more) release(sk, tiles);
            }
            pv ^= on_by(sv, 2, P::NS);
            pk ^= on_by(sk, 2, P::NS);
            pp ^= on_by(pb, uint32_t(tiles), P::NSB);
            on_by(sb, uint32_t(tiles), P::NSB);
            on_by(buf, uint32_t(tiles), NB);
          }
        }
        g += 2 * uint32_t(n);
        kk += uint32_t(steps);
        const uint32_t signals = each ? uint32_t(n) : uint32_t(p.close);
        ends0 += signals;
        if (two) ends1 += signals;
        tails += tail;
        return true;  // through all pieces, turns and all
      });
      if (leader) mma_commit(bar(P::B_DONE + t));
      mbar_wait_bounded(bar(P::B_DONE + t), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + P::T_O + t * D;
    const float sl2 = a.scale_log2;
    uint32_t kk = 0;    // steps of the pieces before (both row tiles)
    uint32_t ends = 0;  // signals on this row tile's products so far
    int q = 0;          // pieces with keys so far
    float m = -INFINITY, l = 0.0f;
    // A weight is exp2(s * c - m * c) in one fused operation whose second term is
    // rounded first.  Where that would show (m * c past 2^16: 2^-8 there, and far
    // past it the largest weight would be any power of two), the warp subtracts
    // m from the scores before it scales them.
    constexpr float kFar = 65536.0f;
    bool far = false;
    pieces([&](const Piece &p, int n, int tiles) {
      // the queries of a piece are released at its end: their tiles serve as
      // staging for its results
      auto release = [&]() {
        if (n == 0) return;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(P::B_Q_EMPTY));
      };
      if (n > 0 && p.open) {
        if (!(ok = wait_warp(bar(P::B_Q_FULL), q & 1, abort_flag))) return false;
        ++q;
      }
      const bool each = signal_each<P::NB>(tiles);
      uint32_t k = kk + uint32_t(t);
      kk += uint32_t(n * tiles);
      if (t >= tiles) {
        if (p.close) release();
        return true;
      }
      const int tok = row / a.G, j0 = p.tok0 + t * c.tpt + tok;
      const bool mine = tok < c.tpt && j0 < p.s.n;
      const int lim = mine ? min(p.k1, visible(p.s, j0)) : 0;
      if (p.open) {
        m = -INFINITY;
        l = 0.0f;
        far = false;
      }
      for (int j = 0; j < n; ++j, k += uint32_t(tiles)) {
        const int kb = p.k0 + j * BN;
        const uint32_t buf = k % P::NB, ts = tmem + lanes + buf * BN;
        const uint32_t step = k % P::NSB;
        if (!(ok = wait_warp(bar(P::B_S + step), (k / P::NSB) & 1, abort_flag))) return false;
        tc_fence_after();
        uint32_t v[4][32];
        // 64 weights under the maximum in use, two to a word
        uint32_t w[32];
        float sum[4], top = -INFINITY;
        auto weigh = [&](int h, float neg) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = 0.0f;
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float x = __uint_as_float(v[2 * h + e / 32][e % 32]);
            float y = __uint_as_float(v[2 * h + e / 32][e % 32 + 1]);
            fma2(x, y, sl2, neg);
            x = ex2(x);
            y = ex2(y);
            add2(sum[e & 2], sum[(e & 2) + 1], x, y);
            w[e / 2] = pack2<DT>(x, y);
          }
        };
        auto top_of = [&](int i) {
          float m0 = __uint_as_float(v[i][0]), m1 = __uint_as_float(v[i][1]);
#pragma unroll
          for (int e = 2; e < 30; e += 4) {
            m0 = max3(m0, __uint_as_float(v[i][e]), __uint_as_float(v[i][e + 1]));
            m1 = max3(m1, __uint_as_float(v[i][e + 2]), __uint_as_float(v[i][e + 3]));
          }
          top = max3(top, max3(m0, __uint_as_float(v[i][30]), __uint_as_float(v[i][31])), m1);
        };
        auto hand_over = [&](int h) {
          tmem_st32(ts + 32 * h, w);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(P::B_P + 2 * step + h));
          l += (sum[0] + sum[2]) + (sum[1] + sum[3]);
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, v[i]);
        wait_ld32(v[0]);
        pin32(v[1]);
        pin32(v[2]);
        pin32(v[3]);
        if (__any_sync(0xffffffffu, kb + BN > lim)) {  // keys out of this row's sight
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (kb + 32 * i + e >= lim) v[i][e] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top_of(i);
        const bool grow = top > m && !((top - m) * sl2 <= 8.0f);
        if (__any_sync(0xffffffffu, grow || far)) {
          const float f = grow && m != -INFINITY ? ex2((m - top) * sl2) : 1.0f;
          if (grow) m = top;
          l *= f;
          if ((j > 0 || !p.open) && __any_sync(0xffffffffu, f != 1.0f)) {
            // the value product of the tile before has to be in
            if (each) {
              const uint32_t end = ends + uint32_t(j) - 1;
              if (!(ok = wait_warp(bar(P::B_O + P::NO * t + end % P::NO), (end / P::NO) & 1, abort_flag))) return false;
              tc_fence_after();
            }
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t o[16];
              tmem_ld16(to + 16 * i, o);
              asm volatile("tcgen05.wait::ld.sync.aligned;"
                           : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]),
                             "+r"(o[6]), "+r"(o[7]), "+r"(o[8]), "+r"(o[9]), "+r"(o[10]), "+r"(o[11]),
                             "+r"(o[12]), "+r"(o[13]), "+r"(o[14]), "+r"(o[15])
                           :
                           : "memory");
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(to + 16 * i, o);
            }
          }
          const float at = m == -INFINITY ? 0.0f : m;
          far = __any_sync(0xffffffffu, fabsf(at) * sl2 > kFar);
          if (far) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 32; ++e) v[i][e] = __float_as_uint(__uint_as_float(v[i][e]) - at);
          }
        }
        const float neg = far || m == -INFINITY ? kWeightUp<DT> : __fmaf_rn(-m, sl2, kWeightUp<DT>);
        weigh(0, neg);
        hand_over(0);
        weigh(1, neg);
        hand_over(1);
      }
      if (!p.close) {
        if (each) ends += uint32_t(n);
        return true;
      }
      // ---- the row's result
      if (n > 0) {
        const uint32_t end = each ? ends + uint32_t(n) - 1 : ends;
        ends = end + 1;
        if (each && (n > 1 || !p.open) &&
            !(ok = wait_warp(bar(P::B_O + P::NO * t + (end - 1) % P::NO), ((end - 1) / P::NO) & 1, abort_flag)))
          return false;
        if (!(ok = wait_warp(bar(P::B_O + P::NO * t + end % P::NO), (end / P::NO) & 1, abort_flag))) return false;
        tc_fence_after();
      }
      const bool none = l == 0.0f;
      const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (none ? 0.0f : l);
      const float lse = lse_of<DT>(m, sl2, l);
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
      // Rows leave through this warp's quarter of its query tile (all products
      // with it are done), so that a store covers whole rows: 16-byte pieces,
      // swizzled, NC a row.  16-bit results go in one pass, float parts in two.
      // With 152 blocks the float parts (128 KB each) take about 3.7 us to L2,
      // all at the same time; 16-bit results a quarter of that.
      constexpr int NC = D / 8, RPI = 32 / NC;  // pieces of a staged row; rows a store covers
      uint8_t *stage = sm + P::OFF_Q + t * P::QB + (warp & 3) * 32 * (D * 2);
      const int64_t off = a.o_part ? ((tg * a.Hq + qh) * a.slots + p.slot) * a.dv
                                   : tg * a.o_token + qh * a.o_head;
      const uint32_t live = __ballot_sync(0xffffffffu, mine && !(a.o_part && none));
#pragma unroll 1
      for (int pass = 0; pass < (a.o_part ? 2 : 1); ++pass) {
        const int cols = a.o_part ? D / 2 : D;  // columns of this pass
#pragma unroll 1
        for (int i = 0; i < cols / 32; ++i) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(to + pass * (D / 2) + 32 * i, o);
            wait_ld32(o);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = none ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
          if (a.o_part) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4 *>(stage + (lane * NC + ((8 * i + e) ^ (lane & (NC - 1)))) * 16) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack2<DT>(__uint_as_float(o[8 * e + 2 * k]), __uint_as_float(o[8 * e + 2 * k + 1]));
              *reinterpret_cast<uint4 *>(stage + (lane * NC + ((4 * i + e) ^ (lane & (NC - 1)))) * 16) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        __syncwarp();
        const int ch = lane % NC;
#pragma unroll 2
        for (int r0 = 0; r0 < 32; r0 += RPI) {
          const int r = r0 + lane / NC;
          const int64_t at = __shfl_sync(0xffffffffu, off, r);
          if (!((live >> r) & 1u)) continue;
          const uint4 x = *reinterpret_cast<const uint4 *>(stage + (r * NC + (ch ^ (r & (NC - 1)))) * 16);
          if (a.o_part) {
            const int d = pass * (D / 2) + ch * 4;
            if (d < a.dv) *reinterpret_cast<uint4 *>(a.o_part + at + d) = x;
          } else if (ch * 8 < a.dv) {
            uint32_t *d = reinterpret_cast<uint32_t *>(a.out + at + ch * 8);
            if (c.out16) {
              *reinterpret_cast<uint4 *>(d) = x;
            } else {
              d[0] = x.x;
              d[1] = x.y;
              d[2] = x.z;
              d[3] = x.w;
            }
          }
        }
        __syncwarp();
      }
      release();
      tc_fence_before();  // O is read before the next piece's first product (through B_P)
      return true;
    });
  }
  if (!ok) {
    *abort_flag = 1;
    set_status(a.status, WQ_ERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == WARP_MMA) tmem_dealloc(tmem, 512);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <class DT, int D>
int launch_one(const AttnArgs &a, Cut c, int64_t blocks, cudaStream_t st) {
  auto *k = attn_tile_kernel<DT, D>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, Plan<D>::SMEM)) return WQ_ERR_LAUNCH;
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
  c.step_pages = BN / a.page_size;
  c.step_place = BN % a.page_size;
  c.out16 = a.o_token % 8 == 0 && a.o_head % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
  int64_t blocks = 0;
  if (a.tc_prefix) {
    c.pairs_p = (a.T + 2 * c.tpt - 1) / (2 * c.tpt);
    c.units_p = (a.P + BN - 1) / BN;
    c.gang = a.p_gang;
    c.gangs = a.p_gangs;
    c.groups = (c.pairs_p + c.gang - 1) / c.gang;
    c.stretch = a.p_stretch;
    blocks = int64_t(c.gang) * c.gangs;
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

// Gangs of the prefix, and the most of them that meet in one item (its partial
// results), on `sms` SMs.  The gang size is the one that leaves the fewest of them
// without rows; whole items per gang where their waves are full to nine
// tenths, else equal pieces of at least two units.
bool plan_prefix_tiles(AttnArgs &a, int sms) {
  const int tpt = BM / a.G;
  const int64_t pairs = (a.T + 2 * tpt - 1) / (2 * tpt), units = (a.P + BN - 1) / BN;
  double best = 0.0;
  for (int64_t g = std::min<int64_t>({pairs, 19, sms}); g >= 1; --g) {
    const int64_t groups = (pairs + g - 1) / g;
    const double use = double(sms / g * g) / sms * double(pairs) / double(groups * g);
    if (use > best + 0.02) best = use, a.p_gang = int(g);
  }
  const int64_t items = (pairs + a.p_gang - 1) / a.p_gang * a.Hkv, total = items * units;
  if (total >= (int64_t(1) << 31)) return false;
  const int64_t most = sms / a.p_gang, waves = (items + most - 1) / most;
  int64_t stretch = units;
  if (items * 10 < waves * most * 9) stretch = std::max<int64_t>((total + most - 1) / most, 2);
  a.p_stretch = int(stretch);
  a.p_gangs = int((total + stretch - 1) / stretch);
  a.sp = 1;
  for (int64_t i = 0; stretch != units && i < items; ++i)  // fewer than sms * waves of them
    a.sp = std::max(a.sp, int(((i + 1) * units - 1) / stretch - i * units / stretch + 1));
  return true;
}

}  // namespace wq
