// Attention over a paged cache for a batch that shares a prefix: the kernel
// for few query rows, the join of partial results, and the plan.
//
// Rows of a key head are (query token, query head of its group) pairs.  A
// work item is a tile of up to 16 or 32 rows of one source (the shared prefix,
// or one sequence's suffix) against one range of its keys.  Ranges are cut so
// that few rows still fill the machine; each item leaves a normalised partial
// result and its log-sum-exp, and a last kernel joins a row's partials:
//   m = max_s lse_s,  out = sum_s exp(lse_s - m) o_s / sum_s exp(lse_s - m).
//
// Few rows are bound by the reading of keys and values.  A warp takes 16-key
// pieces of a range; it keeps its own running maximum, sum and output (the
// softmax of its keys) in registers and its own ring of asynchronous copies,
// so warps never wait for one another inside a range.  With many (sequence,
// key head) pairs a block is one warp and nine blocks share an SM: their
// starts and ends overlap.  With few, four warps take a range's pieces in turn
// and add up their results at its end.  Warp matrix products (16 x 8 x 16) do the arithmetic: with 16
// rows they need 1/5 of their rate to keep up with HBM, and unlike the tensor
// memory path they need no 128-row tile.  Measured (bf16): 64 sequences of up
// to 8192 keys, 8 key heads of 128, no prefix, 196 us, 6.2 TB/s of keys and
// values.
#include <algorithm>
#include <type_traits>

#include "wq_attn.cuh"

namespace wq {
namespace {

using namespace attn;

constexpr int KT = 16;   // keys of a piece

constexpr int NST = 3;   // pieces a warp has in flight

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <class DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<DT, Bf16>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// over the four lanes that share a row
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
template <class DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<DT, Bf16>::value) return pack_bf16x2(lo, hi);
  else return f16x2_rn(lo, hi);
}

// Rows before cu_q[0], at or past cu_q[B] (a batch padded for a recorded
// graph) and past max_q in their sequence are tokens of no sequence and see no
// key: zeros and -inf.  The work on the suffixes writes that or, where there
// are parts to join, marks the rows for the join by a log-sum-exp that no part
// has, since the work on the prefix covers all rows.  (Looking each row's
// sequence up there instead cost the tile kernel 2.5 us a piece.)
constexpr float kNoSequence = INFINITY;

// For one head: rows r0, r0 + by, ... below r1, a warp for each row's query heads in turn
__device__ __forceinline__ void clear_rows(const AttnArgs &a, int head, int r0, int r1, int by) {
  if (r0 >= r1) return;
  const int lane = threadIdx.x & 31, n = ((r1 - r0 - 1) / by + 1) * a.G;
  for (int i = threadIdx.x >> 5; i < n; i += blockDim.x >> 5) {
    const int j = i / a.G, qh = head * a.G + i - j * a.G;
    const int64_t t = r0 + int64_t(j) * by, row = t * a.Hq + qh;
    if (a.o_part && a.max_suffix > 0) {
      if (lane == 0) a.lse_part[(row + 1) * a.slots - 1] = kNoSequence;
    } else {
      uint32_t *o = reinterpret_cast<uint32_t *>(a.out + t * a.o_token + qh * a.o_head);
      for (int d = lane; d < a.dv / 2; d += 32) o[d] = 0u;
      if (lane == 0 && a.lse) a.lse[row] = -INFINITY;
    }
  }
}
// `parts` blocks of each (sequence, head) share the rows past max_q in the
// sequence and a B-th of those outside [cu_q[0], cu_q[B]).
__device__ __forceinline__ void clear_rest(const AttnArgs &a, int seq, const Source &s, int head,
                                           int part, int parts) {
  const int begin = a.cu_q[0], end = max(a.cu_q[a.B], 0), next = a.cu_q[seq + 1];
  const int own = seq * parts + part, all = a.B * parts;
  clear_rows(a, head, s.t0 + s.n + part, min(next, a.T), parts);
  if (begin > 0) clear_rows(a, head, own, min(begin, a.T), all);
  if (end < a.T) clear_rows(a, head, end + own, a.T, all);
}

// D: padded head size (64 or 128), MT: 16-row tiles
template <class DT, int D, int MT, int NW>
struct Small {
  static constexpr int CH = D / 8;                 // 16-byte pieces of a row
  static constexpr int KB = KT * D * 2;            // bytes of 16 keys (or values)
  static constexpr int STAGE = 2 * KB;
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int JOIN = NW == 1 ? 0 : NW * MT * 16 * (D + 4) * 4;  // per-warp results, row pitch D + 4
  static constexpr int SMEM = RING > JOIN ? RING : JOIN;
};

template <class DT, int D, int MT, int NW, bool PAGED>
__global__ void __launch_bounds__(NW * 32) attn_small_kernel(const AttnArgs a, int prefix_items,
                                                             int prefix_tiles, int suffix_tiles) {
  using P = Small<DT, D, MT, NW>;
  constexpr int CH = P::CH, R = 16 * MT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = NW == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  start_next_kernel();

  // ---- the work item: (range, sequence, key head, row tile), row tile innermost
  int64_t it = blockIdx.x;
  int seq = -1, head, tile, split, chunk;
  if (it < prefix_items) {
    tile = int(it % prefix_tiles);
    it /= prefix_tiles;
    head = int(it % a.Hkv);
    split = int(it / a.Hkv);
    chunk = a.p_chunk;
  } else {
    it -= prefix_items;
    tile = int(it % suffix_tiles);
    it /= suffix_tiles;
    head = int(it % a.Hkv);
    it /= a.Hkv;
    seq = int(it % a.B);
    split = int(it / a.B);
    chunk = a.s_chunk;
  }
  const Source s = source_of(a, seq);
  const bool rest = seq >= 0 && a.cu_q && !a.rest_apart && tile == 0 && split == 0;
  const int rows = min(R, s.n * a.G - tile * R);  // rows of this tile
  const bool last_block = blockIdx.x == gridDim.x - 1;
  if (rows <= 0) {
    if (rest) clear_rest(a, seq, s, head, 0, 1);
    if (last_block) wait_last_kernel();
    return;
  }
  const int row0 = tile * R;
  const int k0 = split * chunk;
  // keys that the tile's last token sees, and this range's end
  const int k1 = min(min(s.len, visible(s, (row0 + rows - 1) / a.G)), k0 + chunk);
  const int slot = s.slot0 + split;

  // ---- this thread's rows in every 16-row tile: lane / 4 and + 8
  int lim[MT][2];  // keys each row sees
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + lane / 4;
      lim[m][h] = r < rows ? min(k1, visible(s, (row0 + r) / a.G)) : 0;
    }

  // ---- queries as A fragments, straight from memory
  uint32_t qf[MT][D / 16][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + lane / 4;
      const uint16_t *qp = nullptr;
      if (r < rows) {
        const int j = (row0 + r) / a.G, g = (row0 + r) - j * a.G;
        qp = a.q + int64_t(s.t0 + j) * a.q_token + int64_t(head * a.G + g) * a.q_head;
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int d = k * 16 + c * 8 + (lane & 3) * 2;
          qf[m][k][c * 2 + h] =
              (qp && d < a.dk) ? *reinterpret_cast<const uint32_t *>(qp + d) : 0u;
        }
    }

  // ---- this warp's ring: pieces warp, warp + NW, ... of the range
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                        uint32_t(warp * NST * P::STAGE);
  const int pieces = k1 > k0 ? (k1 - k0 + KT - 1) / KT : 0;
  const int mine = pieces > warp ? (pieces - warp + NW - 1) / NW : 0;

  // The piece that is asked for next: its page is looked up one piece ahead of
  // its copies.  PAGED: pages hold whole pieces, so that a piece has one page
  // and its keys one pitch; else lane (mod 16) r looks up key r.
  const int own = PAGED ? 0 : lane & 15;
  int key = k0 + warp * KT + own;
  int pi = key / a.page_size, place = key - pi * a.page_size;
  int page = mine > 0 && key < k1 ? s.pages[pi] : 0;
  bool bad = false;
  const int lr = lane / CH, lc = lane % CH;  // this lane's row and 16-byte column of a copy
  const uint16_t *kh = a.k + int64_t(head) * a.k_head + (lc * 8 < a.dk ? lc * 8 : 0);
  const uint16_t *vh = a.v + int64_t(head) * a.v_head + (lc * 8 < a.dv ? lc * 8 : 0);
  if constexpr (PAGED) {
    kh += lr * a.k_token;
    vh += lr * a.v_token;
  }
  const uint32_t ldst = ring + uint32_t(lr * CH + (lc ^ lr)) * 16;
  // starts the copies of piece i; returns bit r for key r that is there
  auto issue = [&](int i) -> uint32_t {
    uint32_t on = 0;
    if (i < mine) {
      constexpr int RPC = 32 / CH;  // rows of a copy
      bool there = key < k1;
      if (there && unsigned(page) >= unsigned(a.num_pages)) {
        there = false;
        bad = true;
      }
      const int64_t pg = there ? page : 0;
      const uint32_t d = ldst + uint32_t((i % NST) * P::STAGE);
      if constexpr (PAGED) {
        const int n = there ? min(KT, k1 - key) : 0;
        on = (1u << n) - 1;
        const uint16_t *kp = kh + pg * a.k_page + int64_t(place) * a.k_token;
        const uint16_t *vp = vh + pg * a.v_page + int64_t(place) * a.v_token;
#pragma unroll
        for (int j = 0; j < KT / RPC; ++j) {
          const uint32_t dj = (d ^ uint32_t((j * RPC & 7) << 4)) + uint32_t(j * RPC * CH * 16);
          cp16(dj, kp + int64_t(j * RPC) * a.k_token, j * RPC + lr < n && lc * 8 < a.dk);
          cp16(dj + P::KB, vp + int64_t(j * RPC) * a.v_token, j * RPC + lr < n && lc * 8 < a.dv);
        }
      } else {
        on = __ballot_sync(0xffffffffu, there) & 0xffffu;
        const int64_t ko = pg * a.k_page + int64_t(place) * a.k_token;
        const int64_t vo = pg * a.v_page + int64_t(place) * a.v_token;
#pragma unroll
        for (int j = 0; j < KT / RPC; ++j) {
          const int r = j * RPC + lr;
          const uint32_t dj = (d ^ uint32_t((j * RPC & 7) << 4)) + uint32_t(j * RPC * CH * 16);
          cp16(dj, kh + __shfl_sync(0xffffffffu, ko, r), (on >> r & 1u) && lc * 8 < a.dk);
          cp16(dj + P::KB, vh + __shfl_sync(0xffffffffu, vo, r), (on >> r & 1u) && lc * 8 < a.dv);
        }
      }
      key += NW * KT;
      pi += a.step_pages;
      place += a.step_place;
      if (place >= a.page_size) place -= a.page_size, ++pi;
      if (key < k1) page = s.pages[pi];
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return on;
  };

  // maximum; sum of the weights, for the log-sum-exp, and of the rounded ones
  // that multiply the values, which divides the result: what the weights of a
  // few large keys lose to the rounding cancels (error against 64 bits in bf16
  // 0.0021 -> 0.0018; 194 -> 196.5 us with 64 sequences of up to 8192 keys)
  float m_[MT][2], l_[MT][2], u_[MT][2], o[MT][D / 8][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    m_[m][0] = m_[m][1] = -INFINITY;
    l_[m][0] = l_[m][1] = u_[m][0] = u_[m][1] = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
  }
  int least = lim[0][0];  // every row of the warp sees the keys below
#pragma unroll
  for (int m = 0; m < MT; ++m) least = min(least, min(lim[m][0], lim[m][1]));
  least = __reduce_min_sync(0xffffffffu, least);

  // ldmatrix addresses within a stage: keys for the scores, values transposed
  const int rk = (lane & 7) + ((lane >> 4) & 1) * 8, rv = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t ak = uint32_t(rk * CH * 16 + ((((lane >> 3) & 1) ^ (rk & 7)) << 4));
  const uint32_t av = uint32_t(P::KB + rv * CH * 16 + (((lane >> 4) ^ (rv & 7)) << 4));

  uint32_t on[NST - 1];
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) on[i] = issue(i);
  if (rest) clear_rest(a, seq, s, head, 0, 1);
  for (int i = 0; i < mine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();  // every lane's copies of this piece are in; the slot of piece i - 1 is free
    const uint32_t have = on[0];
#pragma unroll
    for (int k = 0; k + 2 < NST; ++k) on[k] = on[k + 1];
    on[NST - 2] = issue(i + NST - 1);
    const uint32_t st = ring + uint32_t((i % NST) * P::STAGE);

    // scores: 16 keys as two 8-key columns
    float sc[MT][2][4] = {};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b[4];
      ldsm4(b, (st + ak) ^ uint32_t(k << 5));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma<DT>(sc[m][0], qf[m][k], b[0], b[1]);
        mma<DT>(sc[m][1], qf[m][k], b[2], b[3]);
      }
    }
    const int key0 = k0 + (warp + i * NW) * KT;
    if (key0 + KT > least || have != 0xffffu) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = n * 8 + (lane & 3) * 2 + (e & 1);
            if (key0 + c >= lim[m][e >> 1] || !((have >> c) & 1u)) sc[m][n][e] = -INFINITY;
          }
    }
    // The weights stay under the maximum in use until a row outgrows it by
    // 2^8; then its sums are scaled and the new one is used.
    float mx[MT][2];
    bool grow = false;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(fmaxf(sc[m][0][h * 2], sc[m][0][h * 2 + 1]),
                        fmaxf(sc[m][1][h * 2], sc[m][1][h * 2 + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        mx[m][h] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        grow = grow || (mx[m][h] > m_[m][h] && !((mx[m][h] - m_[m][h]) * a.scale_log2 <= 8.0f));
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m_[m][h], mx[m][h]);
          const float f = m_[m][h] == -INFINITY ? 1.0f : ex2((m_[m][h] - mn) * a.scale_log2);
          m_[m][h] = mn;
          l_[m][h] *= f;
          u_[m][h] *= f;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[m][n][h * 2] *= f;
            o[m][n][h * 2 + 1] *= f;
          }
        }
    }
    uint32_t pf[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // subtracted before it is scaled: m * c is rounded, by 2^-8 at 2^16 and by
        // any power of two far past it
        const float at = m_[m][h] == -INFINITY ? 0.0f : m_[m][h];
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float &x = sc[m][n][h * 2 + e];
            x = ex2(__fmaf_rn(x - at, a.scale_log2, kWeightUp<DT>));
            sum += x;
          }
        l_[m][h] += sum;
      }
      pf[m][0] = pack2<DT>(sc[m][0][0], sc[m][0][1]);
      pf[m][1] = pack2<DT>(sc[m][0][2], sc[m][0][3]);
      pf[m][2] = pack2<DT>(sc[m][1][0], sc[m][1][1]);
      pf[m][3] = pack2<DT>(sc[m][1][2], sc[m][1][3]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[4];
        DT::unpack2(pf[m][h], x[0], x[1]);
        DT::unpack2(pf[m][2 + h], x[2], x[3]);
        u_[m][h] += (x[0] + x[1]) + (x[2] + x[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      ldsm4t(b, (st + av) ^ uint32_t(n << 5));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma<DT>(o[m][2 * n], pf[m], b[0], b[1]);
        mma<DT>(o[m][2 * n + 1], pf[m], b[2], b[3]);
      }
    }
    __syncwarp();  // all lanes have read the slot before it is refilled
  }
  if (bad) set_status(a.status, WQ_ERR_INDEX);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (NW == 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + h * 8 + lane / 4;
        const float l = quad_sum(l_[m][h]), w = quad_sum(u_[m][h]);
        if (r >= rows) continue;
        const float inv = w > 0.0f ? __fdiv_rn(1.0f, w) : (l == 0.0f ? 0.0f : w);
        const int j = (row0 + r) / a.G, g = (row0 + r) - j * a.G;
        const int64_t t = s.t0 + j, qh = head * a.G + g;
        if ((lane & 3) == 0) {
          const float lse = lse_of<DT>(m_[m][h], a.scale_log2, l);
          if (a.o_part) a.lse_part[(t * a.Hq + qh) * a.slots + slot] = lse;
          else if (a.lse) a.lse[t * a.Hq + qh] = lse;
        }
        if (a.o_part && l == 0.0f) continue;  // the join skips an empty part
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          const int d = n * 8 + (lane & 3) * 2;
          if (d >= a.dv) continue;
          const float x = o[m][n][h * 2] * inv, y = o[m][n][h * 2 + 1] * inv;
          if (a.o_part)
            *reinterpret_cast<float2 *>(a.o_part + ((t * a.Hq + qh) * a.slots + slot) * a.dv + d) =
                make_float2(x, y);
          else
            *reinterpret_cast<uint32_t *>(a.out + t * a.o_token + qh * a.o_head + d) = pack2<DT>(x, y);
        }
      }
    if (last_block) wait_last_kernel();
    return;
  }
  __syncthreads();  // the ring becomes the exchange of the warps' results

  constexpr int PITCH = D + 4;
  float *xo = reinterpret_cast<float *>(smem);
  __shared__ float xm[NW][R], xl[NW][R], xr[NW][R];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + lane / 4;
      const float l = quad_sum(l_[m][h]), u = quad_sum(u_[m][h]);
      if ((lane & 3) == 0) {
        xm[warp][r] = m_[m][h];
        xl[warp][r] = l;
        xr[warp][r] = u;
      }
      float *w = xo + (warp * R + r) * PITCH + (lane & 3) * 2;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2 *>(w + n * 8) = make_float2(o[m][n][h * 2], o[m][n][h * 2 + 1]);
    }
  __syncthreads();
  // a warp finishes every fourth row, a lane its columns lane * 2 + 64 c
  for (int r = warp; r < rows; r += NW) {
    float mx = xm[0][r];
#pragma unroll
    for (int w = 1; w < NW; ++w) mx = fmaxf(mx, xm[w][r]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    float f[NW], l = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      f[w] = ex2((xm[w][r] - base) * a.scale_log2);
      l = __fmaf_rn(xl[w][r], f[w], l);
      u = __fmaf_rn(xr[w][r], f[w], u);
    }
    const float inv = u > 0.0f ? __fdiv_rn(1.0f, u) : (l == 0.0f ? 0.0f : u);
    const int j = (row0 + r) / a.G, g = (row0 + r) - j * a.G;
    const int64_t t = s.t0 + j, qh = head * a.G + g;
    const float lse = lse_of<DT>(mx, a.scale_log2, l);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int d = c * 64 + lane * 2;
      if (d >= a.dv || (a.o_part && l == 0.0f)) continue;  // the join skips an empty part
      float x = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 v = *reinterpret_cast<const float2 *>(xo + (w * R + r) * PITCH + d);
        x = __fmaf_rn(v.x, f[w], x);
        y = __fmaf_rn(v.y, f[w], y);
      }
      x *= inv;
      y *= inv;
      if (a.o_part)
        *reinterpret_cast<float2 *>(a.o_part + ((t * a.Hq + qh) * a.slots + slot) * a.dv + d) =
            make_float2(x, y);
      else
        *reinterpret_cast<uint32_t *>(a.out + t * a.o_token + qh * a.o_head + d) = pack2<DT>(x, y);
    }
    if (lane == 0) {
      if (a.o_part) a.lse_part[(t * a.Hq + qh) * a.slots + slot] = lse;
      else if (a.lse) a.lse[t * a.Hq + qh] = lse;
    }
  }
  if (last_block) wait_last_kernel();
}

// Joins the partial results of a row: LANES threads, four columns each, walk
// its parts, four parts' columns in flight together.  Every thread finds the
// parts' weights itself (the statistics of a row are a few words of one line).
// A row of no sequence has its mark in the last slot, and others may hold
// anything.
template <class DT, int LANES>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a) {
  const int64_t row = int64_t(blockIdx.x) * (256 / LANES) + threadIdx.x / LANES;
  const int d = int(threadIdx.x) % LANES * 4;
  wait_last_kernel();
  if (row >= int64_t(a.T) * a.Hq || d >= a.dv) return;
  const float *lp = a.lse_part + row * a.slots;
  const float *op = a.o_part + row * a.slots * a.dv + d;
  float mx = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < a.slots; ++s) mx = fmaxf(mx, lp[s]);
  const float base = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f, x[4] = {};
  for (int s0 = 0; s0 < a.slots; s0 += 4) {
    float w[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k;
      w[k] = s < a.slots ? __expf(lp[s] - base) : 0.0f;
      // an empty part (weight zero) holds nothing that may be read
      v[k] = w[k] != 0.0f ? *reinterpret_cast<const float4 *>(op + int64_t(s) * a.dv)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sum += w[k];
      x[0] = __fmaf_rn(v[k].x, w[k], x[0]);
      x[1] = __fmaf_rn(v[k].y, w[k], x[1]);
      x[2] = __fmaf_rn(v[k].z, w[k], x[2]);
      x[3] = __fmaf_rn(v[k].w, w[k], x[3]);
    }
  }
  if (mx == kNoSequence) sum = x[0] = x[1] = x[2] = x[3] = 0.0f;
  const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : (sum == 0.0f ? 0.0f : sum);
  const int64_t t = row / a.Hq, qh = row - t * a.Hq;
  uint32_t *o = reinterpret_cast<uint32_t *>(a.out + t * a.o_token + qh * a.o_head + d);
  o[0] = pack2<DT>(x[0] * inv, x[1] * inv);
  o[1] = pack2<DT>(x[2] * inv, x[3] * inv);
  if (d == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

// The rows of no sequence, for calls whose suffixes the tile kernel takes or
// that have more rows than their sequences may have tokens, and (LAST: after all
// other work) for calls without suffixes.
template <bool LAST>
__global__ void __launch_bounds__(128) attn_rest_kernel(const AttnArgs a, int parts) {
  start_next_kernel();
  const int it = int(blockIdx.x / unsigned(parts)), part = int(blockIdx.x % unsigned(parts));
  const int seq = it / a.Hkv, head = it - seq * a.Hkv;
  if (LAST) wait_last_kernel();
  clear_rest(a, seq, source_of(a, seq), head, part, parts);
  if (!LAST && blockIdx.x == gridDim.x - 1) wait_last_kernel();
}

template <bool LAST>
int launch_rest(const AttnArgs &a, cudaStream_t st) {
  const int parts = std::max(1, a.T / 16 / a.B);  // so that none has many more than 16 rows
  const int64_t blocks = int64_t(a.B) * a.Hkv * parts;
  if (blocks >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  return launch_chained(attn_rest_kernel<LAST>, unsigned(blocks), 128, 0, true, st, a, parts);
}

template <class DT, int D, int MT, int NW, bool PAGED>
int launch_small(const AttnArgs &a, cudaStream_t st) {
  using P = Small<DT, D, MT, NW>;
  auto *k = attn_small_kernel<DT, D, MT, NW, PAGED>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, P::SMEM)) return WQ_ERR_LAUNCH;
  constexpr int R = 16 * MT;
  const int64_t pt = (int64_t(a.T) * a.G + R - 1) / R, stl = (int64_t(a.max_q) * a.G + R - 1) / R;
  const int64_t pi = a.tc_prefix || a.whole ? 0 : a.sp * pt * a.Hkv;
  const int64_t si = a.tc_suffix ? 0 : a.ss * stl * a.Hkv * a.B;
  if (pi + si == 0) return WQ_OK;
  if (pi + si >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  return launch_chained(k, unsigned(pi + si), NW * 32, P::SMEM, a.tc_prefix || a.tc_suffix, st, a,
                        int(pi), int(pt), int(stl));
}

template <class DT, int D, int MT>
int launch_warps(const AttnArgs &a, cudaStream_t st) {
  if (a.page_size % KT) return launch_small<DT, D, MT, 4, false>(a, st);
  return a.one_warp ? launch_small<DT, D, MT, 1, true>(a, st) : launch_small<DT, D, MT, 4, true>(a, st);
}

template <class DT>
int launch_t(const AttnArgs &a, cudaStream_t st) {
  const bool wide = a.dk > 64 || a.dv > 64, two = int64_t(a.max_q) * a.G > 16;
  int rc = launch_attention_tiles(a, std::is_same<DT, Bf16>::value ? WQ_DT_BF16 : WQ_DT_F16, st);
  if (rc != WQ_OK) return rc;
  if (wide) rc = two ? launch_warps<DT, 128, 2>(a, st) : launch_warps<DT, 128, 1>(a, st);
  else rc = two ? launch_warps<DT, 64, 2>(a, st) : launch_warps<DT, 64, 1>(a, st);
  if (rc == WQ_OK && a.cu_q && a.ss > 0 && a.rest_apart) rc = launch_rest<false>(a, st);
  const int64_t rows = int64_t(a.T) * a.Hq;
  if (rc == WQ_OK && a.o_part)
    rc = a.dv <= 64 ? launch_chained(attn_join_kernel<DT, 16>, unsigned((rows + 15) / 16), 256, 0, true, st, a)
                    : launch_chained(attn_join_kernel<DT, 32>, unsigned((rows + 7) / 8), 256, 0, true, st, a);
  if (rc == WQ_OK && a.cu_q && a.ss == 0) rc = launch_rest<true>(a, st);
  return rc;
}

}  // namespace

// Which kernel takes which part, and the cuts of the key ranges.
void plan_attention(AttnArgs &a) {
  // The tensor-memory kernel takes 128-row tiles and loads pages by TMA in
  // boxes of 8 rows or more with pitches that differ from zero.
  const bool pitches = (a.k_token || a.page_size == 1) && (a.k_head || a.Hkv == 1) &&
                       (a.k_page || a.num_pages <= 1) && (a.v_token || a.page_size == 1) &&
                       (a.v_head || a.Hkv == 1) && (a.v_page || a.num_pages <= 1);
  // Its waits end after 1 s, which a range of 2^25 keys does not reach.
  const bool tiles = a.page_size % 8 == 0 && a.num_pages > 0 && pitches &&
                     std::max(a.P, a.max_suffix) <= (1 << 25);
  const int64_t rows_p = int64_t(a.T) * a.G, rows_s = int64_t(a.max_q) * a.G;
  a.tc_suffix = tiles && a.max_suffix > 0 && rows_s > 32;
  // The prefix's products and the reading of short suffixes bind different
  // parts of the machine but do not fit one SM together.  So the prefix gets
  // only as many SMs as let the suffixes be read beside it: about 10 us and
  // 1.65 us a unit on each; suffixes (half their bound) at up to 6 TB/s, which
  // takes about 120 SMs.  Measured with 152 and with the chosen SMs: 64
  // sequences behind 8192 keys 68 and 56 us, 200 behind 30000 157 and 144 us.
  // (Heads of 64, whose units take 1.16 us, get more SMs than they need.)
  int sms = 152;
  if (a.max_suffix > 0 && !a.tc_suffix) {
    const int64_t pair = 2 * (128 / a.G), units = (a.T + pair - 1) / pair * a.Hkv * ((a.P + 127) / 128);
    const double read = 3.0 + double(a.B) * a.Hkv * a.max_suffix * (a.dk + a.dv) / 6e6;
    double best = 1e30;
    for (int k = 152; k >= 32; k -= 8) {
      const double products = 10.0 + 1.65 * double((units + k - 1) / k);
      const double all = products + std::max(0.0, read - products * std::min(1.0, (152 - k) / 120.0));
      if (all < best * 0.97) best = all, sms = k;
    }
  }
  a.tc_prefix = tiles && a.P > 0 && rows_p > 32 && plan_prefix_tiles(a, sms);
  const int64_t R = rows_s > 16 ? 32 : 16;
  const int64_t items_s = (rows_s + R - 1) / R * a.Hkv * a.B;
  // one warp a block where starts and ends weigh more than an even spread: many
  // pairs, ranges that are not long, pieces of 8 KB (heads over 64)
  a.one_warp = a.page_size % KT == 0 && items_s >= 64 && a.max_suffix <= 4096 && (a.dk > 64 || a.dv > 64);
  const int step = KT * (a.one_warp ? 1 : 4);
  a.step_pages = step / a.page_size;
  a.step_place = step % a.page_size;
  // ranges of `grain` keys or multiples, at least `least`, about `want` items
  auto cut = [](int64_t items, int64_t keys, int64_t want, int64_t least, int64_t grain, int &splits,
                int &chunk) {
    if (keys <= 0 || items <= 0) return;
    const int64_t n = std::max<int64_t>(
        std::min({(want + items - 1) / items, (keys + least - 1) / least, int64_t(64)}), 1);
    chunk = int(((keys + n - 1) / n + grain - 1) / grain * grain);
    splits = int((keys + chunk - 1) / chunk);
  };
  // About eight items an SM; twelve where ranges are long, whose ends then weigh
  // less than the unevenness of fewer (64 sequences of up to 8192 keys: 198 us
  // with 1216 items, 194 with 1824).
  const int64_t want = a.max_suffix > 4096 ? 1824 : 1216, least = a.one_warp ? 128 : 256;
  const int64_t grain = a.one_warp ? 16 : 64;
  if (!a.tc_prefix) cut((rows_p + R - 1) / R * a.Hkv, a.P, want, least, grain, a.sp, a.p_chunk);
  if (a.tc_suffix) {
    const int64_t pair = 2 * (128 / a.G);
    cut((a.max_q + pair - 1) / pair * a.Hkv * a.B, a.max_suffix, 152, 256, 128, a.ss, a.s_chunk);
  } else {
    cut(items_s, a.max_suffix, want, least, grain, a.ss, a.s_chunk);
  }
  // Enough row tiles for every SM: one walk over the prefix and the suffix of
  // a sequence's rows, with no partial results to join.
  const int64_t flat = (a.T + 2 * (128 / a.G) - 1) / (2 * (128 / a.G)) * a.Hkv;
  a.whole = a.tc_prefix && a.tc_suffix && a.ss == 1 && flat >= 152;
  if (a.whole) {
    a.tc_prefix = false;
    a.sp = 0;
  }
  if (a.sp + a.ss == 0) a.ss = 1;  // no keys at all: one empty range writes the zeros
  a.slots = a.sp + a.ss;
  a.rest_apart = a.tc_suffix || a.T > int64_t(a.B) * a.max_q;
}

size_t attention_ws_bytes(const AttnArgs &a) {
  if (a.slots == 1) return 0;
  const size_t rows = size_t(a.T) * a.Hq * a.slots;
  return ((rows * a.dv * 4 + 255) & ~size_t(255)) + rows * 4;
}

int launch_attention(const AttnArgs &a, int dtype, cudaStream_t st) {
  return dtype == WQ_DT_BF16 ? launch_t<Bf16>(a, st) : launch_t<F16>(a, st);
}

}  // namespace wq
