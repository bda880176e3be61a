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
// memory path they need no 128-row tile.
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
template <class DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<DT, Bf16>::value) return pack_bf16x2(lo, hi);
  else return f16x2_rn(lo, hi);
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

template <class DT, int D, int MT, int NW>
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
  const int rows = min(R, s.n * a.G - tile * R);  // rows of this tile
  if (rows <= 0) {
    wait_last_kernel();
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
  const uint16_t *kh = a.k + int64_t(head) * a.k_head;
  const uint16_t *vh = a.v + int64_t(head) * a.v_head;

  // page and place of the key that lane (mod 16) looks up for piece i; a key
  // past the range or on a bad page has page -1
  auto look = [&](int i, int &page, int &place) {
    const int key = k0 + (warp + i * NW) * KT + (lane & 15);
    page = -1;
    place = 0;
    if (i < mine && key < k1) {
      const int pi = key / a.page_size;
      place = key - pi * a.page_size;
      page = s.pages[pi];
      if (page < 0 || page >= a.num_pages) {
        set_status(a.status, WQ_ERR_INDEX);
        page = -1;
      }
    }
  };
  // bit r of `on`: key r of the piece is there
  auto issue = [&](int i, int page, int place) -> uint32_t {
    const uint32_t on = __ballot_sync(0xffffffffu, page >= 0) & 0xffffu;
    if (i < mine) {
      const uint32_t st = ring + uint32_t((i % NST) * P::STAGE);
#pragma unroll
      for (int j = 0; j < KT * CH / 32; ++j) {
        const int c = j * 32 + lane, r = c / CH, ch = c % CH;
        const int pg = __shfl_sync(0xffffffffu, page, r), pl = __shfl_sync(0xffffffffu, place, r);
        const bool ok = pg >= 0;
        const uint32_t d = st + uint32_t(r * CH + (ch ^ (r & 7))) * 16;
        const int64_t p64 = ok ? pg : 0;
        const bool kk = ok && ch * 8 < a.dk, vv = ok && ch * 8 < a.dv;
        cp16(d, kh + p64 * a.k_page + int64_t(pl) * a.k_token + (kk ? ch * 8 : 0), kk);
        cp16(d + P::KB, vh + p64 * a.v_page + int64_t(pl) * a.v_token + (vv ? ch * 8 : 0), vv);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return on;
  };

  float m_[MT][2], l_[MT][2], o[MT][D / 8][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    m_[m][0] = m_[m][1] = -INFINITY;
    l_[m][0] = l_[m][1] = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
  }

  uint32_t on[NST];
  int page, place;
  look(0, page, place);
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) {
    on[i] = issue(i, page, place);
    look(i + 1, page, place);
  }
  for (int i = 0; i < mine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();  // every lane's copies of this piece are in; the slot of piece i - 1 is free
    const uint32_t next_on = issue(i + NST - 1, page, place);
    look(i + NST, page, place);
    const uint32_t st = ring + uint32_t((i % NST) * P::STAGE);
    const uint32_t have = on[0];
#pragma unroll
    for (int k = 0; k + 1 < NST - 1; ++k) on[k] = on[k + 1];
    on[NST - 2] = next_on;

    // scores: 16 keys as two 8-key columns
    float sc[MT][2][4] = {};
    {
      const int r = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int ch = k * 2 + ((lane >> 3) & 1);
        uint32_t b[4];
        ldsm4(b, st + uint32_t(r * CH + (ch ^ (r & 7))) * 16);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma<DT>(sc[m][0], qf[m][k], b[0], b[1]);
          mma<DT>(sc[m][1], qf[m][k], b[2], b[3]);
        }
      }
    }
    const int key0 = k0 + (warp + i * NW) * KT;
    uint32_t pf[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = n * 8 + (lane & 3) * 2 + e;
            float &x = sc[m][n][h * 2 + e];
            x = (key0 + c < lim[m][h] && ((have >> c) & 1u)) ? __fmul_rn(x, a.scale_log2)
                                                              : -INFINITY;
            mx = fmaxf(mx, x);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m_[m][h], mx);
        const float base = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet: all weights 0
        const float corr = ex2(m_[m][h] - base);
        m_[m][h] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float &x = sc[m][n][h * 2 + e];
            x = ex2(x - base);
            sum += x;
          }
        l_[m][h] = __fmaf_rn(l_[m][h], corr, sum);
        if (corr != 1.0f) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[m][n][h * 2] *= corr;
            o[m][n][h * 2 + 1] *= corr;
          }
        }
      }
      pf[m][0] = pack2<DT>(sc[m][0][0], sc[m][0][1]);
      pf[m][1] = pack2<DT>(sc[m][0][2], sc[m][0][3]);
      pf[m][2] = pack2<DT>(sc[m][1][0], sc[m][1][1]);
      pf[m][3] = pack2<DT>(sc[m][1][2], sc[m][1][3]);
    }
    {
      const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        const int ch = n * 2 + (lane >> 4);
        uint32_t b[4];
        ldsm4t(b, st + P::KB + uint32_t(r * CH + (ch ^ (r & 7))) * 16);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma<DT>(o[m][2 * n], pf[m], b[0], b[1]);
          mma<DT>(o[m][2 * n + 1], pf[m], b[2], b[3]);
        }
      }
    }
    __syncwarp();  // all lanes have read the slot before it is refilled
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (NW == 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = m * 16 + h * 8 + lane / 4;
        float l = l_[m][h];  // this thread's keys only, so far
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (r >= rows) continue;
        const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);
        const int j = (row0 + r) / a.G, g = (row0 + r) - j * a.G;
        const int64_t t = s.t0 + j, qh = head * a.G + g;
        if ((lane & 3) == 0) {
          const float lse = l == 0.0f ? -INFINITY : (m_[m][h] + log2f(l)) * 0.6931471805599453f;
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
    wait_last_kernel();  // the join waits for this kernel alone
    return;
  }
  __syncthreads();  // the ring becomes the exchange of the warps' results

  constexpr int PITCH = D + 4;
  float *xo = reinterpret_cast<float *>(smem);
  __shared__ float xm[NW][R], xl[NW][R];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + lane / 4;
      float l = l_[m][h];  // this thread's keys only, so far
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if ((lane & 3) == 0) {
        xm[warp][r] = m_[m][h];
        xl[warp][r] = l;
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
    float f[NW], l = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      f[w] = ex2(xm[w][r] - base);
      l = __fmaf_rn(xl[w][r], f[w], l);
    }
    const float inv = l > 0.0f ? __fdiv_rn(1.0f, l) : (l == 0.0f ? 0.0f : l);
    const int j = (row0 + r) / a.G, g = (row0 + r) - j * a.G;
    const int64_t t = s.t0 + j, qh = head * a.G + g;
    const float lse = l == 0.0f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
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
  wait_last_kernel();
}

// A warp joins one row's partial results, 32 at a time: a lane finds one
// part's weight, and four parts' rows are in flight together.
template <class DT>
__global__ void __launch_bounds__(128) attn_join_kernel(const AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  wait_last_kernel();
  if (row >= int64_t(a.T) * a.Hq) return;
  const float *lp = a.lse_part + row * a.slots;
  const int d = min(lane * 4, a.dv - 4);
  const float *op = a.o_part + row * a.slots * a.dv + d;
  float mx = -INFINITY;
  for (int s = lane; s < a.slots; s += 32) mx = fmaxf(mx, lp[s]);
  mx = warp_max(mx);
  const int64_t t = row / a.Hq, qh = row - t * a.Hq;
  const float base = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f, x[4] = {};
  for (int s0 = 0; s0 < a.slots; s0 += 32) {
    const float mine = s0 + lane < a.slots ? __expf(lp[s0 + lane] - base) : 0.0f;
    sum += warp_sum(mine);
    const int n = min(32, a.slots - s0);
    for (int i = 0; i < n; i += 4) {
      float w[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = __shfl_sync(0xffffffffu, mine, (i + k) & 31);
        if (i + k >= n) w[k] = 0.0f;
        // an empty part (weight zero) holds nothing that may be read
        v[k] = w[k] != 0.0f ? *reinterpret_cast<const float4 *>(op + int64_t(s0 + i + k) * a.dv)
                            : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[0] = __fmaf_rn(v[k].x, w[k], x[0]);
        x[1] = __fmaf_rn(v[k].y, w[k], x[1]);
        x[2] = __fmaf_rn(v[k].z, w[k], x[2]);
        x[3] = __fmaf_rn(v[k].w, w[k], x[3]);
      }
    }
  }
  const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : (sum == 0.0f ? 0.0f : sum);
  if (lane * 4 < a.dv) {
    uint32_t *o = reinterpret_cast<uint32_t *>(a.out + t * a.o_token + qh * a.o_head + d);
    o[0] = pack2<DT>(x[0] * inv, x[1] * inv);
    o[1] = pack2<DT>(x[2] * inv, x[3] * inv);
  }
  if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

template <class DT, int D, int MT, int NW>
int launch_small(const AttnArgs &a, cudaStream_t st) {
  using P = Small<DT, D, MT, NW>;
  auto *k = attn_small_kernel<DT, D, MT, NW>;
  static bool sized = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           P::SMEM) == cudaSuccess;
  if (!sized) return WQ_ERR_LAUNCH;
  constexpr int R = 16 * MT;
  const int64_t pt = (int64_t(a.T) * a.G + R - 1) / R, stl = (int64_t(a.max_q) * a.G + R - 1) / R;
  const int64_t pi = a.tc_prefix ? 0 : a.sp * pt * a.Hkv;
  const int64_t si = a.tc_suffix ? 0 : a.ss * stl * a.Hkv * a.B;
  if (pi + si == 0) return WQ_OK;
  if (pi + si >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  return launch_chained(k, unsigned(pi + si), NW * 32, P::SMEM, a.tc_prefix || a.tc_suffix, st, a,
                        int(pi), int(pt), int(stl));
}

template <class DT, int D, int MT>
int launch_warps(const AttnArgs &a, cudaStream_t st) {
  return a.one_warp ? launch_small<DT, D, MT, 1>(a, st) : launch_small<DT, D, MT, 4>(a, st);
}

template <class DT>
int launch_t(const AttnArgs &a, cudaStream_t st) {
  const bool wide = a.dk > 64 || a.dv > 64, two = int64_t(a.max_q) * a.G > 16;
  int rc = launch_attention_tiles(a, std::is_same<DT, Bf16>::value ? WQ_DT_BF16 : WQ_DT_F16, st);
  if (rc != WQ_OK) return rc;
  if (wide) rc = two ? launch_warps<DT, 128, 2>(a, st) : launch_warps<DT, 128, 1>(a, st);
  else rc = two ? launch_warps<DT, 64, 2>(a, st) : launch_warps<DT, 64, 1>(a, st);
  if (rc != WQ_OK || !a.o_part) return rc;
  const int64_t rows = int64_t(a.T) * a.Hq;
  return launch_chained(attn_join_kernel<DT>, unsigned((rows + 3) / 4), 128, 0, true, st, a);
}

}  // namespace

// Which kernel takes which part, and the cuts of the key ranges.
void plan_attention(AttnArgs &a) {
  // The tensor-memory kernel takes 128-row tiles and loads pages by TMA in
  // boxes of 8 rows or more with pitches that differ from zero.
  const bool pitches = (a.k_token || a.page_size == 1) && (a.k_head || a.Hkv == 1) &&
                       (a.k_page || a.num_pages <= 1) && (a.v_token || a.page_size == 1) &&
                       (a.v_head || a.Hkv == 1) && (a.v_page || a.num_pages <= 1);
  const bool tiles = a.page_size % 8 == 0 && a.num_pages > 0 && pitches;
  const int64_t rows_p = int64_t(a.T) * a.G, rows_s = int64_t(a.max_q) * a.G;
  a.tc_prefix = tiles && a.P > 0 && rows_p > 32 && plan_prefix_tiles(a);
  a.tc_suffix = tiles && a.max_suffix > 0 && rows_s > 32;
  const int64_t R = rows_s > 16 ? 32 : 16;
  const int64_t items_s = (rows_s + R - 1) / R * a.Hkv * a.B;
  a.one_warp = items_s >= 4 * 152;
  // ranges of `grain` keys or multiples, at least `least`, about `want` items
  auto cut = [](int64_t items, int64_t keys, int64_t want, int64_t least, int64_t grain, int &splits,
                int &chunk) {
    if (keys <= 0 || items <= 0) return;
    const int64_t n = std::max<int64_t>(
        std::min({(want + items - 1) / items, (keys + least - 1) / least, int64_t(64)}), 1);
    chunk = int(((keys + n - 1) / n + grain - 1) / grain * grain);
    splits = int((keys + chunk - 1) / chunk);
  };
  const int64_t want = a.one_warp ? 2 * 9 * 152 : 4 * 2 * 152, least = a.one_warp ? 128 : 256;
  const int64_t grain = a.one_warp ? 16 : 64;
  if (!a.tc_prefix) cut((rows_p + R - 1) / R * a.Hkv, a.P, want, least, grain, a.sp, a.p_chunk);
  if (a.tc_suffix) {
    const int64_t pair = 2 * (128 / a.G);
    cut((a.max_q + pair - 1) / pair * a.Hkv * a.B, a.max_suffix, 152, 256, 128, a.ss, a.s_chunk);
  } else {
    cut(items_s, a.max_suffix, want, least, grain, a.ss, a.s_chunk);
  }
  if (a.sp + a.ss == 0) a.ss = 1;  // no keys at all: one empty range writes the zeros
  a.slots = a.sp + a.ss;
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
