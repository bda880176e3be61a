// Low-rank adapters of many requests beside a shared projection:
//
//   y[t] += s_a (x[t] A_a^T) B_a^T   for token t with adapter a.
//
// Here: the kernel for few tokens, and the sorting of more than 256 by adapter
// (the products of many are in wq_lora_tc.cu).
//
// Tokens are taken in tiles of up to 16 of one adapter, and a cluster of blocks
// shares a tile: each block multiplies its slice of x and A (the first product's
// long axis), the parts are added through distributed shared memory in the order
// of the blocks, and each block multiplies the sum with its slice of B's rows
// (the second product's long axis) and adds the result to its columns of y.  So
// one launch reads x and the adapter once a tile, and reads and writes y once;
// the intermediate never leaves the cluster.  Every cluster finds its tile among
// up to 256 tokens itself, and in the sorted list of more.  Bound by latency: the
// chain from the adapters' numbers to the tokens' rows, the cluster's barrier, and
// two memory latencies (width 7168, rank 16: one token 6.2 us, of which a launch
// takes 2.5; 128 tokens over 32 adapters 10.5).
//
// x A^T is summed in float32 and enters the second product as 16-bit operands,
// its rounding and what that leaves: three of them in bf16, which hold all 24
// bits, two in fp16, taken relative to a power of two near a row's largest, which
// keeps them in range.  So only y is rounded.
#include <algorithm>

#include "wq_attn.cuh"
#include "wq_tc.cuh"
#include "wq_warp_mma.cuh"

namespace wq {
namespace {

using attn::start_next_kernel;
using attn::wait_last_kernel;

constexpr int NT = 256;
constexpr int kInline = 256;   // tokens that a cluster looks through itself
constexpr int kGroupThreads = 1024;
constexpr int kMostBlocks = 8;  // of a cluster

constexpr int BM = 16;  // tokens of a tile: a row tile of the warp products
constexpr int WK = 8;   // warps, along the long axes
constexpr int KS = 128;  // elements of x a stage of the first product
constexpr int NC = WK * 32;  // columns of y a stage of the second

// RP: rank in whole 16s.  The second product's stages hold rows of B and the
// columns of y that they go to, and the first ones are on their way from the
// start; with ranks over 64 they take the first product's place.
template <class DT, int RP>
struct Plan {
  static constexpr int OPS = kLoraOperands<DT>;
  static constexpr bool EARLY = RP < 128;
  static constexpr int XB = BM * KS * 2, AB = RP * KS * 2;
  static constexpr int N1 = RP < 128 ? 4 : 2;      // stages of the first product
  static constexpr int BP = ((RP / 8) | 1) * 16;   // bytes of a row of B in shared memory
  static constexpr int BB = NC * BP, YB = BM * NC * 2;
  static constexpr int N2 = RP < 128 ? 3 : 2;      // stages of the second
  static constexpr int HP = BP;                    // bytes of a row of the intermediate
  static constexpr int RED = WK * BM * RP * 4;     // the warps' sums
  static constexpr int OFF_1 = 0;                  // first product's stages, then the warps' sums and the operands
  static constexpr int OFF_H = OFF_1 + RED;        // [OPS][BM] rows: the operands, high ones first
  static constexpr int S0 = N1 * (XB + AB) > RED + OPS * BM * HP ? N1 * (XB + AB) : RED + OPS * BM * HP;
  static constexpr int S2 = N2 * (BB + YB);
  static constexpr int OFF_B = EARLY ? S0 : 0;     // second product's stages: rows of B, columns of y
  static constexpr int OFF_Y = OFF_B + N2 * BB;
  static constexpr int OFF_P = EARLY ? S0 + S2 : S0 > S2 ? S0 : S2;  // [BM][RP] float: this block's part
  static constexpr int OFF_UP = OFF_P + BM * RP * 4;                 // [BM] float: the rows' factors
  static constexpr int OFF_TOK = OFF_UP + BM * 4;                    // [BM] int
  static constexpr int OFF_MISC = OFF_TOK + BM * 4;
  static constexpr int SMEM = OFF_MISC + 64;
  static_assert(S0 >= NT * 4, "scratch of find_tile");
  static_assert(SMEM <= 232448, "shared memory plan");
};

__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// The tokens of this cluster's tile into tok; their adapter, or -1.  Without a
// list every thread looks at one token: `scratch` holds the adapters of all.
__device__ __forceinline__ int find_tile(const LoraArgs &a, int tile, int *tok, int *scratch, int *misc, int &count) {
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  if (a.order) {
    attn::wait_last_kernel();
    if (tile >= *a.ntiles) return -1;
    const int4 d = a.tiles[tile];
    if (i < d.z) tok[i] = a.order[d.y + i];
    __syncthreads();
    count = d.z;
    return d.x;
  }
  int id = i < a.T ? a.ids[i] : -1;
  if (id >= a.n) {
    if (tile == 0) set_status(a.status, WQ_ERR_INDEX);
    id = -1;
  }
  scratch[i] = id;
  if (a.T == 1) {
    if (i == 0) tok[0] = 0, misc[0] = id;
    __syncthreads();
    count = 1;
    return misc[0];
  }
  const uint32_t below = (1u << lane) - 1u;
  int before = __popc(__match_any_sync(0xffffffffu, id) & below);  // tokens of this adapter before
  __syncthreads();
  for (int j = 0; j < warp * 8; ++j) {
    const int4 v = reinterpret_cast<const int4 *>(scratch)[j];
    before += int(v.x == id) + int(v.y == id) + int(v.z == id) + int(v.w == id);
  }
  // tiles begin at every BM-th of an adapter's tokens, and count in the order of those
  const bool first = id >= 0 && before % BM == 0;
  const uint32_t m = __ballot_sync(0xffffffffu, first);
  if (lane == 0) misc[warp] = __popc(m);
  if (i == 0) misc[NT / 32] = -1;
  __syncthreads();
  int rank = __popc(m & below);
  for (int w = 0; w < warp; ++w) rank += misc[w];
  if (first && rank == tile) misc[NT / 32] = id, misc[NT / 32 + 1] = before;
  __syncthreads();
  const int own = misc[NT / 32], from = misc[NT / 32 + 1];
  if (own < 0) return -1;
  const bool mine = id == own && before >= from && before < from + BM;
  if (mine) tok[before - from] = i;
  count = __syncthreads_count(mine);
  return own;
}

template <class DT, int RP>
__global__ void __launch_bounds__(NT) lora_kernel(const LoraArgs a) {
  using P = Plan<DT, RP>;
  extern __shared__ __align__(128) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  int *tok = reinterpret_cast<int *>(sm + P::OFF_TOK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = int(cluster_size()), rank = int(tc::cluster_ctarank());
  int count = 0;
  const int id = find_tile(a, int(blockIdx.x) / C, tok, reinterpret_cast<int *>(sm),
                               reinterpret_cast<int *>(sm + P::OFF_MISC), count);
  if (id < 0) return;  // the whole cluster

  // A thread's copies keep their places in a stage, and step along in memory.
  // ---- the block's rows of B, for the second product
  const int chunks = (a.N + NC - 1) / NC;  // of columns of y, dealt out in stretches
  const int c0 = chunks * rank / C, c1 = chunks * (rank + 1) / C;
  constexpr int BP8 = RP / 8, NB = (NC * BP8 + NT - 1) / NT;  // pieces of a row; copies of a thread
  static_assert((NC * BP8 % NT == 0 || NB == 1) && NT % BP8 == 0, "whole copies, or one of some threads");
  const int b_row = threadIdx.x / BP8, b_piece = threadIdx.x % BP8;
  const uint16_t *b_src = a.B + (int64_t(id) * a.N + c0 * NC + b_row) * a.r + b_piece * 8;
  const bool b_on = b_piece * 8 < a.r;
  uint32_t b_to[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    // A thread of the second product gets eight neighbouring columns of y:
    // column 8t + 2p + e of a group of 32 is column 2t + e of its p-th tile
    const int row = b_row + j * (NT / BP8), g = row & 31;
    const int at = (row & ~31) + ((g >> 1) & 3) * 8 + (g >> 3) * 2 + (g & 1);
    b_to[j] = base + P::OFF_B + uint32_t(at * P::BP + b_piece * 16);
  }
  // the columns of y: four lanes of two rows each find their pieces in different banks
  constexpr int YP = NC / 8, YROWS = NT / YP, NY = P::YB / 16 / NT;  // pieces of a row; rows of a copy; copies
  const int y_row = threadIdx.x / YP, y_piece = threadIdx.x % YP;
  uint16_t *y_src[NY];
#pragma unroll
  for (int j = 0; j < NY; ++j) {
    const int row = y_row + j * YROWS;
    y_src[j] = row < count ? a.y + int64_t(tok[row]) * a.ldy + y_piece * 8 : nullptr;
  }
  static_assert(YROWS % 2 == 0, "a thread's rows lie alike");
  const uint32_t y_to = base + P::OFF_Y + uint32_t(y_row * (NC * 2) + ((y_piece ^ ((y_row & 1) << 2)) << 4));
  uint32_t b_stage = 0, y_stage = 0;
  int b_next = c0;
  auto load_b = [&]() {
    if (b_next < c1) {
      const bool in = b_next * NC + y_piece * 8 < a.N;
#pragma unroll
      for (int j = 0; j < NY; ++j) {
        const bool on = in && y_src[j];
        cp16(y_to + y_stage + j * YROWS * (NC * 2), on ? y_src[j] + b_next * NC : a.y, on);
      }
      y_stage = y_stage == (P::N2 - 1) * P::YB ? 0 : y_stage + P::YB;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (NC * BP8 < NT && b_row >= NC) break;
        const bool on = b_on && b_next * NC + b_row + j * (NT / BP8) < a.N;
        cp16(b_to[j] + b_stage, on ? b_src + int64_t(j) * (NT / BP8) * a.r : a.B, on);
      }
      b_src += int64_t(NC) * a.r;
      b_stage = b_stage == (P::N2 - 1) * P::BB ? 0 : b_stage + P::BB;
      ++b_next;
    }
    commit();
  };

  // ---- first product: this block's slice of the long axis
  const int steps = (a.H + KS - 1) / KS, s0 = steps * rank / C, s1 = steps * (rank + 1) / C;
  constexpr int PIECES = KS / 8, NX = BM * PIECES / NT, NA = (RP * PIECES + NT - 1) / NT, ROWS = NT / PIECES;
  static_assert(BM * PIECES % NT == 0 && (RP * PIECES % NT == 0 || NA == 1), "whole copies, or one of some threads");
  const int x_row = threadIdx.x / PIECES, x_piece = threadIdx.x % PIECES;
  const uint32_t x_to = base + P::OFF_1 + uint32_t(x_row * (KS * 2) + ((x_piece ^ (x_row & 7)) << 4));
  const uint16_t *x_src[NX], *a_src = a.A + (int64_t(id) * a.r + x_row) * a.H + s0 * KS + x_piece * 8;
  int x_ahead = 0;  // elements that x_src and a_src are to step on
  bool x_on[NX];
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    const int row = x_row + j * ROWS;
    x_on[j] = row < count;
    x_src[j] = a.x + int64_t(x_on[j] ? tok[row] : 0) * a.ldx + s0 * KS + x_piece * 8;
  }
  uint32_t x_stage = 0;
  int x_next = s0;
  auto load_x = [&]() {
    if (x_next < s1) {
      const bool in = x_next * KS + x_piece * 8 < a.H;
#pragma unroll
      for (int j = 0; j < NX; ++j) {
        const bool on = in && x_on[j];
        cp16(x_to + x_stage + j * ROWS * (KS * 2), on ? x_src[j] + x_ahead : a.x, on);
      }
#pragma unroll
      for (int j = 0; j < NA; ++j) {
        if (RP * PIECES < NT && x_row >= RP) break;
        const bool on = in && x_row + j * ROWS < a.r;
        cp16(x_to + x_stage + P::XB + j * ROWS * (KS * 2), on ? a_src + int64_t(j) * ROWS * a.H + x_ahead : a.A, on);
      }
      x_ahead += KS;
      x_stage = x_stage == (P::N1 - 1) * (P::XB + P::AB) ? 0 : x_stage + P::XB + P::AB;
      ++x_next;
    }
    commit();
  };
#pragma unroll
  for (int i = 0; i < P::N1 - 1; ++i) load_x();
  if constexpr (P::EARLY) {
#pragma unroll
    for (int i = 0; i < P::N2 - 1; ++i) load_b();
  }

  const int wk = warp;
  float acc[RP / 8][4];
#pragma unroll
  for (int i = 0; i < RP / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
  uint32_t xs = base + P::OFF_1;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    // groups of copies in order: x of the first stages, the second product's first, then x of one stage a step
    if (P::EARLY && s - s0 < P::N1 - 1) wait_group<P::N1 - 2 + P::N2 - 1>();
    else wait_group<P::N1 - 2>();
    __syncthreads();
    load_x();
    const uint32_t as = xs + P::XB;
#pragma unroll
    for (int kk = 0; kk < KS / 16 / WK; ++kk) {
      const int step = kk * WK + wk;
      uint32_t fa[4];
      {
        const int row = (lane & 15), piece = 2 * step + (lane >> 4);
        ldsm4(fa, xs + uint32_t(row * (KS * 2) + ((piece ^ (row & 7)) << 4)));
      }
#pragma unroll
      for (int p = 0; p < RP / 16; ++p) {
        uint32_t fb[4];
        const int row = p * 16 + (lane & 7) + ((lane >> 4) << 3), piece = 2 * step + ((lane >> 3) & 1);
        ldsm4(fb, as + uint32_t(row * (KS * 2) + ((piece ^ (row & 7)) << 4)));
        mma<DT>(acc[2 * p], fa, fb[0], fb[1]);
        mma<DT>(acc[2 * p + 1], fa, fb[2], fb[3]);
      }
    }
    xs = xs == base + P::OFF_1 + (P::N1 - 1) * (P::XB + P::AB) ? base + P::OFF_1 : xs + P::XB + P::AB;
  }
  // ---- its sum over the warps, then over the cluster's blocks
  wait_group<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(sm + P::OFF_1), *part = reinterpret_cast<float *>(sm + P::OFF_P);
#pragma unroll
  for (int i = 0; i < RP / 8; ++i) {
    const int row = (lane >> 2), col = i * 8 + (lane & 3) * 2;
    float *to = red + (wk * BM + row) * RP + col;
    *reinterpret_cast<float2 *>(to) = make_float2(acc[i][0], acc[i][1]);
    *reinterpret_cast<float2 *>(to + 8 * RP) = make_float2(acc[i][2], acc[i][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BM * RP / 4; i += NT) {
    float4 v = reinterpret_cast<float4 *>(red)[i];
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const float4 u = reinterpret_cast<float4 *>(red)[w * (BM * RP / 4) + i];
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    reinterpret_cast<float4 *>(part)[i] = v;
  }
  tc::cluster_sync();
  float *h = red;  // [BM][RP], the whole sum
  for (int i = threadIdx.x; i < BM * RP / 4; i += NT) {
    float4 u[kMostBlocks], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < kMostBlocks; ++c)
      if (c < C) u[c] = ld_cluster4(tc::mapa(base + P::OFF_P, uint32_t(c)) + uint32_t(i * 16));
#pragma unroll
    for (int c = 0; c < kMostBlocks; ++c) {
      if (c >= C) break;
      v.x += u[c].x;
      v.y += u[c].y;
      v.z += u[c].z;
      v.w += u[c].w;
    }
    reinterpret_cast<float4 *>(h)[i] = v;
  }
  tc::cluster_arrive();  // the others' parts are read
  __syncthreads();
  // ---- as operands of the second product, a warp a row at a time
  float *up = reinterpret_cast<float *>(sm + P::OFF_UP);
  const float scale = a.scales ? a.scales[id] : 1.0f;
  for (int row = warp; row < BM; row += NT / 32) {
    float down = 1.0f;
    if (std::is_same<DT, F16>::value) {
      float top = 0.0f;
      for (int c = lane; c < a.r; c += 32) top = fmaxf(top, fabsf(h[row * RP + c]));
      top = warp_max(top);
      // 2^-e with the row's largest in [2^e, 2^(e+1)), e within float's normal range
      const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -126), 126);
      down = __uint_as_float(uint32_t(127 - e) << 23);
      if (lane == 0) up[row] = __fmul_rn(scale, __uint_as_float(uint32_t(127 + e) << 23));
    } else if (lane == 0) {
      up[row] = scale;
    }
    for (int c = lane; c < RP; c += 32) {
      // past the rank nothing counts: an infinite x makes NaN of the padding's zeros
      float v = c < a.r ? __fmul_rn(h[row * RP + c], down) : 0.0f;
      uint8_t *to = sm + P::OFF_H + row * P::HP + c * 2;
#pragma unroll
      for (int q = 0; q < P::OPS; ++q) {
        const uint16_t w = DT::from_f(v);
        *reinterpret_cast<uint16_t *>(to + q * BM * P::HP) = w;
        v = lora_rest(v, DT::to_f(w));
      }
    }
  }
  __syncthreads();

  // ---- second product, and the sum with y
  uint32_t fh[P::OPS][RP / 16][4];
#pragma unroll
  for (int q = 0; q < P::OPS; ++q)
#pragma unroll
    for (int k = 0; k < RP / 16; ++k)
      ldsm4(fh[q][k], base + P::OFF_H + uint32_t((q * BM + (lane & 15)) * P::HP + (2 * k + (lane >> 4)) * 16));
  const int r0 = (lane >> 2), r1 = r0 + 8;
  const float up0 = up[r0], up1 = up[r1];
  uint16_t *y0 = a.y + int64_t(r0 < count ? tok[r0] : 0) * a.ldy, *y1 = a.y + int64_t(r1 < count ? tok[r1] : 0) * a.ldy;
  auto col_of = [&](int c) { return c * NC + wk * 32 + (lane & 3) * 8; };
  using V = Vec<DT, 8>;
  if constexpr (!P::EARLY) {
    __syncthreads();  // the operands are in registers: their place is the stages' now
#pragma unroll
    for (int i = 0; i < P::N2 - 1; ++i) load_b();
  }
  uint32_t ys = P::OFF_Y;
  uint32_t bs = base + P::OFF_B + uint32_t(wk * 32 * P::BP);
  const uint32_t b_end = bs + P::N2 * P::BB;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    wait_group<P::N2 - 2>();
    __syncthreads();
    load_b();
    const int piece = ((wk * 4 + (lane & 3)) ^ ((r0 & 1) << 2)) << 4;  // r1 = r0 + 8
    const V o0{*reinterpret_cast<const uint4 *>(sm + ys + r0 * (NC * 2) + piece)};
    const V o1{*reinterpret_cast<const uint4 *>(sm + ys + r1 * (NC * 2) + piece)};
    if ((ys += P::YB) == P::OFF_Y + P::N2 * P::YB) ys = P::OFF_Y;
    float d[4][4];
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[p][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < RP / 16; ++k) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t fb[4];
        ldsm4(fb, bs + uint32_t((p * 16 + (lane & 7) + ((lane >> 4) << 3)) * P::BP + (2 * k + ((lane >> 3) & 1)) * 16));
#pragma unroll
        for (int q = 0; q < P::OPS; ++q) {
          mma<DT>(d[2 * p], fh[q][k], fb[0], fb[1]);
          mma<DT>(d[2 * p + 1], fh[q][k], fb[2], fb[3]);
        }
      }
    }
    const int col = col_of(c);
    if (col < a.N) {
      float f[8];
      if (r0 < count) {
        o0.get(f);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          f[2 * p] = __fmaf_rn(d[p][0], up0, f[2 * p]);
          f[2 * p + 1] = __fmaf_rn(d[p][1], up0, f[2 * p + 1]);
        }
        V w;
        w.set(f);
        w.store(y0 + col);
      }
      if (r1 < count) {
        o1.get(f);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          f[2 * p] = __fmaf_rn(d[p][2], up1, f[2 * p]);
          f[2 * p + 1] = __fmaf_rn(d[p][3], up1, f[2 * p + 1]);
        }
        V w;
        w.set(f);
        w.store(y1 + col);
      }
    }
    if ((bs += P::BB) == b_end) bs -= P::N2 * P::BB;
  }
  wait_group<0>();
  tc::cluster_wait();  // this block's part has been read by all
}

// Tokens by adapter, and the tiles: one block.  The order of an adapter's
// tokens is left to chance; no result depends on a token's place in a tile.
__global__ void __launch_bounds__(kGroupThreads) lora_group_kernel(const LoraArgs a, int size) {
  extern __shared__ int cnt[];  // [n] tokens, then first places
  __shared__ int part[2][32];
  start_next_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int E = 8;  // tokens a thread looks at together
  auto load = [&](int t0, int(&id)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = t0 + e * kGroupThreads + int(threadIdx.x);
      id[e] = t < a.T ? a.ids[t] : -1;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (id[e] >= a.n) set_status(a.status, WQ_ERR_INDEX);
      id[e] = id[e] >= a.n || id[e] < 0 ? -1 : id[e];
    }
  };
  int id[E];
  load(0, id);
  for (int i = threadIdx.x; i < a.n; i += kGroupThreads) cnt[i] = 0;
  __syncthreads();
  // one atomic for the lanes that agree
  auto take = [&](int id) {
    const uint32_t m = __match_any_sync(0xffffffffu, id);
    const int lead = __ffs(int(m)) - 1;
    int at = 0;
    if (lane == lead && id >= 0) at = atomicAdd(&cnt[id], __popc(m));
    return __shfl_sync(0xffffffffu, at, lead) + __popc(m & ((1u << lane) - 1u));
  };
  int place[E];  // among the adapter's tokens; kept where one look takes all
  for (int t0 = 0; t0 < a.T; t0 += E * kGroupThreads) {
    if (t0) load(t0, id);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (t0 + e * kGroupThreads >= a.T) break;
      place[e] = take(id[e]);
    }
  }
  __syncthreads();
  // first place and first tile of each adapter: a thread has a stretch of them
  const int per = (a.n + kGroupThreads - 1) / kGroupThreads, n0 = min(int(threadIdx.x) * per, a.n), n1 = min(n0 + per, a.n);
  int tokens = 0, tiles = 0;
  for (int i = n0; i < n1; ++i) tokens += cnt[i], tiles += (cnt[i] + size - 1) / size;
  int st = tokens, sl = tiles;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, st, o), v = __shfl_up_sync(0xffffffffu, sl, o);
    if (lane >= o) st += u, sl += v;
  }
  if (lane == 31) part[0][warp] = st, part[1][warp] = sl;
  __syncthreads();
  int pt = part[0][lane], pl = part[1][lane];
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, pt, o), v = __shfl_up_sync(0xffffffffu, pl, o);
    if (lane >= o) pt += u, pl += v;
  }
  const int before = max(warp - 1, 0), all = __shfl_sync(0xffffffffu, pl, 31);
  const int bt = __shfl_sync(0xffffffffu, pt, before), bl = __shfl_sync(0xffffffffu, pl, before);
  int at = st - tokens + (warp ? bt : 0), tile = sl - tiles + (warp ? bl : 0);
  for (int i = n0; i < n1; ++i) {
    const int c = cnt[i];
    for (int k = 0; k < c; k += size) {
      if (a.tickets) a.tickets[tile] = 0;
      a.tiles[tile++] = make_int4(i, at + k, min(size, c - k), 0);
    }
    cnt[i] = at;
    at += c;
  }
  if (threadIdx.x == 0) *a.ntiles = all;
  __syncthreads();
  if (a.T <= E * kGroupThreads) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (id[e] >= 0) a.order[cnt[id[e]] + place[e]] = e * kGroupThreads + int(threadIdx.x);
    return;
  }
  for (int t0 = 0; t0 < a.T; t0 += E * kGroupThreads) {
    load(t0, id);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int to = take(id[e]);
      if (id[e] >= 0) a.order[to] = t0 + e * kGroupThreads + int(threadIdx.x);
    }
  }
}

template <class DT, int RP>
int launch_one(const LoraArgs &a, int64_t tiles, int C, cudaStream_t st) {
  using P = Plan<DT, RP>;
  auto *k = lora_kernel<DT, RP>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, P::SMEM)) return WQ_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(tiles * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = size_t(P::SMEM);
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.order ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, k, a) != cudaSuccess) return WQ_ERR_LAUNCH;
  return launched(1);
}

template <class DT>
int launch_rank(const LoraArgs &a, int64_t tiles, int C, cudaStream_t st) {
  if (a.r <= 16) return launch_one<DT, 16>(a, tiles, C, st);
  if (a.r <= 32) return launch_one<DT, 32>(a, tiles, C, st);
  if (a.r <= 64) return launch_one<DT, 64>(a, tiles, C, st);
  return launch_one<DT, 128>(a, tiles, C, st);
}

// Whether this kernel takes the tokens.  Its tiles read the adapter once for 16
// tokens, but need no second launch.  Width 7168, 8 adapters in runs of tokens,
// bf16, us here and with 128 tokens a tile:
//   rank 16    1024 tokens 16 23, 1536 tokens 24 26 | 2048 tokens 24 30, 3000 tokens 44 36
//   rank 32    1024 tokens 25 27 | 1536 tokens 39 29
//   rank 64    512 tokens 35 31 | 768 tokens 34 34, 1024 tokens 34 35, 2048 tokens 57 43
//   rank 128   288 tokens 38 43 | 384 tokens 38 46, 768 tokens 53 49
// The rule's border is at the bars: it gives away up to a fifth beside it, where
// either kernel's last round of blocks is nearly empty.
inline bool few(int64_t T, int r) { return T * std::max(r, 24) <= 36864; }
// Tokens of a tile, here and in the kernels for many; tiles at most
inline int tile_of(int64_t T, int r) { return few(T, r) ? BM : kLoraTile; }
inline int64_t tiles_of(int64_t T, int64_t n, int r) { return std::min(T, n + T / tile_of(T, r)); }
// Tiles to expect, by which the blocks of a tile are chosen: a batch of single
// tokens mixes adapters, prompts are runs of tokens.  (By the most, a few prompts
// among 512 adapters, 8192 tokens, took 143 us, and 90 so.)  Which adapters a batch
// uses is not known here.  Width 7168, rank 16, us by the most tiles and by runs: 256
// mixed tokens of 64 adapters 13 and 19, of 256 35 and 50, but 256 tokens that use 3
// of 512 26 and 20; past 256 tokens, 512 mixed ones of 32 15 and 18, of 256 40 and 57.
inline int64_t tiles_like(int64_t T, int64_t n, int r) {
  return T <= kInline ? tiles_of(T, n, r) : T / tile_of(T, r) + std::min(n, T / 256 + 1);
}

// Parts of the first product that any batch of up to T tokens has, each one's
// tokens times its slices.  A smaller batch may have more slices: s > 1 of them
// where 2 * 152 / s tiles or fewer are to be expected, which are more than
// tokens / kLoraTile, so that its parts stay below 2 * 152 * kLoraTile.
inline int64_t most_parts(int64_t T) {
  return std::max(T, std::min<int64_t>(T * kLoraSlices, 2 * 152 * kLoraTile));
}

// The workspace, from `at` on (nullptr: its size alone).  A larger T, n or r
// takes no less: a workspace made for the largest batch serves all.
size_t lora_lay_out(LoraArgs &a, char *at) {
  const int64_t tiles = tiles_of(a.T, a.n, a.r), T = a.T, RP = lora_rank(a.r);
  size_t n = 0;
  auto take = [&](auto *&p, int64_t count) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(at + n);
    n += (size_t(count) * sizeof(*p) + 15) / 16 * 16;
  };
  take(a.ntiles, 1);
  take(a.tiles, tiles);
  take(a.order, T);
  if (!few(T, a.r)) {
    take(a.tickets, tiles);
    take(a.factors, T);
    take(a.operands, T * RP / 2 * kLoraMostOperands);
    take(a.parts, most_parts(T) * RP);
  }
  return n;
}

}  // namespace

size_t lora_ws_bytes(int64_t T, int64_t n, int r) {
  if (T <= kInline) return 0;
  LoraArgs a{};
  a.T = int(T);
  a.n = int(n);
  a.r = r;
  return lora_lay_out(a, nullptr);
}

int launch_lora(LoraArgs a, int dtype, void *ws, cudaStream_t st) {
  const int64_t tiles = tiles_of(a.T, a.n, a.r);
  if (a.T > kInline) {
    lora_lay_out(a, static_cast<char *>(ws));
    lora_group_kernel<<<1, kGroupThreads, size_t(a.n) * 4, st>>>(a, tile_of(a.T, a.r));
    const int rc = launched(1);
    if (rc != WQ_OK) return rc;
    if (!few(a.T, a.r)) return launch_lora_tiles(a, dtype, tiles, tiles_like(a.T, a.n, a.r), st);
  }
  // Blocks of a tile: as many as let about all tiles run at the same time, two
  // blocks an SM
  int C = kMostBlocks;
  while (C > 1 && tiles_like(a.T, a.n, a.r) * C > 2 * 152 * 9 / 8) C /= 2;
  return dtype == WQ_DT_BF16 ? launch_rank<Bf16>(a, tiles, C, st) : launch_rank<F16>(a, tiles, C, st);
}

}  // namespace wq
