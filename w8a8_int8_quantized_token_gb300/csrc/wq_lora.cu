// Low-rank adapters of many requests beside a shared projection:
//
//   y[t] += s_a (x[t] A_a^T) B_a^T   for token t with adapter a.
//
// Tokens are taken in tiles of one adapter.  A cluster of blocks shares a tile:
// each block multiplies its slice of x and A (the first product's long axis),
// the parts are added through distributed shared memory in the order of the
// blocks, and each block multiplies the sum with its slice of B's rows (the
// second product's long axis) and adds the result to its columns of y.  So one
// launch reads x and the adapter once a tile, and reads and writes y once; the
// intermediate never leaves the cluster.  Bound by HBM: a rank of 16 needs 16
// operations a byte, one of 64 about 60.
//
// x A^T is summed in float32 and enters the second product as two 16-bit
// operands, its rounding and what that leaves (16 bits of it together), so that
// only y is rounded.  fp16 operands are taken relative to a power of two near a
// row's largest, which keeps them in range.
//
// Up to 256 tokens every cluster finds its tile itself: that of token t exists
// if t is the first of its adapter's tokens or comes a multiple of a tile after
// it.  With more tokens a first kernel sorts them by adapter.
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

// BM: tokens of a tile; RP: rank in whole 16s
template <int BM, int RP>
struct Plan {
  static constexpr int WM = BM / 16, WK = 8 / WM;  // warps along tokens, and along the first product's axis
  static constexpr int KS = BM == 16 ? 128 : 64;   // elements of x a stage
  static constexpr int XB = BM * KS * 2, AB = RP * KS * 2;
  static constexpr int N1 = RP < 128 ? 4 : BM == 16 ? 2 : 3;     // stages of the first product
  static constexpr int NC = WK * 32;               // columns of y a stage of the second
  static constexpr int BP = ((RP / 8) | 1) * 16;   // bytes of a row of B in shared memory
  static constexpr int BB = NC * BP;
  static constexpr int N2 = RP < 64 ? 4 : RP == 64 ? 3 : BM == 16 ? 2 : 3;      // its stages
  static constexpr int HP = BP;                    // bytes of a row of the intermediate
  static constexpr int OFF_1 = 0;                  // first product's stages, then the warps' sums and the operands
  static constexpr int RED = WK * BM * RP * 4;
  static constexpr int OFF_H = OFF_1 + RED;            // [2][BM] rows: high and low operands
  static constexpr int S1 = N1 * (XB + AB) > RED + 2 * BM * HP ? N1 * (XB + AB) : RED + 2 * BM * HP;
  static constexpr int OFF_B = OFF_1 + S1;
  static constexpr int OFF_P = OFF_B + N2 * BB;        // [BM][RP] float: this block's part
  static constexpr int OFF_UP = OFF_P + BM * RP * 4;   // [BM] float: the rows' factors
  static constexpr int OFF_TOK = OFF_UP + BM * 4;      // [BM] int
  static constexpr int OFF_MISC = OFF_TOK + BM * 4;
  static constexpr int SMEM = OFF_MISC + 64;
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The tokens of this cluster's tile into tok; their adapter, or -1
template <int BM>
__device__ __forceinline__ int find_tile(const LoraArgs &a, int tile, int *tok, int *misc, int &count) {
  if (a.order) {
    wait_last_kernel();
    if (tile >= *a.ntiles) return -1;
    const int4 d = a.tiles[tile];
    for (int i = threadIdx.x; i < d.z; i += NT) tok[i] = a.order[d.y + i];
    __syncthreads();
    count = d.z;
    return d.x;
  }
  // token `tile` and those after it with its adapter, if a tile begins there
  const int id = a.ids[tile], i = threadIdx.x;
  if (id < 0 || id >= a.n) {
    if (id >= a.n && i == 0) set_status(a.status, WQ_ERR_INDEX);
    return -1;
  }
  const bool same = i < a.T && a.ids[i] == id;
  const uint32_t m = __ballot_sync(0xffffffffu, same);
  if ((i & 31) == 0) misc[i >> 5] = int(m);
  __syncthreads();
  int before = 0, mine = __popc(m & ((1u << (i & 31)) - 1u)), all = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const uint32_t v = uint32_t(misc[w]);
    if (w < i >> 5) mine += __popc(v);
    before += w < tile >> 5 ? __popc(v) : w == tile >> 5 ? __popc(v & ((1u << (tile & 31)) - 1u)) : 0;
    all += __popc(v);
  }
  if (before % BM) return -1;
  if (same && mine >= before && mine < before + BM) tok[mine - before] = i;
  __syncthreads();
  count = min(BM, all - before);
  return id;
}

template <class DT, int BM, int RP>
__global__ void __launch_bounds__(NT) lora_kernel(const LoraArgs a) {
  using P = Plan<BM, RP>;
  extern __shared__ __align__(128) uint8_t sm[];
  const uint32_t base = tc::smem_u32(sm);
  int *tok = reinterpret_cast<int *>(sm + P::OFF_TOK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = int(cluster_size()), rank = int(tc::cluster_ctarank());
  int count = 0;
  const int id = find_tile<BM>(a, int(blockIdx.x) / C, tok, reinterpret_cast<int *>(sm + P::OFF_MISC), count);
  if (id < 0) return;  // the whole cluster

  // ---- the block's rows of B, ahead of all else
  const uint16_t *B = a.B + int64_t(id) * a.N * a.r;
  const int chunks = (a.N + P::NC - 1) / P::NC;  // of columns of y, dealt out in stretches
  const int c0 = chunks * rank / C, c1 = chunks * (rank + 1) / C;
  auto load_b = [&](int c) {
    if (c < c1) {
      const uint32_t to = base + P::OFF_B + uint32_t((c - c0) % P::N2 * P::BB);
      for (int i = threadIdx.x; i < P::NC * (RP / 8); i += NT) {
        // A thread of the second product gets eight neighbouring columns of y:
        // column 8t + 2p + e of a group of 32 is column 2t + e of its p-th tile
        const int row = i / (RP / 8), piece = i % (RP / 8), n = c * P::NC + row;
        const int g = row & 31, at = (row & ~31) + ((g >> 1) & 3) * 8 + (g >> 3) * 2 + (g & 1);
        const bool on = n < a.N && piece * 8 < a.r;
        cp16(to + uint32_t(at * P::BP + piece * 16), B + (on ? int64_t(n) * a.r + piece * 8 : 0), on);
      }
    }
    commit();
  };

  // ---- first product: this block's slice of the long axis
  const uint16_t *A = a.A + int64_t(id) * a.r * a.H;
  const int steps = (a.H + P::KS - 1) / P::KS, s0 = steps * rank / C, s1 = steps * (rank + 1) / C;
  constexpr int PIECES = P::KS / 8;
  auto load_x = [&](int s) {
    if (s < s1) {
      const uint32_t to = base + P::OFF_1 + uint32_t((s - s0) % P::N1 * (P::XB + P::AB));
      for (int i = threadIdx.x; i < (BM + RP) * PIECES; i += NT) {
        const int row = i / PIECES, piece = i % PIECES, k = s * P::KS + piece * 8;
        const bool isx = row < BM;
        const int rr = isx ? row : row - BM;
        const bool on = k < a.H && (isx ? rr < count : rr < a.r);
        const uint16_t *src = isx ? a.x + int64_t(on ? tok[rr] : 0) * a.ldx : A + int64_t(on ? rr : 0) * a.H;
        cp16(to + uint32_t(row * (P::KS * 2) + ((piece ^ (row & 7)) << 4)), src + (on ? k : 0), on);
      }
    }
    commit();
  };
#pragma unroll
  for (int i = 0; i < P::N1 - 1; ++i) load_x(s0 + i);
#pragma unroll
  for (int i = 0; i < P::N2 - 1; ++i) load_b(c0 + i);

  const int wm = warp % P::WM, wk = warp / P::WM;
  float acc[RP / 8][4];
#pragma unroll
  for (int i = 0; i < RP / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    // groups of copies in order: x of the first stages, all of B's, then x of one stage a step
    if (s - s0 < P::N1 - 1) wait_group<P::N1 - 2 + P::N2 - 1>();
    else wait_group<P::N1 - 2>();
    __syncthreads();
    load_x(s + P::N1 - 1);
    const uint32_t xs = base + P::OFF_1 + uint32_t((s - s0) % P::N1 * (P::XB + P::AB)), as = xs + P::XB;
#pragma unroll
    for (int kk = 0; kk < P::KS / 16 / P::WK; ++kk) {
      const int step = kk * P::WK + wk;
      uint32_t fa[4];
      {
        const int row = wm * 16 + (lane & 15), piece = 2 * step + (lane >> 4);
        ldsm4(fa, xs + uint32_t(row * (P::KS * 2) + ((piece ^ (row & 7)) << 4)));
      }
#pragma unroll
      for (int p = 0; p < RP / 16; ++p) {
        uint32_t fb[4];
        const int row = p * 16 + (lane & 7) + ((lane >> 4) << 3), piece = 2 * step + ((lane >> 3) & 1);
        ldsm4(fb, as + uint32_t(row * (P::KS * 2) + ((piece ^ (row & 7)) << 4)));
        mma<DT>(acc[2 * p], fa, fb[0], fb[1]);
        mma<DT>(acc[2 * p + 1], fa, fb[2], fb[3]);
      }
    }
  }
  // ---- its sum over the warps, then over the cluster's blocks
  wait_group<0>();
  __syncthreads();
  float *red = reinterpret_cast<float *>(sm + P::OFF_1), *part = reinterpret_cast<float *>(sm + P::OFF_P);
#pragma unroll
  for (int i = 0; i < RP / 8; ++i) {
    const int row = wm * 16 + (lane >> 2), col = i * 8 + (lane & 3) * 2;
    float *to = red + (wk * BM + row) * RP + col;
    *reinterpret_cast<float2 *>(to) = make_float2(acc[i][0], acc[i][1]);
    *reinterpret_cast<float2 *>(to + 8 * RP) = make_float2(acc[i][2], acc[i][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BM * RP / 4; i += NT) {
    float4 v = reinterpret_cast<float4 *>(red)[i];
#pragma unroll
    for (int w = 1; w < P::WK; ++w) {
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
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = 0; c < C; ++c) {
      const float4 u = ld_cluster4(tc::mapa(base + P::OFF_P, uint32_t(c)) + uint32_t(i * 16));
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    reinterpret_cast<float4 *>(h)[i] = v;
  }
  cluster_arrive();  // the others' parts are read
  __syncthreads();
  // ---- as operands of the second product, a warp a row at a time
  float *up = reinterpret_cast<float *>(sm + P::OFF_UP);
  const float scale = a.scales ? a.scales[id] : 1.0f;
  for (int row = warp; row < BM; row += NT / 32) {
    float down = 1.0f;
    if (std::is_same<DT, F16>::value) {
      float top = 0.0f;
      for (int c = lane; c < RP; c += 32) top = fmaxf(top, fabsf(h[row * RP + c]));
      top = warp_max(top);
      // 2^-e with the row's largest in [2^e, 2^(e+1)), e within float's normal range
      const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -126), 126);
      down = __uint_as_float(uint32_t(127 - e) << 23);
      if (lane == 0) up[row] = __fmul_rn(scale, __uint_as_float(uint32_t(127 + e) << 23));
    } else if (lane == 0) {
      up[row] = scale;
    }
    for (int c = lane; c < RP; c += 32) {
      const float v = __fmul_rn(h[row * RP + c], down);
      const uint16_t hi = DT::from_f(v);
      const float f = DT::to_f(hi);
      uint8_t *to = sm + P::OFF_H + row * P::HP + c * 2;
      *reinterpret_cast<uint16_t *>(to) = hi;
      *reinterpret_cast<uint16_t *>(to + BM * P::HP) = fabsf(f) == INFINITY ? uint16_t(0) : DT::from_f(v - f);
    }
  }
  __syncthreads();

  // ---- second product, and the sum with y
  uint32_t fh[2][RP / 16][4];
#pragma unroll
  for (int part2 = 0; part2 < 2; ++part2)
#pragma unroll
    for (int k = 0; k < RP / 16; ++k)
      ldsm4(fh[part2][k], base + P::OFF_H + uint32_t((part2 * BM + wm * 16 + (lane & 15)) * P::HP + (2 * k + (lane >> 4)) * 16));
  const int r0 = wm * 16 + (lane >> 2), r1 = r0 + 8;
  const float up0 = up[r0], up1 = up[r1];
  uint16_t *y0 = a.y + int64_t(r0 < count ? tok[r0] : 0) * a.ldy, *y1 = a.y + int64_t(r1 < count ? tok[r1] : 0) * a.ldy;
  auto col_of = [&](int c) { return c * P::NC + wk * 32 + (lane & 3) * 8; };
  using V = Vec<DT, 8>;
  V v0{}, v1{};
  auto load_y = [&](int c) {
    const int col = col_of(c);
    if (c < c1 && col < a.N) {
      if (r0 < count) v0 = V::load(y0 + col);
      if (r1 < count) v1 = V::load(y1 + col);
    }
  };
  load_y(c0);
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    wait_group<P::N2 - 2>();
    __syncthreads();
    load_b(c + P::N2 - 1);
    const V o0 = v0, o1 = v1;
    load_y(c + 1);
    const uint32_t bs = base + P::OFF_B + uint32_t((c - c0) % P::N2 * P::BB + wk * 32 * P::BP);
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
        for (int q = 0; q < 2; ++q) {
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
  }
  wait_group<0>();
  cluster_wait();  // this block's part has been read by all
}

// Tokens by adapter, and the tiles: one block.  The order of an adapter's
// tokens is left to chance; no result depends on a token's place in a tile.
__global__ void __launch_bounds__(kGroupThreads) lora_group_kernel(const LoraArgs a, int BM) {
  extern __shared__ int cnt[];  // [n] tokens, then first places
  __shared__ int part[2][32];
  start_next_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.n; i += kGroupThreads) cnt[i] = 0;
  __syncthreads();
  auto id_of = [&](int t) {
    const int id = t < a.T ? a.ids[t] : -1;
    if (id >= a.n) set_status(a.status, WQ_ERR_INDEX);
    return id >= a.n || id < 0 ? -1 : id;
  };
  // one atomic for the lanes that agree
  auto take = [&](int id) {
    const uint32_t m = __match_any_sync(0xffffffffu, id);
    const int lead = __ffs(int(m)) - 1;
    int at = 0;
    if (lane == lead && id >= 0) at = atomicAdd(&cnt[id], __popc(m));
    return __shfl_sync(0xffffffffu, at, lead) + __popc(m & ((1u << lane) - 1u));
  };
  for (int t0 = 0; t0 < a.T; t0 += kGroupThreads) take(id_of(t0 + int(threadIdx.x)));
  __syncthreads();
  // first place and first tile of each adapter: a thread has a stretch of them
  const int per = (a.n + kGroupThreads - 1) / kGroupThreads, n0 = min(int(threadIdx.x) * per, a.n), n1 = min(n0 + per, a.n);
  int tokens = 0, tiles = 0;
  for (int i = n0; i < n1; ++i) tokens += cnt[i], tiles += (cnt[i] + BM - 1) / BM;
  int st = tokens, sl = tiles;
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, st, o), v = __shfl_up_sync(0xffffffffu, sl, o);
    if (lane >= o) st += u, sl += v;
  }
  if (lane == 31) part[0][warp] = st, part[1][warp] = sl;
  __syncthreads();
  int at = st - tokens, tile = sl - tiles, all = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) at += part[0][w], tile += part[1][w];
    all += part[1][w];
  }
  for (int i = n0; i < n1; ++i) {
    const int c = cnt[i];
    for (int k = 0; k < c; k += BM) a.tiles[tile++] = make_int4(i, at + k, min(BM, c - k), 0);
    cnt[i] = at;
    at += c;
  }
  if (threadIdx.x == 0) *a.ntiles = all;
  __syncthreads();
  for (int t0 = 0; t0 < a.T; t0 += kGroupThreads) {
    const int t = t0 + int(threadIdx.x), id = id_of(t), to = take(id);
    if (id >= 0) a.order[to] = t;
  }
}

template <class DT, int BM, int RP>
int launch_one(const LoraArgs &a, int64_t tiles, int C, cudaStream_t st) {
  using P = Plan<BM, RP>;
  auto *k = lora_kernel<DT, BM, RP>;
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

template <class DT, int BM>
int launch_rank(const LoraArgs &a, int64_t tiles, int C, cudaStream_t st) {
  if (a.r <= 16) return launch_one<DT, BM, 16>(a, tiles, C, st);
  if (a.r <= 32) return launch_one<DT, BM, 32>(a, tiles, C, st);
  if (a.r <= 64) return launch_one<DT, BM, 64>(a, tiles, C, st);
  return launch_one<DT, BM, 128>(a, tiles, C, st);
}

// Tokens of a tile, by their number
inline int tile_of(int64_t T) { return T > 1024 ? 64 : 16; }
// Tiles at most
inline int64_t tiles_of(int64_t T, int64_t n) {
  return T <= kInline ? T : std::min(T, n) + T / tile_of(T);
}

}  // namespace

size_t lora_ws_bytes(int64_t T, int64_t n) {
  if (T <= kInline) return 0;
  return 16 + size_t(tiles_of(T, n)) * 16 + size_t(T) * 4;
}

int launch_lora(LoraArgs a, int dtype, void *ws, cudaStream_t st) {
  const int BM = a.T <= kInline ? 16 : tile_of(a.T);
  const int64_t tiles = tiles_of(a.T, a.n);
  if (a.T > kInline) {
    char *p = static_cast<char *>(ws);
    a.ntiles = reinterpret_cast<int *>(p);
    a.tiles = reinterpret_cast<int4 *>(p + 16);
    a.order = reinterpret_cast<int *>(p + 16 + tiles * 16);
    lora_group_kernel<<<1, kGroupThreads, size_t(a.n) * 4, st>>>(a, BM);
    const int rc = launched(1);
    if (rc != WQ_OK) return rc;
  }
  const int C = BM == 16 ? 8 : 4;
  if (dtype == WQ_DT_BF16) return BM == 16 ? launch_rank<Bf16, 16>(a, tiles, C, st) : launch_rank<Bf16, 64>(a, tiles, C, st);
  return BM == 16 ? launch_rank<F16, 16>(a, tiles, C, st) : launch_rank<F16, 64>(a, tiles, C, st);
}

}  // namespace wq
