// Low-rank adapters for many tokens (tcgen05, sm_103a): a cluster of blocks
// takes 128 tokens of one adapter.
//
//   H = x A^T (128 x r),  y += s H B^T (128 x N)
//
// Each block multiplies its slice of x and A into tensor memory, the blocks'
// parts of H are added through distributed shared memory in the order of the
// blocks, and each block multiplies the sum with its slice of B's rows and adds
// the result to its columns of y, 64 at a time.
//   warps 0-3  H's sum, y: a thread owns a token
//   warps 4-7  copies into one ring of stages: x and A, then B and y; they run
//              ahead into the second product while H is being added
//   warp 8     MMA issue; owns the tensor memory
// H enters the second product from tensor memory as two 16-bit operands, its
// rounding and what that leaves, as in the kernel for few tokens; a token's
// thread holds the whole row, so fp16's factor costs nothing but the maximum.
//
// Tokens of an adapter lie anywhere, so rows of x and y are copied by 16-byte
// pieces (eight lanes a row), which land in the products' swizzled layout.
// Bound by HBM: two blocks share an SM, so that one's sum over the cluster
// passes in the other's copies.
//
// Every wait on a memory barrier is bounded (1 s); on expiry the kernel records
// WQ_ERR_TIMEOUT, waits (bounded) for its own copies and MMAs, frees tensor
// memory and exits; the cluster's barriers are served whatever the waits said.
#include <algorithm>
#include <type_traits>

#include "wq_attn.cuh"
#include "wq_tc.cuh"
#include "wq_warp_mma.cuh"

namespace wq {
namespace {

using namespace tc;

constexpr int BM = 128, KS = 64, NC = 64;  // tokens; elements of x, columns of y a stage
constexpr int THREADS = 288, WARP_COPY = 4, WARP_MMA = 8;
constexpr int MOST_BLOCKS = 8;             // of a cluster

template <int RP>
struct Plan {
  static constexpr int XB = BM * 128, AB = RP * 128;                  // a first product's stage
  static constexpr int BB = (RP + 63) / 64 * NC * 128, YB = BM * 128; // a second one's
  static constexpr int STAGE = XB + AB > BB + YB ? XB + AB : BB + YB;
  static constexpr int NS = RP == 16 ? 4 : 3;
  static constexpr int OFF_P = NS * STAGE;          // [BM][RP] float: parts of H, then its operands
  static constexpr int OFF_UP = OFF_P + BM * RP * 4;  // [BM] float: the rows' factors
  static constexpr int OFF_TOK = OFF_UP + BM * 4;
  static constexpr int OFF_BAR = OFF_TOK + BM * 4;
  static constexpr int B_FULL = 0, B_EMPTY = NS, B_D1 = 2 * NS, B_H = B_D1 + 1, B_D2_FULL = B_H + 1,
                       B_D2_EMPTY = B_D2_FULL + 2, B_DONE = B_D2_EMPTY + 2,
                       B_X = B_DONE + 1,  // [3] the exchange's steps, over the cluster
                       NBAR = B_X + 3;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8, OFF_ABORT = OFF_TMEM + 4;
  static constexpr int SMEM = OFF_ABORT + 4 + 1024;
  static_assert(STAGE % 1024 == 0 && SMEM <= 232448, "shared memory plan");
  // tensor memory: the first product's result, whose place H takes as two
  // operands of RP / 2 columns each; two buffers of the second one's
  static constexpr uint32_t T_H = 0, T_D2 = RP, COLS = 256;
  static_assert(T_D2 + 2 * NC <= COLS, "tensor memory plan");
};

template <class DT>
constexpr uint32_t kTypes = std::is_same<DT, Bf16>::value ? (1u << 7) | (1u << 10) : 0u;

// piece p of 16 bytes of row r in a tile of 128-byte rows
__device__ __forceinline__ uint32_t place(int r, int p) { return uint32_t(r * 128 + ((p ^ (r & 7)) << 4)); }

template <class DT, int RP>
__global__ void __launch_bounds__(THREADS, RP <= 64 ? 2 : 1) lora_tc_kernel(const LoraArgs a) {
  using P = Plan<RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::OFF_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + P::OFF_TMEM);
  int *tok = reinterpret_cast<int *>(sm + P::OFF_TOK);
  auto bar = [&](int i) { return base + P::OFF_BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t csize;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
  const int C = int(csize), rank = int(cluster_ctarank()), tile = int(blockIdx.x) / C;

  attn::wait_last_kernel();  // the list of tiles
  if (tile >= *a.ntiles) return;  // the whole cluster
  const int4 d = a.tiles[tile];
  const int id = d.x, count = d.z;
  for (int i = threadIdx.x; i < count; i += THREADS) tok[i] = a.order[d.y + i];
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < P::NBAR; ++i)
      mbar_init(bar(i), i < P::B_EMPTY ? 128                      // copying threads
                        : i < P::B_D1  ? 5                        // the products, and the tokens' warps
                        : i >= P::B_X  ? 4 * C                      // tokens' warps of the cluster
                        : i == P::B_H || (i >= P::B_D2_EMPTY && i < P::B_DONE) ? 4 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == WARP_MMA) tmem_alloc(smem_u32(tmem_slot), P::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // this block's slices: elements of x, columns of y
  const int steps = (a.H + KS - 1) / KS, s0 = steps * rank / C, n1 = steps * (rank + 1) / C - s0;
  const int chunks = (a.N + NC - 1) / NC, c0 = chunks * rank / C, n2 = chunks * (rank + 1) / C - c0;
  bool ok = true;  // this role's waits all ended in time
  cluster_arrive();  // this block's barriers can be used

  if (warp >= WARP_COPY && warp < WARP_MMA) {
    // -------------------------------------------------------------- copies
    const int t = threadIdx.x - WARP_COPY * 32, row = t / 8, piece = t % 8;  // rows row + 16 j
    const uint32_t to = base + place(row, piece);
    // rows of x and of y (0 elements on from a token's)
    const uint16_t *xs[BM / 16], *ys[BM / 16];
#pragma unroll
    for (int j = 0; j < BM / 16; ++j) {
      const int r = row + 16 * j, k = r < count ? tok[r] : -1;
      xs[j] = k < 0 ? nullptr : a.x + int64_t(k) * a.ldx + s0 * KS + piece * 8;
      ys[j] = k < 0 ? nullptr : a.y + int64_t(k) * a.ldy + c0 * NC + piece * 8;
    }
    const uint16_t *A = a.A + (int64_t(id) * a.r + row) * a.H + s0 * KS + piece * 8;
    const uint16_t *B = a.B + (int64_t(id) * a.N + c0 * NC + row) * a.r + piece * 8;
    uint32_t slot = 0, par = 1;
#pragma unroll 1
    for (int g = 0; g < n1 + n2; ++g) {
      if (!(ok = wait_warp(bar(P::B_EMPTY) + 8 * slot, par, abort_flag))) break;
      const uint32_t at = to + slot * P::STAGE;
      if (g < n1) {
        const bool in = (s0 + g) * KS + piece * 8 < a.H;
#pragma unroll
        for (int j = 0; j < BM / 16; ++j) {
          const bool on = in && xs[j];
          cp16(at + j * 16 * 128, on ? xs[j] + g * KS : a.x, on);
        }
#pragma unroll
        for (int j = 0; j < RP / 16; ++j) {
          const bool on = in && row + 16 * j < a.r;
          cp16(at + P::XB + j * 16 * 128, on ? A + int64_t(16 * j) * a.H + g * KS : a.A, on);
        }
      } else {
        const int c = g - n1;  // from c0 on
        const bool in = (c0 + c) * NC + piece * 8 < a.N;
#pragma unroll
        for (int j = 0; j < NC / 16; ++j) {
          const bool on = (c0 + c) * NC + row + 16 * j < a.N;
#pragma unroll
          for (int p = 0; p < (RP + 63) / 64; ++p) {
            const bool has = on && p * 64 + piece * 8 < a.r;
            if (RP >= 64 || piece * 8 < RP)
              cp16(at + p * NC * 128 + j * 16 * 128,
                   has ? B + (int64_t(c) * NC + 16 * j) * a.r + p * 64 : a.B, has);
          }
        }
#pragma unroll
        for (int j = 0; j < BM / 16; ++j) {
          const bool on = in && ys[j];
          cp16(at + P::BB + j * 16 * 128, on ? ys[j] + c * NC : a.y, on);
        }
      }
      // arrives once this thread's copies so far are in
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(P::B_FULL) + 8 * slot) : "memory");
      if (++slot == P::NS) slot = 0, par ^= 1;
    }
    if (!ok) *abort_flag = 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    cluster_wait();
  } else if (warp == WARP_MMA) {
    // -------------------------------------------------------------- products
    if (elect_one()) {
      auto wait = [&](uint32_t b, uint32_t parity) {
        if (ok) ok = wait_one(b, parity, abort_flag);
      };
      const uint32_t id1 = idesc_f16(BM, RP) | kTypes<DT>, id2 = idesc_f16(BM, NC) | kTypes<DT>;
      const int ks = (a.r + 15) / 16;  // steps of the second product
      uint32_t slot = 0, par = 0;
#pragma unroll 1
      for (int g = 0; g < n1 && ok; ++g) {
        wait(bar(P::B_FULL) + 8 * slot, par);
        fence_async_smem();  // the copies are ordinary writes, which the products are to read
        tc_fence_after();
        if (ok) {
          const uint64_t dx = sdesc(base + slot * P::STAGE), da = sdesc(base + slot * P::STAGE + P::XB);
#pragma unroll
          for (int i = 0; i < KS / 16; ++i) mma_f16(tmem, dx + 2 * i, da + 2 * i, id1, g | i ? 1u : 0u);
          for (int i = 0; i < 4; ++i) mbar_arrive(bar(P::B_EMPTY) + 8 * slot);  // for the tokens' warps
          mma_commit(bar(P::B_EMPTY) + 8 * slot);
        }
        if (++slot == P::NS) slot = 0, par ^= 1;
      }
      if (ok) mma_commit(bar(P::B_D1));
      if (n2 > 0) wait(bar(P::B_H), 0);
#pragma unroll 1
      for (int c = 0; c < n2 && ok; ++c) {
        const uint32_t buf = c & 1;
        wait(bar(P::B_FULL) + 8 * slot, par);
        fence_async_smem();
        wait(bar(P::B_D2_EMPTY) + 8 * buf, ((c >> 1) & 1) ^ 1);
        tc_fence_after();
        if (ok) {
          const uint64_t db = sdesc(base + slot * P::STAGE);
          const uint32_t to = tmem + P::T_D2 + buf * NC;
          for (int i = 0; i < ks; ++i) {
            const uint64_t b = db + ((i / 4) * (NC * 128) + (i % 4) * 32 >> 4);
            mma_f16_ts(to, tmem + P::T_H + 8 * i, b, id2, i ? 1u : 0u);
            mma_f16_ts(to, tmem + P::T_H + RP / 2 + 8 * i, b, id2, 1u);
          }
          mma_commit(bar(P::B_EMPTY) + 8 * slot);
          mma_commit(bar(P::B_D2_FULL) + 8 * buf);
        }
        if (++slot == P::NS) slot = 0, par ^= 1;
      }
      if (!ok) *abort_flag = 1;
      mma_commit(bar(P::B_DONE));
      mbar_wait_bounded(bar(P::B_DONE), 0);
    }
    __syncwarp();
    cluster_wait();
  } else {
    // -------------------------------------------------------------- tokens
    const int r = threadIdx.x;  // the token of this thread
    const uint32_t mine = tmem + (uint32_t(warp * 32) << 16);
    // H's sum: each block adds up the parts of 128 / C rows, which the blocks
    // have put into its memory, and gives every block the operands they make.
    // (Were every block to fetch all parts, the sum alone took 27 us for 8.)
    constexpr int Q = RP / 4;  // 16-byte pieces of a row, parts or operands
    const int share = BM / C;  // rows
    auto at = [](int row, int q) { return P::OFF_P + uint32_t(row * (RP * 4) + ((q ^ (row & (Q < 8 ? Q - 1 : 7))) << 4)); };
    // a step's end: all that the cluster's warps have written before it is there
    auto step = [&](int i) {
      __syncwarp();
      if (lane == 0)
        for (int c = 0; c < C; ++c) mbar_arrive_cluster(mapa(bar(P::B_X + i), uint32_t(c)));
      if (ok) ok = mbar_wait_cluster(bar(P::B_X + i), 0, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
    };
    if (n1 > 0) {
      ok = wait_warp(bar(P::B_D1), 0, abort_flag);
      tc_fence_after();
    }
    cluster_wait();  // the others' barriers can be used
    {
      const uint32_t owner = uint32_t(r / share);
      const int row = rank * share + r % share;  // of the owner's place: block by block
#pragma unroll
      for (int i = 0; i < RP; i += 16) {
        uint32_t v[16];
        tmem_ld16(mine + i, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(v[e]));
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = n1 > 0 ? v[e] : 0u;
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          st_cluster_v4(mapa(base + at(row, (i + e) / 4), owner), v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    step(0);
    const float scale = a.scales ? a.scales[id] : 1.0f;
    // units of a row's piece: at most (128 / C) Q of them, all threads in step
    uint32_t hi[Q][2], lo[Q][2];
    float up_row[Q];
    const int units = (share * Q + BM - 1) / BM;  // of a thread, a row's pieces in neighbouring lanes
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (i >= units) break;
      const int u = min(i * BM + r, share * Q - Q + r % Q), row = u / Q, q = u % Q;
      float4 v = *reinterpret_cast<const float4 *>(sm + at(row, q));
      for (int c = 1; c < C; ++c) {
        const float4 w = *reinterpret_cast<const float4 *>(sm + at(c * share + row, q));
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      float f = 1.0f;  // the row's factor
      if constexpr (std::is_same<DT, F16>::value) {
        float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
        for (int o = Q / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^-e with the row's largest in [2^e, 2^(e+1)), e within float's normal range
        const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -126), 126);
        const float down = __uint_as_float(uint32_t(127 - e) << 23);
        f = __uint_as_float(uint32_t(127 + e) << 23);
        v.x *= down;
        v.y *= down;
        v.z *= down;
        v.w *= down;
      }
      up_row[i] = scale * f;
      auto low = [](float x, float h) { return fabsf(h) == INFINITY ? 0.0f : x - h; };
      float x, y;
      hi[i][0] = DT::pack2(v.x, v.y);
      DT::unpack2(hi[i][0], x, y);
      lo[i][0] = DT::pack2(low(v.x, x), low(v.y, y));
      hi[i][1] = DT::pack2(v.z, v.w);
      DT::unpack2(hi[i][1], x, y);
      lo[i][1] = DT::pack2(low(v.z, x), low(v.w, y));
    }
    step(1);  // the parts are read: their place is the operands' now
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (i >= units) break;
      const int u = i * BM + r, row = rank * share + u / Q, q = u % Q;
      if (u >= share * Q) break;
      for (int c = 0; c < C; ++c) {
        const uint32_t to_hi = base + at(row, q / 2) + (q & 1) * 8, to_lo = base + at(row, Q / 2 + q / 2) + (q & 1) * 8;
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(mapa(to_hi, uint32_t(c))), "r"(hi[i][0]), "r"(hi[i][1]) : "memory");
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(mapa(to_lo, uint32_t(c))), "r"(lo[i][0]), "r"(lo[i][1]) : "memory");
        if (q == 0)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(mapa(base + P::OFF_UP + row * 4, uint32_t(c))), "f"(up_row[i]) : "memory");
      }
    }
    step(2);
    const float up = *reinterpret_cast<const float *>(sm + P::OFF_UP + r * 4);
#pragma unroll
    for (int i = 0; i < Q; i += 4) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 x = *reinterpret_cast<const uint4 *>(sm + at(r, i + e));
        w[4 * e] = x.x;
        w[4 * e + 1] = x.y;
        w[4 * e + 2] = x.z;
        w[4 * e + 3] = x.w;
      }
      tmem_st16(mine + P::T_H + 4 * i, w);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(P::B_H));
    // where a lane's pieces of the warp's rows go: eight lanes a row, rows 4 i + lane / 8
    uint16_t *rows[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = warp * 32 + 4 * i + lane / 8;
      rows[i] = q < count ? a.y + int64_t(tok[q]) * a.ldy + c0 * NC + (lane & 7) * 8 : nullptr;
    }
    using V = Vec<DT, 8>;
#pragma unroll 1
    for (int c = 0; c < n2 && ok; ++c) {
      const int g = n1 + c;
      const uint32_t slot = uint32_t(g) % P::NS, buf = c & 1;
      ok = wait_warp(bar(P::B_FULL) + 8 * slot, (uint32_t(g) / P::NS) & 1, abort_flag) &&
           wait_warp(bar(P::B_D2_FULL) + 8 * buf, (c >> 1) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      uint8_t *ty = sm + slot * P::STAGE + P::BB;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[32];
        tmem_ld32(mine + P::T_D2 + buf * NC + 32 * half, v);
        wait_ld32(v);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          V y{*reinterpret_cast<const uint4 *>(ty + place(r, 4 * half + p))};
          float f[8];
          y.get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __fmaf_rn(__uint_as_float(v[8 * p + e]), up, f[e]);
          y.set(f);
          *reinterpret_cast<uint4 *>(ty + place(r, 4 * half + p)) = y.w;
        }
      }
      tc_fence_before();
      __syncwarp();  // the warp's rows are written
      if (lane == 0) mbar_arrive(bar(P::B_D2_EMPTY) + 8 * buf);
      const bool in = (c0 + c) * NC + (lane & 7) * 8 < a.N;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 w = *reinterpret_cast<const uint4 *>(ty + place(warp * 32 + 4 * i + lane / 8, lane & 7));
        if (in && rows[i]) *reinterpret_cast<uint4 *>(rows[i] + c * NC) = w;
      }
      __syncwarp();  // and read
      if (lane == 0) mbar_arrive(bar(P::B_EMPTY) + 8 * slot);
    }
    if (!ok) *abort_flag = 1;
  }
  if (!ok) {
    *abort_flag = 1;
    set_status(a.status, WQ_ERR_TIMEOUT);
  }
  __syncthreads();
  if (warp == WARP_MMA) tmem_dealloc(tmem, P::COLS);
  cluster_sync();  // no block ends while another may write to it
}

template <class DT, int RP>
int launch_one(const LoraArgs &a, int64_t tiles, int C, cudaStream_t st) {
  using P = Plan<RP>;
  auto *k = lora_tc_kernel<DT, RP>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, P::SMEM)) return WQ_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(tiles * C));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = size_t(P::SMEM);
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(C);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
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

}  // namespace

// tiles: at most so many tiles of 128 tokens in a.tiles
int launch_lora_tiles(const LoraArgs &a, int dtype, int64_t tiles, cudaStream_t st) {
  // Blocks of a tile: as many as let about all tiles run at the same time
  // (some may not be there)
  const int slots = (a.r <= 64 ? 2 : 1) * 152;
  int C = MOST_BLOCKS;
  while (C > 1 && tiles * C > slots * 9 / 8) C /= 2;
  return dtype == WQ_DT_BF16 ? launch_rank<Bf16>(a, tiles, C, st) : launch_rank<F16>(a, tiles, C, st);
}

}  // namespace wq
