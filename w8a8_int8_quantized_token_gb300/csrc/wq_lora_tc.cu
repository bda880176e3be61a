// Low-rank adapters for many tokens (tcgen05, sm_103a), 128 of one adapter a
// tile, in two kernels:
//
//   lora_down_kernel  H = x A^T (128 x r), the long axis cut into slices, whose
//                     parts go to the workspace in float32; the last block of a
//                     tile adds them, in the order of the slices
//   lora_up_kernel    y += s H B^T (128 x N), a stretch of columns a block, 64 at a
//                     time
//
// One kernel for both, whose blocks shared a tile in a cluster and added the
// parts through distributed shared memory, took 89 us at 8192 tokens of width
// 7168 and rank 64: the sum held each block up for 10 us.
//
// Blocks have warps that copy, one that issues the products, and warps that own
// a token a thread.  Tokens of an adapter lie anywhere, so rows of x and y are
// copied by 16-byte pieces (eight lanes a row), which land in the products'
// swizzled layout.  H enters the second product from tensor memory as 16-bit
// operands, its rounding and what that leaves, as in the kernel for few tokens.
// Bound by HBM: x once, y twice; the adapters come from L2.  8192 tokens of width
// 7168 and rank 64 take 90 us (3.9 TB/s), the list of tiles among them (7); two
// bf16 operands in place of three took 85, and 0.2% of y's elements then rounded
// otherwise than from a float32 H.  With cold caches and 4096 tokens 29 us (2.0
// TB/s of x: the parts' sum and the start are as long as the steps) and 34 (3.5 TB/s
// of y).
//
// Every wait on a memory barrier is bounded (1 s); on expiry the kernel records
// WQ_ERR_TIMEOUT, waits (bounded) for its own copies and MMAs, frees tensor
// memory and exits.
#include <algorithm>
#include <type_traits>

#include "wq_attn.cuh"
#include "wq_tc.cuh"
#include "wq_warp_mma.cuh"

namespace wq {
namespace {

using namespace tc;

constexpr int BM = kLoraTile, KS = 64, NC = 64;  // tokens; elements of x, columns of y a stage
constexpr int RING = 110 * 1024;           // bytes of a block's stages, at most: two blocks share an SM

template <class DT>
constexpr uint32_t kTypes = std::is_same<DT, Bf16>::value ? (1u << 7) | (1u << 10) : 0u;

// piece p of 16 bytes of row r in a tile of 128-byte rows
__device__ __forceinline__ uint32_t place(int r, int p) { return uint32_t(r * 128 + ((p ^ (r & 7)) << 4)); }

// Barriers of a ring of stages, and what follows them in shared memory
template <int NS, int MORE>
struct Bars {
  static constexpr int FULL = 0, EMPTY = NS, REST = 2 * NS, N = REST + MORE;
};

// A thread's arrival on a barrier once its copies so far are in
__device__ __forceinline__ void arrive_copied(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------ H's parts
template <int RP>
struct Down {
  static constexpr int THREADS = 160, WARP_MMA = 4;  // warps 0-3 copy, then write the result
  static constexpr int XB = BM * 128, STAGE = XB + RP * 128;
  static constexpr int NS = RING / STAGE < 6 ? RING / STAGE : 6;
  using B = Bars<NS, 1>;
  static constexpr int DONE = B::REST;
  static constexpr int OFF_TOK = NS * STAGE, OFF_BAR = OFF_TOK + BM * 4, OFF_TMEM = OFF_BAR + B::N * 8,
                       OFF_ABORT = OFF_TMEM + 4, SMEM = OFF_ABORT + 4 + 1024;
  // A product's sum loses what lies below the last bit of what it is added to,
  // always towards zero; stages take turns among several sums, which makes those
  // chains a quarter (rank 128: half) as long.
  static constexpr int SUMS = RP < 128 ? 4 : 2;
  static constexpr uint32_t COLS = SUMS * RP;
};

template <class DT, int RP>
__global__ void __launch_bounds__(Down<RP>::THREADS, 2) lora_down_kernel(const LoraArgs a) {
  using P = Down<RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::OFF_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + P::OFF_TMEM);
  int *tok = reinterpret_cast<int *>(sm + P::OFF_TOK);
  auto bar = [&](int i) { return base + P::OFF_BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = int(blockIdx.x) / a.slices, slice = int(blockIdx.x) - tile * a.slices;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < P::B::N; ++i) mbar_init(bar(i), i < P::B::EMPTY ? 128 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  attn::wait_last_kernel();  // the list of tiles; in every block
  attn::start_next_kernel();  // which may then rely on the list too
  if (tile >= *a.ntiles) return;
  const int4 d = a.tiles[tile];
  const int id = d.x, count = d.z;
  for (int i = threadIdx.x; i < count; i += P::THREADS) tok[i] = a.order[d.y + i];
  if (warp == P::WARP_MMA) tmem_alloc(smem_u32(tmem_slot), P::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int steps = (a.H + KS - 1) / KS, s0 = steps * slice / a.slices, n = steps * (slice + 1) / a.slices - s0;
  bool ok = true;  // this role's waits all ended in time

  if (warp < P::WARP_MMA) {
    const int row = threadIdx.x / 8, piece = threadIdx.x % 8;  // rows row + 16 j
    const uint32_t to = base + place(row, piece);
    const uint16_t *xs[BM / 16];
#pragma unroll
    for (int j = 0; j < BM / 16; ++j) {
      const int r = row + 16 * j;
      xs[j] = r < count ? a.x + int64_t(tok[r]) * a.ldx + s0 * KS + piece * 8 : nullptr;
    }
    const uint16_t *A = a.A + (int64_t(id) * a.r + row) * a.H + s0 * KS + piece * 8;
    uint32_t slot = 0, par = 1;
#pragma unroll 1
    for (int g = 0; g < n; ++g) {
      if (!(ok = wait_warp(bar(P::B::EMPTY) + 8 * slot, par, abort_flag))) break;
      const uint32_t at = to + slot * P::STAGE;
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
      arrive_copied(bar(P::B::FULL) + 8 * slot);
      if (++slot == P::NS) slot = 0, par ^= 1;
    }
    if (!ok) *abort_flag = 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
    // ---- the result: a thread owns a token
    if (ok) ok = wait_warp(bar(P::DONE), 0, abort_flag);
    tc_fence_after();
    const int r = threadIdx.x;
    float *h = a.parts + (int64_t(slice) * a.T + d.y + r) * RP;
#pragma unroll
    for (int i = 0; i < RP; i += 16) {
      uint32_t v[P::SUMS][16];
#pragma unroll
      for (int s = 0; s < P::SUMS; ++s) tmem_ld16(tmem + (uint32_t(warp * 32) << 16) + s * RP + i, v[s]);
      tmem_wait_ld();
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = 0.0f;
#pragma unroll
      for (int s = 0; s < P::SUMS; ++s) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          asm volatile("" : "+r"(v[s][e]));
          if (s < n) f[e] += __uint_as_float(v[s][e]);  // no stage added to the others
        }
      }
      if (r < count) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)  // past the rank nothing counts: an infinite x makes NaN of the padding's zeros
          *reinterpret_cast<float4 *>(h + i + e) =
              i + e < a.r ? make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
    tc_fence_before();
    // ---- the tile's last block adds the parts, in the order of the slices
    __threadfence();
    named_sync(1, 128);
    if (threadIdx.x == 0) tok[0] = atomicAdd(&a.tickets[tile], 1);
    named_sync(1, 128);
    if (tok[0] == a.slices - 1) {
      __threadfence();
      constexpr int Q = RP / 4;  // 16-byte pieces of a row, in neighbouring lanes
      const float scale = a.scales ? a.scales[id] : 1.0f;
      constexpr int U = 4;  // units whose loads are in flight together
#pragma unroll 1
      for (int u0 = r; u0 < BM * Q; u0 += U * 128) {
        float4 w[U][kLoraSlices];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int u = u0 + k * 128, row = d.y + min(u / Q, count - 1);
          const float4 *from = reinterpret_cast<const float4 *>(a.parts + int64_t(row) * RP) + u % Q;
#pragma unroll
          for (int c = 0; c < kLoraSlices; ++c)
            if (c < a.slices) w[k][c] = __ldcg(from + int64_t(c) * a.T * Q);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int u = u0 + k * 128, q = u % Q;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < kLoraSlices; ++c) {
            if (c >= a.slices) break;
            v.x += w[k][c].x;
            v.y += w[k][c].y;
            v.z += w[k][c].z;
            v.w += w[k][c].w;
          }
          float up = scale;
          if constexpr (std::is_same<DT, F16>::value) {
            float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
            for (int o = Q / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // 2^-e with the row's largest in [2^e, 2^(e+1)), e within float's normal range
            const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -126), 126);
            const float down = __uint_as_float(uint32_t(127 - e) << 23);
            up *= __uint_as_float(uint32_t(127 + e) << 23);
            v.x *= down;
            v.y *= down;
            v.z *= down;
            v.w *= down;
          }
          if (u / Q < count) {
            constexpr int OPS = kLoraOperands<DT>;
            uint2 *to = reinterpret_cast<uint2 *>(a.operands + int64_t(d.y + u / Q) * (OPS * RP / 2));
#pragma unroll
            for (int o = 0; o < OPS; ++o) {
              const uint2 w = make_uint2(DT::pack2(v.x, v.y), DT::pack2(v.z, v.w));
              to[o * Q + q] = w;
              float x0, x1, x2, x3;
              DT::unpack2(w.x, x0, x1);
              DT::unpack2(w.y, x2, x3);
              v = make_float4(lora_rest(v.x, x0), lora_rest(v.y, x1), lora_rest(v.z, x2), lora_rest(v.w, x3));
            }
            if (q == 0) a.factors[d.y + u / Q] = up;
          }
        }
      }
    }
  } else {
    if (elect_one()) {
      const uint32_t idesc = idesc_f16(BM, RP) | kTypes<DT>;
      uint32_t slot = 0, par = 0;
#pragma unroll 1
      for (int g = 0; g < n && ok; ++g) {
        ok = wait_one(bar(P::B::FULL) + 8 * slot, par, abort_flag);
        fence_async_smem();  // the copies are ordinary writes, which the products are to read
        tc_fence_after();
        if (ok) {
          const uint64_t dx = sdesc(base + slot * P::STAGE), da = sdesc(base + slot * P::STAGE + P::XB);
#pragma unroll
          for (int i = 0; i < KS / 16; ++i)
            mma_f16(tmem + g % P::SUMS * RP, dx + 2 * i, da + 2 * i, idesc, g >= P::SUMS || i ? 1u : 0u);
          mma_commit(bar(P::B::EMPTY) + 8 * slot);
        }
        if (++slot == P::NS) slot = 0, par ^= 1;
      }
      if (!ok) *abort_flag = 1;
      mma_commit(bar(P::DONE));
      mbar_wait_bounded(bar(P::DONE), 0);
    }
    __syncwarp();
  }
  if (!ok) set_status(a.status, WQ_ERR_TIMEOUT);
  __syncthreads();
  if (warp == P::WARP_MMA) tmem_dealloc(tmem, P::COLS);
}

// ------------------------------------------------------------------ y
template <class DT, int RP>
struct Up {
  // warps 0-7 own tokens (two threads a token, 32 columns each), 8-11 copy
  static constexpr int THREADS = 416, WARP_COPY = 8, WARP_MMA = 12;
  static constexpr int BB = (RP + 63) / 64 * NC * 128, YB = BM * 128, STAGE = BB + YB;
  static constexpr int NS = RING / STAGE;
  using B = Bars<NS, 6>;
  static constexpr int H = B::REST, D_FULL = H + 1, D_EMPTY = D_FULL + 2, DONE = D_EMPTY + 2;
  static constexpr int OFF_TOK = NS * STAGE, OFF_BAR = OFF_TOK + BM * 4,
                       OFF_TMEM = OFF_BAR + B::N * 8, OFF_ABORT = OFF_TMEM + 4, SMEM = OFF_ABORT + 4 + 1024;
  // tensor memory: H's operands, RP / 2 columns each, and buffers of 64 columns of
  // the result, one where three operands of rank 128 leave no more room
  static constexpr int OPS = kLoraOperands<DT>;
  static constexpr uint32_t T_D = (OPS * RP / 2 + 31) / 32 * 32, COLS = 256, ND = T_D + 2 * NC <= COLS ? 2 : 1;
  static_assert(T_D + ND * NC <= COLS, "tensor memory plan");
};

template <class DT, int RP>
__global__ void __launch_bounds__(Up<DT, RP>::THREADS, 2) lora_up_kernel(const LoraArgs a) {
  using P = Up<DT, RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *sm = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + P::OFF_ABORT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + P::OFF_TMEM);
  int *tok = reinterpret_cast<int *>(sm + P::OFF_TOK);
  auto bar = [&](int i) { return base + P::OFF_BAR + 8u * uint32_t(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = int(blockIdx.x) / a.stretches, stretch = int(blockIdx.x) - tile * a.stretches;

  // The list of tiles is there: the kernel before let this one start when it had
  // waited for it.  Only H is not, so y and B are on their way before it is.
  if (tile >= *a.ntiles) {
    attn::wait_last_kernel();  // in every block: what follows this kernel may rely on the one before
    return;
  }
  const int4 d = a.tiles[tile];
  const int id = d.x, count = d.z;
  for (int i = threadIdx.x; i < count; i += P::THREADS) tok[i] = a.order[d.y + i];
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < P::B::N; ++i)
      mbar_init(bar(i), i < P::B::EMPTY  ? 128  // copying threads
                        : i < P::B::REST ? 9    // the products, and the tokens' warps
                        : i == P::H || (i >= P::D_EMPTY && i < P::DONE) ? 8 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == P::WARP_MMA) tmem_alloc(smem_u32(tmem_slot), P::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int chunks = (a.N + NC - 1) / NC, c0 = chunks * stretch / a.stretches, n = chunks * (stretch + 1) / a.stretches - c0;
  bool ok = true;  // this role's waits all ended in time

  if (warp >= P::WARP_COPY && warp < P::WARP_MMA) {
    const int t = threadIdx.x - P::WARP_COPY * 32, row = t / 8, piece = t % 8;  // rows row + 16 j
    const uint32_t to = base + place(row, piece);
    const uint16_t *ys[BM / 16];
#pragma unroll
    for (int j = 0; j < BM / 16; ++j) {
      const int r = row + 16 * j;
      ys[j] = r < count ? a.y + int64_t(tok[r]) * a.ldy + c0 * NC + piece * 8 : nullptr;
    }
    const uint16_t *B = a.B + (int64_t(id) * a.N + c0 * NC + row) * a.r + piece * 8;
    uint32_t slot = 0, par = 1;
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
      if (!(ok = wait_warp(bar(P::B::EMPTY) + 8 * slot, par, abort_flag))) break;
      const uint32_t at = to + slot * P::STAGE;
      const bool in = (c0 + c) * NC + piece * 8 < a.N;
#pragma unroll
      for (int j = 0; j < BM / 16; ++j) {
        const bool on = in && ys[j];
        cp16(at + P::BB + j * 16 * 128, on ? ys[j] + c * NC : a.y, on);
      }
#pragma unroll
      for (int j = 0; j < NC / 16; ++j) {
        const bool on = (c0 + c) * NC + row + 16 * j < a.N;
#pragma unroll
        for (int p = 0; p < (RP + 63) / 64; ++p) {
          const bool has = on && p * 64 + piece * 8 < a.r;
          if (RP >= 64 || piece * 8 < RP)
            cp16(at + p * NC * 128 + j * 16 * 128, has ? B + (int64_t(c) * NC + 16 * j) * a.r + p * 64 : a.B, has);
        }
      }
      arrive_copied(bar(P::B::FULL) + 8 * slot);
      if (++slot == P::NS) slot = 0, par ^= 1;
    }
    if (!ok) *abort_flag = 1;
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == P::WARP_MMA) {
    if (elect_one()) {
      auto wait = [&](uint32_t b, uint32_t parity) {
        if (ok) ok = wait_one(b, parity, abort_flag);
      };
      const uint32_t idesc = idesc_f16(BM, NC) | kTypes<DT>;
      const int ks = (a.r + 15) / 16;
      uint32_t slot = 0, par = 0;
      wait(bar(P::H), 0);
#pragma unroll 1
      for (int c = 0; c < n && ok; ++c) {
        const uint32_t buf = c % P::ND;
        wait(bar(P::B::FULL) + 8 * slot, par);
        fence_async_smem();  // the copies are ordinary writes, which the products are to read
        wait(bar(P::D_EMPTY) + 8 * buf, ((c / P::ND) & 1) ^ 1);
        tc_fence_after();
        if (ok) {
          const uint64_t db = sdesc(base + slot * P::STAGE);
          const uint32_t to = tmem + P::T_D + buf * NC;
          for (int i = 0; i < ks; ++i) {
            const uint64_t b = db + (((i / 4) * (NC * 128) + (i % 4) * 32) >> 4);
#pragma unroll
            for (int o = 0; o < P::OPS; ++o) mma_f16_ts(to, tmem + o * (RP / 2) + 8 * i, b, idesc, i | o ? 1u : 0u);
          }
          mma_commit(bar(P::B::EMPTY) + 8 * slot);
          mma_commit(bar(P::D_FULL) + 8 * buf);
        }
        if (++slot == P::NS) slot = 0, par ^= 1;
      }
      if (!ok) *abort_flag = 1;
      mma_commit(bar(P::DONE));
      mbar_wait_bounded(bar(P::DONE), 0);
    }
    __syncwarp();
  } else {
    const int r = threadIdx.x & 127, half = warp >> 2;  // token, columns 32 half ..
    const uint32_t mine = tmem + (uint32_t((warp & 3) * 32) << 16);
    // ---- H's operands of this token, 16 elements a group: even groups by one thread, odd ones by the other
    attn::wait_last_kernel();
    const int64_t at_row = int64_t(d.y) + min(r, count - 1);
    constexpr int GROUPS = P::OPS * RP / 16, AT_ONCE = 6;  // loads in flight: 48 registers
    const uint4 *from = reinterpret_cast<const uint4 *>(a.operands + at_row * (P::OPS * RP / 2));
    const float up = a.factors[at_row];
#pragma unroll
    for (int g0 = 0; g0 < GROUPS; g0 += 2 * AT_ONCE) {
      uint4 w[AT_ONCE][2];
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int g = g0 + 2 * i + half;
        if (g < GROUPS) w[i][0] = from[2 * g], w[i][1] = from[2 * g + 1];
      }
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) {
        const int g = g0 + 2 * i + half;
        if (g >= GROUPS) break;  // the same for the whole warp
        const uint32_t x[8] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w, w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
        tmem_st8(mine + 8 * g, x);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(P::H));
    // where a lane's pieces of the warp's rows go: four lanes a row, rows 8 i + lane / 4
    uint16_t *rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = (warp & 3) * 32 + 8 * i + lane / 4;
      rows[i] = q < count ? a.y + int64_t(tok[q]) * a.ldy + c0 * NC + half * 32 + (lane & 3) * 8 : nullptr;
    }
    using V = Vec<DT, 8>;
    uint32_t slot = 0, par = 0;
#pragma unroll 1
    for (int c = 0; c < n && ok; ++c) {
      const uint32_t buf = c % P::ND;
      ok = wait_warp(bar(P::B::FULL) + 8 * slot, par, abort_flag) &&
           wait_warp(bar(P::D_FULL) + 8 * buf, (c / P::ND) & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      uint8_t *ty = sm + slot * P::STAGE + P::BB;
      uint32_t v[32];
      tmem_ld32(mine + P::T_D + buf * NC + 32 * half, v);
      V y[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) y[p].w = *reinterpret_cast<const uint4 *>(ty + place(r, 4 * half + p));
      wait_ld32(v);
      tc_fence_before();
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float f[8];
        y[p].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fmaf_rn(__uint_as_float(v[8 * p + e]), up, f[e]);
        y[p].set(f);
        *reinterpret_cast<uint4 *>(ty + place(r, 4 * half + p)) = y[p].w;
      }
      __syncwarp();  // the warp's rows are written
      if (lane == 0) mbar_arrive(bar(P::D_EMPTY) + 8 * buf);
      const bool in = (c0 + c) * NC + half * 32 + (lane & 3) * 8 < a.N;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = *reinterpret_cast<const uint4 *>(ty + place((warp & 3) * 32 + 8 * i + lane / 4, 4 * half + (lane & 3)));
        if (in && rows[i]) *reinterpret_cast<uint4 *>(rows[i] + c * NC) = w;
      }
      __syncwarp();  // and read
      if (lane == 0) mbar_arrive(bar(P::B::EMPTY) + 8 * slot);
      if (++slot == P::NS) slot = 0, par ^= 1;
    }
    if (!ok) *abort_flag = 1;
  }
  if (!ok) set_status(a.status, WQ_ERR_TIMEOUT);
  __syncthreads();
  if (warp == P::WARP_MMA) tmem_dealloc(tmem, P::COLS);
}

template <class DT, int RP>
int launch_one(const LoraArgs &a, int64_t tiles, cudaStream_t st) {
  // lora_up_kernel's blocks may be there before lora_down_kernel's have their
  // tensor memory, and wait for those: no SM holds two of the first and one of
  // the second, so that there is always some left.
  using U = Up<DT, RP>;
  static_assert(2 * U::SMEM + Down<RP>::SMEM > 228 * 1024 && U::COLS + Down<RP>::COLS <= 512,
                "tensor memory of blocks that share an SM");
  auto *down = lora_down_kernel<DT, RP>;
  auto *up = lora_up_kernel<DT, RP>;
  static OncePerDevice sized, sized_up;
  if (!allow_smem(sized, down, Down<RP>::SMEM) || !allow_smem(sized_up, up, U::SMEM)) return WQ_ERR_LAUNCH;
  const int rc = attn::launch_chained(down, unsigned(tiles * a.slices), Down<RP>::THREADS, Down<RP>::SMEM, true, st, a);
  return rc != WQ_OK ? rc
                     : attn::launch_chained(up, unsigned(tiles * a.stretches), U::THREADS, U::SMEM, true, st, a);
}

template <class DT>
int launch_rank(const LoraArgs &a, int64_t tiles, cudaStream_t st) {
  if (a.r <= 16) return launch_one<DT, 16>(a, tiles, st);
  if (a.r <= 32) return launch_one<DT, 32>(a, tiles, st);
  if (a.r <= 64) return launch_one<DT, 64>(a, tiles, st);
  return launch_one<DT, 128>(a, tiles, st);
}

}  // namespace

// Slices and stretches of a tile: as many as let about all tiles, of which there
// are likely `like`, run at the same time, two blocks an SM
int lora_slices(int64_t like) { return int(std::max<int64_t>(1, std::min<int64_t>(kLoraSlices, 2 * 152 / like))); }

// The rank in shared memory and in the workspace
int lora_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

int launch_lora_tiles(LoraArgs a, int dtype, int64_t tiles, int64_t like, cudaStream_t st) {
  a.slices = lora_slices(like);
  a.stretches = int(std::max<int64_t>(1, std::min<int64_t>((a.N + NC - 1) / NC, 2 * 152 / like)));
  if (tiles * std::max(a.slices, a.stretches) >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  return dtype == WQ_DT_BF16 ? launch_rank<Bf16>(a, tiles, st) : launch_rank<F16>(a, tiles, st);
}

}  // namespace wq
