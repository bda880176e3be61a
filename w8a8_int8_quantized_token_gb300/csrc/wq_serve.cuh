// Element types and vectors shared by the serving kernels (norms, rotary
// positions, paged append, attention).
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "wq_common.cuh"
#include "wq_once.h"
#include "wq_weights_line.h"

namespace wq {

struct Bf16 {
  using Raw = uint16_t;
  static constexpr int kVec = 8;  // elements of a 16-byte access
  static __device__ __forceinline__ float to_f(uint16_t v) { return bf16_to_f(v); }
  static __device__ __forceinline__ uint16_t from_f(float f) { return f_to_bf16(f); }
  static __device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
struct F16 {
  using Raw = uint16_t;
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to_f(uint16_t v) {
    return __half2float(__ushort_as_half(v));
  }
  static __device__ __forceinline__ uint16_t from_f(float f) {
    return __half_as_ushort(__float2half_rn(f));
  }
  static __device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x;
    hi = f.y;
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return f16x2_rn(lo, hi); }
};
struct F32 {
  using Raw = float;
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float to_f(float v) { return v; }
  static __device__ __forceinline__ float from_f(float f) { return f; }
};

// VW consecutive elements as they lie in memory: one 16-byte access
template <class DT, int VW>
struct Vec {
  static_assert(VW == DT::kVec, "one 16-byte access");
  uint4 w;
  static __device__ __forceinline__ Vec load(const typename DT::Raw *p) {
    return {*reinterpret_cast<const uint4 *>(p)};
  }
  __device__ __forceinline__ void store(typename DT::Raw *p) const { *reinterpret_cast<uint4 *>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[VW]) const {
    if constexpr (VW == 8) {
      DT::unpack2(w.x, f[0], f[1]);
      DT::unpack2(w.y, f[2], f[3]);
      DT::unpack2(w.z, f[4], f[5]);
      DT::unpack2(w.w, f[6], f[7]);
    } else {
      f[0] = __uint_as_float(w.x);
      f[1] = __uint_as_float(w.y);
      f[2] = __uint_as_float(w.z);
      f[3] = __uint_as_float(w.w);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[VW]) {
    if constexpr (VW == 8)
      w = make_uint4(DT::pack2(f[0], f[1]), DT::pack2(f[2], f[3]), DT::pack2(f[4], f[5]),
                     DT::pack2(f[6], f[7]));
    else
      w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
  }
};

// Two floats in a register pair, for the packed float32 instructions (each
// lane rounds once).  Kept as one 64-bit value: split into single floats
// between operations, every one of them cost up to four moves.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split(Pair p, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair fma_p(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ Pair mul_p(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair add_p(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---- launchers (host) ----
int device_ok();  // WQ_OK on an sm_103 device

// Lets a kernel have `bytes` of dynamic shared memory on the current device
template <class Kernel>
bool allow_smem(OncePerDevice &once, Kernel *k, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  return once(dev, [&] {
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return true;
    cudaGetLastError();  // told by the return value: no later launch is to report it
    return false;
  });
}

struct BlockNormArgs {
  const void *block, *residual, *gate, *w_post, *b_post, *w_pre, *b_pre;
  int64_t ldb, ldr, ldg, ldx, ldy;
  float scale, eps;
  int post, pre;
  int64_t T;
  int H;
  void *x_out, *y;
  int reach;  // 0: 16-byte pieces, 1: such pieces with rows shifted alike, 2: single elements
};
int launch_block_norm(const BlockNormArgs &a, int dtype, cudaStream_t st);

// One tensor of heads that a rotary launch reads and writes
struct RopeSeg {
  const void *src = nullptr;
  void *dst = nullptr;
  int64_t s_token = 0, s_head = 0;
  int64_t d_token = 0, d_head = 0, d_page = 0;  // d_page: cache segments only
  int heads = 0, D = 0, rot = 0;
  bool paged = false;
};
struct RopeArgs {
  RopeSeg seg[3];
  int nseg;
  const int32_t *positions;
  const int64_t *slots;
  const float *table;
  int64_t max_pos, T, num_slots;
  int page_size, rot, layout;
  float sign;  // -1: inverse
  int32_t *status;
};
// Threads that a token takes pair by pair, and the most that a launch has room for
inline int64_t rope_pair_threads(const RopeArgs &a) {
  int64_t n = 0;
  for (int i = 0; i < a.nseg; ++i) n += int64_t(a.seg[i].heads) * (a.seg[i].D - a.seg[i].rot / 2);
  return n;
}
constexpr int64_t kRopeMostThreads = 65535 * 256;
int launch_rope(const RopeArgs &a, int dtype, bool vec, cudaStream_t st);
// Norms of heads in the same pass: norm[i] says whether segment i has one
struct HeadNormArgs {
  RopeArgs r;
  const void *weight[3];  // [D], nullptr: ones
  bool norm[3];
  float inv_d[3];  // 1 / D
  float eps;
};
int launch_head_norm(const HeadNormArgs &h, int dtype, bool vec, cudaStream_t st);
int launch_rope_table(float *table, int64_t max_pos, int rot, double base, int scaling,
                      double factor, double trained, double beta_fast, double beta_slow,
                      double mscale, cudaStream_t st);

struct AttnArgs {
  const uint16_t *q;
  int64_t q_token, q_head;
  int T, B, max_q, Hq, Hkv, G;
  const int32_t *cu_q;
  const uint16_t *k, *v;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token, num_pages;
  int page_size, dk, dv;
  const int32_t *prefix_pages;
  int P;
  const int32_t *page_table;
  int64_t ld_table;
  const int32_t *suffix_len;
  int max_suffix;
  float scale_log2;  // scale * log2(e)
  uint16_t *out;
  int64_t o_token, o_head;
  float *lse;
  int32_t *status;
  // plan
  int sp, p_chunk;  // prefix: splits and keys of each (0: no prefix)
  int ss, s_chunk;  // suffixes: splits and keys of each
  bool tc_prefix, tc_suffix;  // taken by the tensor-memory kernel
  bool whole;       // it takes prefix and suffix of a sequence's rows in one walk
  bool rest_apart;  // rows of no sequence have a kernel of their own
  bool one_warp;    // blocks of one warp in the kernel for few rows
  int step_pages, step_place;  // from a warp's piece to its next: pages, and places beyond them
  int p_gang, p_gangs, p_stretch;  // its blocks on the prefix: gangs of p_gang, units of a gang
  int slots;        // sp + ss partial results a row
  float *o_part;    // [T][Hq][slots][dv], nullptr when slots == 1
  float *lse_part;  // [T][Hq][slots]
};
void plan_attention(AttnArgs &a);
bool plan_prefix_tiles(AttnArgs &a, int sms);
int launch_attention_tiles(const AttnArgs &a, int dtype, cudaStream_t st);
size_t attention_ws_bytes(const AttnArgs &a);
int launch_attention(const AttnArgs &a, int dtype, cudaStream_t st);

struct WeightArgs : WeightsLine {
  const uint16_t *q;
  int64_t q_token, q_head;
  int Hq, G;
  const uint16_t *k;
  int64_t k_page, k_head, k_token, num_pages;
  int page_size, dk;
  const int32_t *page_table;
  int64_t ld_table;
  float scale_log2, decay;
  const float *lse;  // [T][Hq]
  float *w;
  int64_t w_seq, w_head;
  int32_t *status;
  // plan, beside the line's
  int cols;     // rows of a query tile, in whole 16s
  int box;      // cache rows of one TMA box
  int step_pages, step_place;  // a pair of key tiles on: pages, and places beyond them
  int blocks;   // that share the line of units
  bool tiles;   // the tensor-memory kernel takes it
  bool split;   // a pair of key tiles may be cut between blocks
  float *part;  // [blocks][2][256], nullptr unless split
};
void plan_weights(WeightArgs &a);
size_t weights_ws_bytes(const WeightArgs &a);
int launch_weights(const WeightArgs &a, int dtype, cudaStream_t st);

struct EvictArgs {
  const float *w;
  int64_t w_seq, w_head;
  uint16_t *k, *v;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token, num_pages;
  int page_size, heads, dk, dv, B;
  const int32_t *page_table, *out_table;
  int64_t ld_table, ld_out;
  const int32_t *key_len;
  int max_len, budget, recent, first;
  bool in_place;
  float *w_out;
  int64_t o_seq, o_head;
  int32_t *new_len, *kept;
  int32_t *status;
  int4 *ways;       // [B][heads][budget]: page and place that a row that stays comes from, and goes to
  int32_t *moving;  // sequences with rows to move: their number, then each
  // of the moving kernel: parts of the columns of keys and of values, of the rows
  int k_parts, v_parts, row_blocks;
};
int launch_evict(const EvictArgs &a, bool vec, cudaStream_t st);

constexpr int kLoraTile = 128;  // tokens of a tile where there are many
constexpr int kLoraSlices = 8;  // of the first product's long axis, at most
// 16-bit operands that a float32 element of x A^T is cut into: bf16 has 8 bits,
// so three hold its 24; fp16's two hold 22, counted from a row's largest
constexpr int kLoraMostOperands = 3;
template <class DT>
constexpr int kLoraOperands = std::is_same<DT, F16>::value ? 2 : kLoraMostOperands;
// What is left of v after an operand (of infinity: nothing)
__device__ __forceinline__ float lora_rest(float v, float operand) {
  return fabsf(operand) == INFINITY ? 0.0f : v - operand;
}
struct LoraArgs {
  const uint16_t *x;
  int64_t ldx;
  uint16_t *y;
  int64_t ldy;
  const uint16_t *A, *B;  // [n][r][H], [n][N][r]
  const float *scales;    // [n], nullptr: ones
  const int32_t *ids;     // [T]
  int T, H, N, r, n;
  int32_t *status;
  // tokens in the order of their adapters and the tiles (adapter, first place,
  // tokens), nullptr where each cluster looks for its own
  int *order, *ntiles;
  int4 *tiles;
  // Many tokens: slices of the first product's long axis, and stretches of y's
  // columns; the slices' parts of its result [slices][T][lora_rank(r)], how many
  // of a tile's are there, and the operands that they make, in the order of the tokens
  int slices, stretches;
  int *tickets;        // [tiles]
  float *parts;
  uint32_t *operands;  // [T][kLoraOperands][lora_rank(r) / 2]: high ones first, in pairs
  float *factors;      // [T]
};
int lora_slices(int64_t like);
int lora_rank(int r);
size_t lora_ws_bytes(int64_t T, int64_t n, int r);
int launch_lora_tiles(LoraArgs a, int dtype, int64_t tiles, int64_t like, cudaStream_t st);
int launch_lora(LoraArgs a, int dtype, void *ws, cudaStream_t st);

}  // namespace wq
