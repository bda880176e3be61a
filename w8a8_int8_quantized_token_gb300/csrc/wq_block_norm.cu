// Norms after and before a block, fused with the gate, the residual scale and
// the residual sum:
//   h = residual + scale * (gate * N_post(block)),  x_out = h,  y = N_pre(h)
//
// A row stays in registers from its one load to its stores: block, residual
// and gate are read once, both outputs written once, and the two norms (the
// second needs the whole of h) cost two or four block reductions in between.
// Bound by HBM: 4 T H elements, 5 with a gate per token; 8192 x 7168 bf16 take
// 89 us, 5.3 TB/s.  Rows that are not whole 16-byte pieces are bound by their
// instructions (weights are read element by element there): 1021 x 4099 fp16
// with a gate take 28.7 us, 1.46 TB/s.  Arithmetic goes in packed float32
// pairs: in single operations on 16-bit elements the kernel was bound by its
// instructions (53 an element).
#include <algorithm>

#include "wq_serve.cuh"

namespace wq {
namespace {

// Sum over the row's threads.  `red` is this reduction's own 32 floats, so
// that one barrier between write and read is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
  v = warp_sum(v);
  if constexpr (WARP) return v;
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (l == 0) red[w] = v;
  __syncthreads();
  return warp_sum(l < nw ? red[l] : 0.0f);
}

// The elements of a row that a thread holds: NV pieces of VW.  Where H and the
// pitches are whole pieces, piece k begins at i0 + k * step.  Else (SHIFT) a
// row begins some elements after a 16-byte boundary, the pieces are the
// aligned ones around it, and the row's first and last piece are taken
// element by element.
//
// FULL: every thread holds NV pieces (no bounds to ask for).
template <class DT, int VW, int NV, bool WARP, bool SHIFT, bool FULL = false>
struct Row {
  using Raw = typename DT::Raw;
  using V = Vec<DT, VW>;
  static constexpr int kPieces = NV;
  static constexpr int NP = VW / 2;  // pairs of a piece
  Pair v[NV][NP];
  int i0, step, H;

  __device__ __forceinline__ int at(int k) const { return i0 + k * step; }
  __device__ __forceinline__ bool in(int k) const {  // some of piece k
    return FULL ? true : SHIFT ? at(k) < H && at(k) + VW > 0 : at(k) < H;
  }
  __device__ __forceinline__ bool whole(int k) const { return at(k) >= 0 && at(k) + VW <= H; }
  __device__ __forceinline__ bool has(int k, int e) const {
    return SHIFT ? unsigned(at(k) + e) < unsigned(H) : in(k);
  }
  static __device__ __forceinline__ void pairs(const V &x, Pair (&p)[NP]) {
    float f[VW];
    x.get(f);
#pragma unroll
    for (int i = 0; i < NP; ++i) p[i] = pair(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ V each(const Raw *p, int k) const {
    uint32_t w[4];
    if (whole(k)) {  // no bounds to ask for
      const Raw *x = p + at(k);
      if constexpr (VW == 8) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) w[e / 2] = __byte_perm(x[e], x[e + 1], 0x5410);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[e]);
      }
    } else if constexpr (VW == 8) {
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        w[e / 2] = (has(k, e) ? uint32_t(p[at(k) + e]) : 0u) |
                   (has(k, e + 1) ? uint32_t(p[at(k) + e + 1]) << 16 : 0u);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = has(k, e) ? __float_as_uint(p[at(k) + e]) : 0u;
    }
    return {make_uint4(w[0], w[1], w[2], w[3])};
  }
  __device__ __forceinline__ V load(const Raw *p, int k) const {
    if constexpr (!SHIFT) return V::load(p + at(k));
    else return whole(k) ? V::load(p + at(k)) : each(p, k);
  }
  // a weight, a bias or a shared gate: its pieces lie shifted against the row's
  __device__ __forceinline__ V load_weight(const Raw *p, int k) const {
    if constexpr (!SHIFT) return V::load(p + at(k));
    else return each(p, k);
  }
  __device__ __forceinline__ void store(Raw *p, int k) const {
    float f[VW];
#pragma unroll
    for (int i = 0; i < NP; ++i) split(v[k][i], f[2 * i], f[2 * i + 1]);
    if (!SHIFT || whole(k)) {
      V x;
      x.set(f);
      x.store(p + at(k));
    } else if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (has(k, e)) p[at(k) + e] = DT::from_f(f[e]);
    }
  }
  __device__ __forceinline__ void clear_past(int k) {  // 0 outside the row
    if (SHIFT ? whole(k) : in(k)) return;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!has(k, 2 * i) || !has(k, 2 * i + 1)) {
        float x, y;
        split(v[k][i], x, y);
        v[k][i] = pair(has(k, 2 * i) ? x : 0.0f, has(k, 2 * i + 1) ? y : 0.0f);
      }
    }
  }

  // v = residual + scale * (gate * v) for piece k
  __device__ __forceinline__ void add(int k, const V *gate, float scale, const V *residual) {
    Pair r[NP] = {};
    if (residual) pairs(*residual, r);
    if (gate) {
      Pair g[NP];
      pairs(*gate, g);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[k][i] = mul_p(v[k][i], g[i]);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) v[k][i] = fma_p(v[k][i], pair(scale, scale), r[i]);
  }

  // v = N(v)
  __device__ __forceinline__ void norm(int kind, const void *weight, const void *bias, float eps,
                                       float (*red)[32]) {
    if (kind == WQ_NORM_NONE) return;
    const bool layer = kind == WQ_NORM_LAYER;
    const auto *w = static_cast<const Raw *>(weight);
    const auto *c = static_cast<const Raw *>(layer ? bias : nullptr);
    // weights are asked for ahead of the reductions where registers allow
    constexpr bool kAhead = NV <= 2 || (NV <= 4 && !SHIFT), kBiasAhead = NV <= 2;
    V wv[NV], cv[NV];
    if (kAhead && w) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (in(k)) wv[k] = load_weight(w, k);
    }
    if (kBiasAhead && c) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (in(k)) cv[k] = load_weight(c, k);
    }
    const float over_h = __frcp_rn(float(H));
    float x, y;
    if (layer) {
      Pair s = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k)  // 0 past the row
#pragma unroll
        for (int i = 0; i < NP; ++i) s = add_p(s, v[k][i]);
      split(s, x, y);
      const float m = -row_sum<WARP>(x + y, red[0]) * over_h;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < NP; ++i) v[k][i] = add_p(v[k][i], pair(m, m));
        clear_past(k);
      }
    }
    Pair s = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i) s = fma_p(v[k][i], v[k][i], s);
    split(s, x, y);
    const float r = rsqrtf(__fmaf_rn(row_sum<WARP>(x + y, red[1]), over_h, eps));
    if (w) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
        if (!kAhead) wv[k] = load_weight(w, k);
        Pair f[NP];
        pairs(wv[k], f);
#pragma unroll
        for (int i = 0; i < NP; ++i) v[k][i] = mul_p(mul_p(v[k][i], pair(r, r)), f[i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < NP; ++i) v[k][i] = mul_p(v[k][i], pair(r, r));
    }
    if (c) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!in(k)) continue;
        Pair f[NP];
        if (!kBiasAhead) cv[k] = load_weight(c, k);
        pairs(cv[k], f);
#pragma unroll
        for (int i = 0; i < NP; ++i) v[k][i] = add_p(v[k][i], f[i]);
        if (SHIFT) clear_past(k);
      }
    }
  }
};

// h is in the registers: x_out, N_pre and y
template <class R>
__device__ __forceinline__ void finish(const BlockNormArgs &a, int64_t t, R &row, float (*red)[32]) {
  using Raw = typename R::Raw;
  if (a.x_out) {
#pragma unroll
    for (int k = 0; k < R::kPieces; ++k)
      if (row.in(k)) row.store(static_cast<Raw *>(a.x_out) + t * a.ldx, k);
  }
  if (!a.y) return;
  row.norm(a.pre, a.w_pre, a.b_pre, a.eps, red);
#pragma unroll
  for (int k = 0; k < R::kPieces; ++k)
    if (row.in(k)) row.store(static_cast<Raw *>(a.y) + t * a.ldy, k);
}
__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

// Threads of a block at most, and blocks that share an SM at least: the rows
// in flight hide the reductions of each.
template <int NV, bool WARP>
constexpr int max_threads() { return WARP ? 128 : (NV == 1 ? 1024 : (NV <= 4 ? 288 : 512)); }
template <int NV, bool WARP>
constexpr int min_blocks() { return WARP ? 6 : (NV == 1 ? 1 : (NV <= 4 ? 3 : 1)); }

template <class DT, int VW, int NV, bool WARP, bool SHIFT, bool GATE>
__global__ void __launch_bounds__(max_threads<NV, WARP>(), min_blocks<NV, WARP>())
    block_norm_kernel(const BlockNormArgs a) {
  using Raw = typename DT::Raw;
  using V = Vec<DT, VW>;
  __shared__ float red[4][32];
  const int64_t t = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.T) return;  // a whole warp: no block barrier in the warp form
  const Raw *bp = static_cast<const Raw *>(a.block) + t * a.ldb;
  const Raw *rp = static_cast<const Raw *>(a.residual) + t * a.ldr;
  const Raw *gp = static_cast<const Raw *>(a.gate) + t * a.ldg;
  Row<DT, VW, NV, WARP, SHIFT> row;
  row.H = a.H;
  row.i0 = (WARP ? threadIdx.x & 31 : threadIdx.x) * VW;
  row.step = (WARP ? 32 : blockDim.x) * VW;
  if (SHIFT) row.i0 -= int(reinterpret_cast<uintptr_t>(bp) / sizeof(Raw) % VW);
  // The residual and the gate are asked for together with the block, ahead of
  // the first norm, unless the row is too wide to keep them beside it.
  constexpr bool kEarly = NV * VW * sizeof(Raw) <= 64;
  V b[NV], r[NV], g[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (row.in(k)) b[k] = row.load(bp, k);
  if (kEarly && a.residual) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (row.in(k)) r[k] = row.load(rp, k);
  }
  if (GATE && kEarly) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (row.in(k)) g[k] = SHIFT && a.ldg == 0 ? row.load_weight(gp, k) : row.load(gp, k);
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (row.in(k)) {
      row.pairs(b[k], row.v[k]);
    } else {
#pragma unroll
      for (int i = 0; i < row.NP; ++i) row.v[k][i] = 0;
    }
  }
  row.norm(a.post, a.w_post, a.b_post, a.eps, red);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!row.in(k)) continue;
    if (!kEarly) {
      if (a.residual) r[k] = row.load(rp, k);
      if (GATE) g[k] = SHIFT && a.ldg == 0 ? row.load_weight(gp, k) : row.load(gp, k);
    }
    row.add(k, GATE ? &g[k] : nullptr, a.scale, a.residual ? &r[k] : nullptr);
  }
  finish(a, t, row, red + 2);
}

// Many rows: a block walks rows t, t + grid, ... and each thread copies its own
// pieces of the row after the one at hand into shared memory while it works
// on that, so that loads are always in flight and no thread waits for another
// outside the reductions (a thread reads back only what it copied itself).
template <class DT, int NV, bool GATE, bool FULL>
__global__ void __launch_bounds__(256, 3) block_norm_stream_kernel(const BlockNormArgs a) {
  using Raw = typename DT::Raw;
  constexpr int VW = DT::kVec;
  using V = Vec<DT, VW>;
  __shared__ float red[2][4][32];  // by parity of the row
  extern __shared__ __align__(16) uint8_t smem[];
  Row<DT, VW, NV, false, false, FULL> row;
  row.H = a.H;
  row.i0 = threadIdx.x * VW;
  row.step = blockDim.x * VW;
  const int pitch = row.step * NV;  // staged elements of one array
  constexpr int ARR = GATE ? 3 : 2;
  auto piece = [&](int buf, int arr, int k) {
    return reinterpret_cast<Raw *>(smem) + (buf * ARR + arr) * pitch + row.at(k);
  };
  auto fetch = [&](int64_t t, int buf) {
    if (t < a.T) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!row.in(k)) continue;
        copy16(piece(buf, 0, k), static_cast<const Raw *>(a.block) + t * a.ldb + row.at(k));
        if (a.residual)
          copy16(piece(buf, 1, k), static_cast<const Raw *>(a.residual) + t * a.ldr + row.at(k));
        if (GATE) copy16(piece(buf, ARR - 1, k), static_cast<const Raw *>(a.gate) + t * a.ldg + row.at(k));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(blockIdx.x, 0);
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, buf ^= 1) {
    fetch(t + gridDim.x, buf ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (row.in(k)) {
        row.pairs(V::load(piece(buf, 0, k)), row.v[k]);
      } else {
#pragma unroll
        for (int i = 0; i < row.NP; ++i) row.v[k][i] = 0;
      }
    }
    row.norm(a.post, a.w_post, a.b_post, a.eps, red[buf]);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!row.in(k)) continue;
      V r, g;
      if (a.residual) r = V::load(piece(buf, 1, k));
      if (GATE) g = V::load(piece(buf, ARR - 1, k));
      row.add(k, GATE ? &g : nullptr, a.scale, a.residual ? &r : nullptr);
    }
    finish(a, t, row, red[buf] + 2);
  }
}

// Any width and alignment: the row as floats in shared memory, an element at a
// time.  Very wide rows, and tensors whose rows do not start alike against
// 16-byte boundaries.
template <class DT>
struct AnyRow {
  using Raw = typename DT::Raw;
  float *v;
  int H;

  __device__ __forceinline__ void norm(int kind, const void *weight, const void *bias, float eps,
                                       float (*red)[32]) {
    if (kind == WQ_NORM_NONE) return;
    const bool layer = kind == WQ_NORM_LAYER;
    const auto *w = static_cast<const Raw *>(weight);
    const auto *c = static_cast<const Raw *>(layer ? bias : nullptr);
    const float over_h = __frcp_rn(float(H));
    float m = 0.0f, s = 0.0f;
    if (layer) {
      for (int i = threadIdx.x; i < H; i += blockDim.x) s += v[i];
      m = row_sum<false>(s, red[0]) * over_h;
      s = 0.0f;
    }
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      v[i] -= m;
      s = __fmaf_rn(v[i], v[i], s);
    }
    const float r = rsqrtf(__fmaf_rn(row_sum<false>(s, red[1]), over_h, eps));
    for (int i = threadIdx.x; i < H; i += blockDim.x)
      v[i] = __fmaf_rn(v[i] * r, w ? DT::to_f(w[i]) : 1.0f, c ? DT::to_f(c[i]) : 0.0f);
  }
  __device__ __forceinline__ void store(Raw *p) const {
    for (int i = threadIdx.x; i < H; i += blockDim.x) p[i] = DT::from_f(v[i]);
  }
};
template <class DT>
__global__ void __launch_bounds__(512) block_norm_any_kernel(const BlockNormArgs a) {
  using Raw = typename DT::Raw;
  __shared__ float red[4][32];
  extern __shared__ __align__(16) uint8_t smem[];
  const int64_t t = blockIdx.x;
  const Raw *bp = static_cast<const Raw *>(a.block) + t * a.ldb;
  const Raw *rp = static_cast<const Raw *>(a.residual) + t * a.ldr;
  const Raw *gp = static_cast<const Raw *>(a.gate) + t * a.ldg;
  // a thread works on its own elements of the row throughout
  AnyRow<DT> row{reinterpret_cast<float *>(smem), a.H};
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) row.v[i] = DT::to_f(bp[i]);
  row.norm(a.post, a.w_post, a.b_post, a.eps, red);
  for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
    float x = row.v[i];
    if (a.gate) x *= DT::to_f(gp[i]);
    row.v[i] = __fmaf_rn(x, a.scale, a.residual ? DT::to_f(rp[i]) : 0.0f);
  }
  if (a.x_out) row.store(static_cast<Raw *>(a.x_out) + t * a.ldx);
  if (!a.y) return;
  row.norm(a.pre, a.w_pre, a.b_pre, a.eps, red + 2);
  row.store(static_cast<Raw *>(a.y) + t * a.ldy);
}

template <class DT>
int launch_any(const BlockNormArgs &a, cudaStream_t st) {
  auto *k = block_norm_any_kernel<DT>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, 32768 * 4)) return WQ_ERR_LAUNCH;
  const int threads = std::min(512, (a.H + 31) / 32 * 32);
  k<<<unsigned(a.T), threads, a.H * 4, st>>>(a);
  return launched(1);
}

template <class DT, int VW, int NV, bool WARP, bool SHIFT>
int launch_one(const BlockNormArgs &a, int threads, cudaStream_t st) {
  const int64_t blocks = WARP ? (a.T + threads / 32 - 1) / (threads / 32) : a.T;
  if (a.gate) block_norm_kernel<DT, VW, NV, WARP, SHIFT, true><<<unsigned(blocks), threads, 0, st>>>(a);
  else block_norm_kernel<DT, VW, NV, WARP, SHIFT, false><<<unsigned(blocks), threads, 0, st>>>(a);
  return launched(1);
}

inline int threads_for(int pieces, int nv) { return ((pieces + nv - 1) / nv + 31) / 32 * 32; }

template <class DT, int NV, bool GATE, bool FULL>
int launch_stream_g(const BlockNormArgs &a, int pieces, cudaStream_t st) {
  auto *k = block_norm_stream_kernel<DT, NV, GATE, FULL>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, 2 * (GATE ? 3 : 2) * 256 * NV * 16)) return WQ_ERR_LAUNCH;
  const int threads = threads_for(pieces, NV), smem = 2 * (GATE ? 3 : 2) * threads * NV * 16;
  // as many blocks as fit: three of 256 threads by registers, fewer by shared memory
  const int per_sm = std::max(1, std::min(768 / threads, std::min(233472 / (smem + 2048), 8)));
  k<<<unsigned(std::min<int64_t>(a.T, 152 * per_sm)), threads, smem, st>>>(a);
  return launched(1);
}
template <class DT, int NV>
int launch_stream(const BlockNormArgs &a, int pieces, cudaStream_t st) {
  if (pieces % (32 * NV) == 0)
    return a.gate ? launch_stream_g<DT, NV, true, true>(a, pieces, st)
                  : launch_stream_g<DT, NV, false, true>(a, pieces, st);
  return a.gate ? launch_stream_g<DT, NV, true, false>(a, pieces, st)
                : launch_stream_g<DT, NV, false, false>(a, pieces, st);
}

template <class DT, bool SHIFT>
int launch_t(const BlockNormArgs &a, cudaStream_t st) {
  constexpr int VW = DT::kVec;
  const int pieces = (a.H + VW - 1) / VW + (SHIFT ? 1 : 0);
  if (pieces <= 32) return launch_one<DT, VW, 1, true, SHIFT>(a, 128, st);
  if (pieces <= 64) return launch_one<DT, VW, 2, true, SHIFT>(a, 128, st);
  // Few rows: a thread per piece, for the shortest chain of loads.  Many: some
  // pieces a thread, and where rows are whole pieces the next row under way.
  if (a.T <= 2 * 152 && pieces <= 1024)
    return launch_one<DT, VW, 1, false, SHIFT>(a, threads_for(pieces, 1), st);
  if constexpr (!SHIFT) {
    if (a.T > 6 * 152 && pieces <= 4 * 256)
      return pieces <= 2 * 256 ? launch_stream<DT, 2>(a, pieces, st) : launch_stream<DT, 4>(a, pieces, st);
  }
  if (pieces <= 2 * 288) return launch_one<DT, VW, 2, false, SHIFT>(a, threads_for(pieces, 2), st);
  if (pieces <= 4 * 288) return launch_one<DT, VW, 4, false, SHIFT>(a, threads_for(pieces, 4), st);
  if constexpr (!SHIFT) {
    if (pieces <= 8 * 512) return launch_one<DT, VW, 8, false, SHIFT>(a, threads_for(pieces, 8), st);
  }
  return launch_any<DT>(a, st);
}

// How a row is reached: pieces of 16 bytes; such pieces with every row's start
// shifted alike; single elements
template <class DT>
int launch_dt(const BlockNormArgs &a, cudaStream_t st) {
  switch (a.reach) {
    case 0: return launch_t<DT, false>(a, st);
    case 1: return launch_t<DT, true>(a, st);
    default: return launch_any<DT>(a, st);
  }
}

}  // namespace

int launch_block_norm(const BlockNormArgs &a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case WQ_DT_BF16: return launch_dt<Bf16>(a, st);
    case WQ_DT_F16: return launch_dt<F16>(a, st);
    default: return launch_dt<F32>(a, st);
  }
}

}  // namespace wq
