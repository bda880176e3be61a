// Norms after and before a block, fused with the gate, the residual scale and
// the residual sum:
//   h = residual + scale * (gate * N_post(block)),  x_out = h,  y = N_pre(h)
//
// A row stays in registers from its one load to its stores: block, residual
// and gate are read once, both outputs written once, and the two norms (the
// second needs the whole of h) cost two or four block reductions in between.
// Bound by HBM: 4 T H elements, 5 with a gate per token.
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

template <class DT, int VW, int NV, bool WARP>
struct Row {
  float v[NV][VW];
  int i0, step, H;  // this thread's elements: i0 + k * step + [0, VW)

  __device__ __forceinline__ bool in(int k) const { return i0 + k * step < H; }

  // v = N(v)
  __device__ __forceinline__ void norm(int kind, const void *weight, const void *bias, float eps,
                                       float (*red)[32]) {
    using V = Vec<DT, VW>;
    const auto *w = static_cast<const typename DT::Raw *>(weight);
    const auto *c = static_cast<const typename DT::Raw *>(bias);
    if (kind == WQ_NORM_NONE) return;
    if (kind == WQ_NORM_LAYER) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VW; ++e) s = __fadd_rn(s, v[k][e]);  // 0 past the row
      const float m = __fdiv_rn(row_sum<WARP>(s, red[0]), float(H));
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < VW; ++e) v[k][e] = in(k) ? __fsub_rn(v[k][e], m) : 0.0f;
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < VW; ++e) s = __fadd_rn(s, __fmul_rn(v[k][e], v[k][e]));
    const float r = __fdiv_rn(
        1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(row_sum<WARP>(s, red[1]), float(H)), eps)));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in(k)) continue;
      V wv, cv;
      if (w) wv = V::load(w + i0 + k * step);
      if (kind == WQ_NORM_LAYER && c) cv = V::load(c + i0 + k * step);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float x = __fmul_rn(v[k][e], r);
        if (w) x = __fmul_rn(x, wv.f(e));
        if (kind == WQ_NORM_LAYER && c) x = __fadd_rn(x, cv.f(e));
        v[k][e] = x;
      }
    }
  }
};

// Threads of a block at most: with more than one piece a thread, half of what
// a block may have, so that a thread may hold its pieces in 128 registers
template <int NV, bool WARP>
constexpr int max_threads() { return WARP ? 128 : (NV == 1 ? 1024 : 512); }

template <class DT, int VW, int NV, bool WARP>
__global__ void __launch_bounds__(max_threads<NV, WARP>()) block_norm_kernel(const BlockNormArgs a) {
  using Raw = typename DT::Raw;
  using V = Vec<DT, VW>;
  __shared__ float red[4][32];
  const int64_t t = WARP ? int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (t >= a.T) return;  // a whole warp: no block barrier in the warp form
  Row<DT, VW, NV, WARP> row;
  row.H = a.H;
  row.i0 = (WARP ? threadIdx.x & 31 : threadIdx.x) * VW;
  row.step = (WARP ? 32 : blockDim.x) * VW;
  const Raw *bp = static_cast<const Raw *>(a.block) + t * a.ldb + row.i0;
  const Raw *rp = static_cast<const Raw *>(a.residual) + t * a.ldr + row.i0;
  const Raw *gp = static_cast<const Raw *>(a.gate) + t * a.ldg + row.i0;
  // The residual and the gate are asked for together with the block, ahead of
  // the first norm, unless the row is too wide to keep them beside it.
  constexpr bool kEarly = NV * VW * sizeof(Raw) <= 64;
  V b[NV], r[NV], g[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (row.in(k)) b[k] = V::load(bp + k * row.step);
  if (kEarly && a.residual) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (row.in(k)) r[k] = V::load(rp + k * row.step);
  }
  if (kEarly && a.gate) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (row.in(k)) g[k] = V::load(gp + k * row.step);
  }
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < VW; ++e) row.v[k][e] = row.in(k) ? b[k].f(e) : 0.0f;
  row.norm(a.post, a.w_post, a.b_post, a.eps, red);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!row.in(k)) continue;
    if (!kEarly) {
      if (a.residual) r[k] = V::load(rp + k * row.step);
      if (a.gate) g[k] = V::load(gp + k * row.step);
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      float x = row.v[k][e];
      if (a.gate) x = __fmul_rn(g[k].f(e), x);
      x = __fmul_rn(a.scale, x);
      if (a.residual) x = __fadd_rn(r[k].f(e), x);
      row.v[k][e] = x;
    }
  }
  if (a.x_out) {
    Raw *xp = static_cast<Raw *>(a.x_out) + t * a.ldx + row.i0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!row.in(k)) continue;
      V o;
#pragma unroll
      for (int e = 0; e < VW; ++e) o.set(e, row.v[k][e]);
      o.store(xp + k * row.step);
    }
  }
  if (!a.y) return;
  row.norm(a.pre, a.w_pre, a.b_pre, a.eps, red + 2);
  Raw *yp = static_cast<Raw *>(a.y) + t * a.ldy + row.i0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!row.in(k)) continue;
    V o;
#pragma unroll
    for (int e = 0; e < VW; ++e) o.set(e, row.v[k][e]);
    o.store(yp + k * row.step);
  }
}

template <class DT, int VW, int NV, bool WARP>
int launch_one(const BlockNormArgs &a, int threads, cudaStream_t st) {
  const int64_t blocks = WARP ? (a.T + threads / 32 - 1) / (threads / 32) : a.T;
  block_norm_kernel<DT, VW, NV, WARP><<<unsigned(blocks), threads, 0, st>>>(a);
  return launched(1);
}

inline int threads_for(int pieces, int nv) { return ((pieces + nv - 1) / nv + 31) / 32 * 32; }

template <class DT, int VW>
int launch_t(const BlockNormArgs &a, cudaStream_t st) {
  const int pieces = (a.H + VW - 1) / VW;
  if (pieces <= 32) return launch_one<DT, VW, 1, true>(a, 128, st);
  if (pieces <= 64) return launch_one<DT, VW, 2, true>(a, 128, st);
  if (pieces <= 128) return launch_one<DT, VW, 4, true>(a, 128, st);
  // Few rows: a thread per piece, for the shortest chain of loads.  Many: four
  // or more pieces a thread, so that a row's loads are in flight together.
  if (a.T <= 2 * 152 && pieces <= 1024) return launch_one<DT, VW, 1, false>(a, threads_for(pieces, 1), st);
  if (pieces <= 4 * 512) return launch_one<DT, VW, 4, false>(a, threads_for(pieces, 4), st);
  if (pieces <= 8 * 512) return launch_one<DT, VW, 8, false>(a, threads_for(pieces, 8), st);
  if constexpr (VW < 8) {
    if (pieces <= 16 * 512) return launch_one<DT, VW, 16, false>(a, threads_for(pieces, 16), st);
  }
  if constexpr (VW == 1) return launch_one<DT, VW, 64, false>(a, threads_for(pieces, 64), st);
  return WQ_ERR_UNSUPPORTED;
}

}  // namespace

int launch_block_norm(const BlockNormArgs &a, int dtype, bool vec, cudaStream_t st) {
  switch (dtype) {
    case WQ_DT_BF16: return vec ? launch_t<Bf16, 8>(a, st) : launch_t<Bf16, 1>(a, st);
    case WQ_DT_F16: return vec ? launch_t<F16, 8>(a, st) : launch_t<F16, 1>(a, st);
    default: return vec ? launch_t<F32, 4>(a, st) : launch_t<F32, 1>(a, st);
  }
}

}  // namespace wq
