// The norm of each query and key head and its rotary position in one pass,
// and the same on the way into a paged cache.
//
//   y = R(p) (x r w),  r = 1 / sqrt(mean(x^2) + eps)  over a head's D elements,
//
// where R(p) turns the pairs below rot.  A lane owns two 16-byte vectors of a
// head, which hold both elements of every pair they touch (half a rotation
// apart in the half layout, adjacent in the interleaved one), so one read
// serves the sum of squares and the rotation.  The lanes of a head are
// neighbours in a warp and add their sums by shuffles; with many tokens a lane
// takes the same place of several heads, whose loads are in flight together and
// which share the table row's and the weight's part.  Bound by HBM: every
// element is read once and written once; table rows come from L2.
#include "wq_serve.cuh"

namespace wq {
namespace {

// Where token t of a segment goes, or nullptr (skipped)
template <class Raw>
__device__ __forceinline__ Raw *dst_of(const RopeArgs &a, const RopeSeg &s, int64_t t, bool tell) {
  Raw *d = static_cast<Raw *>(s.dst);
  if (!s.paged) return d + t * s.d_token;
  const int64_t slot = a.slots[t];
  if (slot < 0) return nullptr;
  if (slot >= a.num_slots) {
    if (tell) set_status(a.status, WQ_ERR_INDEX);
    return nullptr;
  }
  const int64_t page = slot / a.page_size;
  return d + page * s.d_page + (slot - page * a.page_size) * s.d_token;
}

// Sum over the `lanes` neighbours that share a head, lane `place` of them at
// this thread; all of them get it.  The order depends on `lanes` alone.
__device__ __forceinline__ float head_sum(float v, int lanes, int place, int top) {
  for (int o = top; o > 0; o >>= 1) {
    const float w = __shfl_down_sync(0xffffffffu, v, o);
    if (place + o < lanes && place < o) v = __fadd_rn(v, w);
  }
  return __shfl_sync(0xffffffffu, v, (threadIdx.x & 31) - place);
}

__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
  const float u = __fmaf_rn(x, c, -__fmul_rn(y, s));
  y = __fmaf_rn(y, c, __fmul_rn(x, s));
  x = u;
}

// Lanes of one head: two vectors of W elements each
__host__ __device__ inline int lanes_of(const RopeSeg &s, int W) {
  return s.rot / (2 * W) + (s.D - s.rot / (2 * W) * (2 * W) + 2 * W - 1) / (2 * W);
}
// Warps that a token takes in a segment: 32 / lanes heads side by side, KH deep
__host__ __device__ inline int warps_of(const RopeSeg &s, int W, int KH) {
  const int side = 32 / lanes_of(s, W);
  return (s.heads + side * KH - 1) / (side * KH);
}

template <class DT, int KH>
__global__ void __launch_bounds__(256) head_norm_vec_kernel(const HeadNormArgs h, int per_token) {
  using Raw = typename DT::Raw;
  constexpr int W = DT::kVec;
  using V = Vec<DT, W>;
  const RopeArgs &a = h.r;
  const int64_t item = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t t = item / per_token;
  if (t >= a.T) return;  // whole warps
  int rest = int(item - t * per_token), i = 0;
  while (rest >= warps_of(a.seg[i], W, KH)) rest -= warps_of(a.seg[i], W, KH), ++i;
  const RopeSeg &s = a.seg[i];
  const int lanes = lanes_of(s, W), side = 32 / lanes, lane = threadIdx.x & 31;
  const int own = lane / lanes, piece = lane - own * lanes;
  const int head0 = (rest * KH) * side + own;  // heads head0 + k * side
  const bool live = own < side;
  const bool half = piece < s.rot / (2 * W) && a.layout == WQ_ROPE_HALF;
  const int o0 = half ? piece * W : piece * 2 * W, o1 = half ? o0 + s.rot / 2 : o0 + W;
  const bool two = o1 < s.D;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token;
  V p[KH], q[KH];
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int head = head0 + k * side;
    p[k].w = q[k].w = make_uint4(0, 0, 0, 0);
    if (live && head < s.heads) {
      p[k] = V::load(x + head * s.s_head + o0);
      if (two) q[k] = V::load(x + head * s.s_head + o1);
    }
  }
  const bool tell = rest == 0 && lane == 0;
  Raw *d = dst_of<Raw>(a, s, t, tell);
  const float2 *row = nullptr;
  bool write = d != nullptr;
  if (s.rot || (s.paged && a.rot)) {
    const int at = a.positions[t];
    if (at < 0 || at >= a.max_pos) {
      if (tell && write) set_status(a.status, WQ_ERR_INDEX);
      write = false;
    } else {
      row = reinterpret_cast<const float2 *>(a.table) + int64_t(at) * (a.rot / 2);
    }
  }
  if (!write) return;  // the same for the whole warp
  // pairs of the first and of the second vector that turn
  const bool inter = a.layout == WQ_ROPE_INTERLEAVED;
  const bool first = live && (half || (inter && o0 < s.rot));
  const bool second = live && inter && o1 < s.rot;
  float c[W], n[W];  // cos and sin of the pairs
  if (first) {
    const float2 *r = row + (half ? o0 : o0 / 2);
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      if (e < W / 2 || half || second) {
        const float4 w = *reinterpret_cast<const float4 *>(r + e);
        c[e] = w.x;
        n[e] = w.y;
        c[e + 1] = w.z;
        n[e + 1] = w.w;
      }
    }
  }
  float wp[W], wq_[W];
#pragma unroll
  for (int e = 0; e < W; ++e) wp[e] = wq_[e] = 1.0f;
  if (h.weight[i] && live) {
    const Raw *w = static_cast<const Raw *>(h.weight[i]);
    V::load(w + o0).get(wp);
    if (two) V::load(w + o1).get(wq_);
  }
  int top = 1;  // the first step of the heads' sums
  while (2 * top < lanes) top *= 2;
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int head = head0 + k * side;
    if (__all_sync(0xffffffffu, head >= s.heads)) break;
    if (h.norm[i]) {
      float f[W], g[W];
      p[k].get(f);
      q[k].get(g);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < W; ++e) sum = __fmaf_rn(f[e], f[e], sum);
#pragma unroll
      for (int e = 0; e < W; ++e) sum = __fmaf_rn(g[e], g[e], sum);
      sum = head_sum(sum, lanes, piece, top);
      const float r = rsqrtf(__fmaf_rn(sum, h.inv_d[i], h.eps));
#pragma unroll
      for (int e = 0; e < W; ++e) {
        f[e] = __fmul_rn(__fmul_rn(f[e], r), wp[e]);
        g[e] = __fmul_rn(__fmul_rn(g[e], r), wq_[e]);
      }
      if (first) {
        if (half) {
#pragma unroll
          for (int e = 0; e < W; ++e) turn(f[e], g[e], c[e], n[e]);
        } else {
#pragma unroll
          for (int e = 0; e < W / 2; ++e) turn(f[2 * e], f[2 * e + 1], c[e], n[e]);
          if (second) {
#pragma unroll
            for (int e = 0; e < W / 2; ++e) turn(g[2 * e], g[2 * e + 1], c[W / 2 + e], n[W / 2 + e]);
          }
        }
      }
      p[k].set(f);
      q[k].set(g);
    }
    if (live && head < s.heads) {
      p[k].store(d + head * s.d_head + o0);
      if (two) q[k].store(d + head * s.d_head + o1);
    }
  }
}

// Any size, pitch and alignment: a warp per head, a lane per pair or element
template <class DT>
__global__ void __launch_bounds__(256) head_norm_any_kernel(const HeadNormArgs h, int per_token) {
  using Raw = typename DT::Raw;
  const RopeArgs &a = h.r;
  const int64_t item = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t t = item / per_token;
  if (t >= a.T) return;
  int head = int(item - t * per_token), i = 0;
  while (head >= a.seg[i].heads) head -= a.seg[i].heads, ++i;
  const RopeSeg &s = a.seg[i];
  const int lane = threadIdx.x & 31;
  const bool tell = head == 0 && lane == 0;
  Raw *d = dst_of<Raw>(a, s, t, tell);
  if (!d) return;
  const float2 *row = nullptr;
  if (s.rot || (s.paged && a.rot)) {
    const int at = a.positions[t];
    if (at < 0 || at >= a.max_pos) {
      if (tell) set_status(a.status, WQ_ERR_INDEX);
      return;
    }
    row = reinterpret_cast<const float2 *>(a.table) + int64_t(at) * (a.rot / 2);
  }
  d += head * s.d_head;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + head * s.s_head;
  if (!h.norm[i]) {  // values
    for (int e = lane; e < s.D; e += 32) d[e] = x[e];
    return;
  }
  const Raw *w = static_cast<const Raw *>(h.weight[i]);
  float sum = 0.0f;
  for (int e = lane; e < s.D; e += 32) {
    const float f = DT::to_f(x[e]);
    sum = __fmaf_rn(f, f, sum);
  }
  const float r = rsqrtf(__fmaf_rn(warp_sum(sum), h.inv_d[i], h.eps));
  auto normed = [&](int e) {
    const float f = __fmul_rn(DT::to_f(x[e]), r);
    return w ? __fmul_rn(f, DT::to_f(w[e])) : f;
  };
  for (int e = lane; e < s.rot / 2; e += 32) {
    const int o0 = a.layout == WQ_ROPE_HALF ? e : 2 * e;
    const int o1 = a.layout == WQ_ROPE_HALF ? e + s.rot / 2 : o0 + 1;
    float f = normed(o0), g = normed(o1);
    turn(f, g, row[e].x, row[e].y);
    d[o0] = DT::from_f(f);
    d[o1] = DT::from_f(g);
  }
  for (int e = s.rot + lane; e < s.D; e += 32) d[e] = DT::from_f(normed(e));
}

template <class DT, int KH>
int launch_vec(const HeadNormArgs &h, cudaStream_t st) {
  int per_token = 0;
  for (int i = 0; i < h.r.nseg; ++i) per_token += warps_of(h.r.seg[i], DT::kVec, KH);
  const int64_t blocks = (h.r.T * per_token + 7) / 8;
  if (blocks >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  head_norm_vec_kernel<DT, KH><<<unsigned(blocks), 256, 0, st>>>(h, per_token);
  return launched(1);
}

template <class DT>
int launch_t(const HeadNormArgs &h, bool vec, cudaStream_t st) {
  constexpr int W = DT::kVec;
  int64_t lanes = 0;
  for (int i = 0; i < h.r.nseg; ++i) {
    vec = vec && lanes_of(h.r.seg[i], W) <= 32;
    lanes += h.r.T * h.r.seg[i].heads * lanes_of(h.r.seg[i], W);
  }
  // two heads a lane once that leaves each SM a few blocks
  if (vec) return lanes > 2 * 256 * 152 * 8 ? launch_vec<DT, 2>(h, st) : launch_vec<DT, 1>(h, st);
  int per_token = 0;
  for (int i = 0; i < h.r.nseg; ++i) per_token += h.r.seg[i].heads;
  const int64_t blocks = (h.r.T * per_token + 7) / 8;
  if (blocks >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  head_norm_any_kernel<DT><<<unsigned(blocks), 256, 0, st>>>(h, per_token);
  return launched(1);
}

}  // namespace

int launch_head_norm(const HeadNormArgs &h, int dtype, bool vec, cudaStream_t st) {
  switch (dtype) {
    case WQ_DT_BF16: return launch_t<Bf16>(h, vec, st);
    case WQ_DT_F16: return launch_t<F16>(h, vec, st);
    default: return launch_t<F32>(h, vec, st);
  }
}

}  // namespace wq
