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
#include <algorithm>

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
  // a division of 64 bits takes as long as everything else here
  const int64_t page = slot >> 32 ? slot / a.page_size : int64_t(uint32_t(slot) / uint32_t(a.page_size));
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
inline int lanes_of(const RopeSeg &s, int W) {
  return s.rot / (2 * W) + (s.D - s.rot / (2 * W) * (2 * W) + 2 * W - 1) / (2 * W);
}

// How a launch's warps share a token's segments (host values): the heads of a
// segment side by side in a warp and KH deep
struct Cut {
  int per_token;           // warps
  int tokens;              // of a block of at most 8 warps (1 where a token takes more)
  int lanes[3], side[3];   // of a head; heads side by side
  int warps[3], top[3];    // warps of a segment; first step of a head's sum
};

// A vector's elements as pairs of floats
template <int W, class V>
__device__ __forceinline__ void get_pairs(const V &v, Pair (&p)[W / 2]) {
  float f[W];
  v.get(f);
#pragma unroll
  for (int e = 0; e < W; e += 2) p[e / 2] = pair(f[e], f[e + 1]);
}
template <int W, class V>
__device__ __forceinline__ void set_pairs(V &v, const Pair (&p)[W / 2]) {
  float f[W];
#pragma unroll
  for (int e = 0; e < W; e += 2) split(p[e / 2], f[e], f[e + 1]);
  v.set(f);
}
// (x, y) -> (x c - y s, y c + x s): pairs of neighbours (interleaved layout)
__device__ __forceinline__ Pair turn_inner(Pair p, float c, float s) {
  float x, y;
  split(p, x, y);
  return fma_p(p, pair(c, c), mul_p(pair(y, x), pair(-s, s)));
}

template <class DT, int KH>
__global__ void __launch_bounds__(256) head_norm_vec_kernel(const __grid_constant__ HeadNormArgs h,
                                                            const __grid_constant__ Cut cut) {
  using Raw = typename DT::Raw;
  constexpr int W = DT::kVec, P = W / 2;
  using V = Vec<DT, W>;
  const RopeArgs &a = h.r;
  const int warp = threadIdx.x >> 5, own_token = warp / cut.per_token;
  int rest = int(blockIdx.y) * 8 + warp - own_token * cut.per_token, i = 0;
  const int64_t t = int64_t(blockIdx.x) * cut.tokens + own_token;
  if (t >= a.T || rest >= cut.per_token) return;  // whole warps
  while (rest >= cut.warps[i]) rest -= cut.warps[i], ++i;
  const RopeSeg &s = a.seg[i];
  const int lanes = cut.lanes[i], side = cut.side[i], lane = threadIdx.x & 31;
  const int own = lane / lanes, piece = lane - own * lanes;
  const int head0 = (rest * KH) * side + own;  // heads head0 + k * side
  const bool live = own < side;
  const bool half = a.layout == WQ_ROPE_HALF && piece * 2 * W < s.rot;
  const int o0 = half ? piece * W : piece * 2 * W, o1 = half ? o0 + s.rot / 2 : o0 + W;
  const bool two = o1 < s.D;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + head0 * s.s_head;
  V p[KH], q[KH];
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    p[k].w = q[k].w = make_uint4(0, 0, 0, 0);
    if (live && head0 + k * side < s.heads) {
      p[k] = V::load(x + k * side * s.s_head + o0);
      if (two) q[k] = V::load(x + k * side * s.s_head + o1);
    }
  }
  V w0, w1;
  w0.w = w1.w = make_uint4(0, 0, 0, 0);
  const Raw *weight = static_cast<const Raw *>(h.weight[i]);
  if (weight && live) {
    w0 = V::load(weight + o0);
    if (two) w1 = V::load(weight + o1);
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
  d += head0 * s.d_head;
  if (!h.norm[i]) {  // values
#pragma unroll
    for (int k = 0; k < KH; ++k)
      if (live && head0 + k * side < s.heads) {
        p[k].store(d + k * side * s.d_head + o0);
        if (two) q[k].store(d + k * side * s.d_head + o1);
      }
    return;
  }
  // pairs of the first and of the second vector that turn
  const bool inter = a.layout == WQ_ROPE_INTERLEAVED;
  const bool first = live && (half || (inter && o0 < s.rot)), second = live && inter && o1 < s.rot;
  float4 cs[P];  // cos and sin of two of the lane's pairs of elements each
  if (first) {
    const float2 *r = row + (half ? o0 : o0 / 2);
#pragma unroll
    for (int e = 0; e < P; ++e)
      if (e < P / 2 || half || second) cs[e] = *reinterpret_cast<const float4 *>(r + 2 * e);
  }
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int head = head0 + k * side;
    if (__all_sync(0xffffffffu, head >= s.heads)) break;
    Pair f[P], g[P], sq = pair(0.0f, 0.0f);
    get_pairs<W>(p[k], f);
    get_pairs<W>(q[k], g);
#pragma unroll
    for (int e = 0; e < P; ++e) sq = fma_p(f[e], f[e], sq);
#pragma unroll
    for (int e = 0; e < P; ++e) sq = fma_p(g[e], g[e], sq);
    float sum, more;
    split(sq, sum, more);
    sum = head_sum(__fadd_rn(sum, more), lanes, piece, cut.top[i]);
    const float r = rsqrtf(__fmaf_rn(sum, h.inv_d[i], h.eps));
    const Pair rr = pair(r, r);
#pragma unroll
    for (int e = 0; e < P; ++e) f[e] = mul_p(f[e], rr), g[e] = mul_p(g[e], rr);
    if (weight) {
      Pair u[P];
      get_pairs<W>(w0, u);
#pragma unroll
      for (int e = 0; e < P; ++e) f[e] = mul_p(f[e], u[e]);
      get_pairs<W>(w1, u);
#pragma unroll
      for (int e = 0; e < P; ++e) g[e] = mul_p(g[e], u[e]);
    }
    if (first) {
      if (half) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const Pair c = pair(cs[e].x, cs[e].z), n = pair(cs[e].y, cs[e].w), m = pair(-cs[e].y, -cs[e].w);
          const Pair u = fma_p(f[e], c, mul_p(g[e], m));
          g[e] = fma_p(g[e], c, mul_p(f[e], n));
          f[e] = u;
        }
      } else {
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          f[e] = turn_inner(f[e], cs[e / 2].x, cs[e / 2].y);
          f[e + 1] = turn_inner(f[e + 1], cs[e / 2].z, cs[e / 2].w);
        }
        if (second) {
#pragma unroll
          for (int e = 0; e < P; e += 2) {
            g[e] = turn_inner(g[e], cs[(P + e) / 2].x, cs[(P + e) / 2].y);
            g[e + 1] = turn_inner(g[e + 1], cs[(P + e) / 2].z, cs[(P + e) / 2].w);
          }
        }
      }
    }
    if (live && head < s.heads) {
      set_pairs<W>(p[k], f);
      p[k].store(d + k * side * s.d_head + o0);
      if (two) {
        set_pairs<W>(q[k], g);
        q[k].store(d + k * side * s.d_head + o1);
      }
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
  Cut c{};
  for (int i = 0; i < h.r.nseg; ++i) {
    const RopeSeg &s = h.r.seg[i];
    c.lanes[i] = lanes_of(s, DT::kVec);
    c.side[i] = 32 / c.lanes[i];
    c.warps[i] = (s.heads + c.side[i] * KH - 1) / (c.side[i] * KH);
    for (c.top[i] = 1; 2 * c.top[i] < c.lanes[i];) c.top[i] *= 2;
    c.per_token += c.warps[i];
  }
  c.tokens = std::max(1, 8 / c.per_token);
  const dim3 grid(unsigned((h.r.T + c.tokens - 1) / c.tokens), unsigned((c.per_token + 7) / 8));
  if (grid.y > 65535) return WQ_ERR_UNSUPPORTED;
  const int warps = c.tokens * std::min(c.per_token, 8);
  if (c.per_token > 8) c.tokens = 1;
  head_norm_vec_kernel<DT, KH><<<grid, unsigned(warps * 32), 0, st>>>(h, c);
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
