// The norm of each query and key head and its rotary position in one pass,
// and the same on the way into a paged cache.
//
//   y = R(p) (x r w),  r = 1 / sqrt(mean(x^2) + eps)  over a head's D elements,
//
// where R(p) turns the pairs below rot.  A lane owns two 16-byte vectors of a
// head, which hold both elements of every pair they touch (half a rotation
// apart in the half layout), so one read serves the sum of squares and the
// rotation.  The lanes of a head are neighbours in a warp and add their sums by
// shuffles; with many tokens a lane takes the same place of two heads, which
// share the table row's and the weight's part.  Bound by HBM: every element is
// read once and written once; table rows come from L2.
#include <algorithm>

#include "wq_warp_mma.cuh"

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

// A lane's place in a token: its segment, its heads (head0 + k * side) and the
// vectors at o0 and o1 of each
template <int W>
struct Place {
  int i, head0, side, lanes, piece, top;
  int o0, o1;
  bool live, two;          // a lane with a head; with a second vector
  bool half;               // its two vectors turn against each other
  bool first, second;      // else: the pairs inside the first, the second vector turn
  __device__ __forceinline__ Place(const HeadNormArgs &h, const Cut &cut, int rest, int KH) {
    const int lane = threadIdx.x & 31;
    i = 0;
    while (rest >= cut.warps[i]) rest -= cut.warps[i], ++i;
    const RopeSeg &s = h.r.seg[i];
    lanes = cut.lanes[i];
    side = cut.side[i];
    top = cut.top[i];
    const int own = lane / lanes;
    piece = lane - own * lanes;
    head0 = rest * KH * side + own;
    live = own < side;
    // Half layout: the rotated vectors half a rotation apart, then the rest;
    // interleaved: all vectors.  The lanes of a head take neighbours each time.
    const int turned = h.r.layout == WQ_ROPE_HALF ? s.rot / (2 * W) : 0, from = turned * 2 * W;
    half = piece < turned;
    o0 = half ? piece * W : from + (piece - turned) * W;
    o1 = half ? o0 + s.rot / 2 : o0 + (lanes - turned) * W;
    two = o1 < s.D;
    const bool inter = h.r.layout == WQ_ROPE_INTERLEAVED;
    first = live && inter && o0 < s.rot;
    second = live && inter && o1 < s.rot;
    half = half && live;
  }
};

// The table row's part of a lane: cos and sin of two pairs of elements in each
template <int W>
__device__ __forceinline__ void load_turns(const Place<W> &l, const float2 *row, float4 (&cs)[W / 2]) {
#pragma unroll
  for (int e = 0; e < W / 4; ++e) {
    if (l.half || l.first) cs[e] = *reinterpret_cast<const float4 *>(row + (l.half ? l.o0 : l.o0 / 2) + 2 * e);
    if (l.half || l.second)
      cs[W / 4 + e] = *reinterpret_cast<const float4 *>(row + (l.half ? l.o0 + W / 2 : l.o1 / 2) + 2 * e);
  }
}

// Norm and rotation of one head's two vectors, in place
template <class DT, int W = DT::kVec>
__device__ __forceinline__ void norm_turn(Vec<DT, W> &p, Vec<DT, W> &q, const Vec<DT, W> &w0, const Vec<DT, W> &w1,
                                          bool weighted, const float4 (&cs)[W / 2], const Place<W> &l, float inv_d,
                                          float eps) {
  constexpr int P = W / 2;
  Pair f[P], g[P], sq = pair(0.0f, 0.0f);
  get_pairs<W>(p, f);
  get_pairs<W>(q, g);
#pragma unroll
  for (int e = 0; e < P; ++e) sq = fma_p(f[e], f[e], sq);
#pragma unroll
  for (int e = 0; e < P; ++e) sq = fma_p(g[e], g[e], sq);
  float sum, more;
  split(sq, sum, more);
  sum = head_sum(__fadd_rn(sum, more), l.lanes, l.piece, l.top);
  const float r = rsqrtf(__fmaf_rn(sum, inv_d, eps));
  const Pair rr = pair(r, r);
#pragma unroll
  for (int e = 0; e < P; ++e) f[e] = mul_p(f[e], rr), g[e] = mul_p(g[e], rr);
  if (weighted) {
    Pair u[P];
    get_pairs<W>(w0, u);
#pragma unroll
    for (int e = 0; e < P; ++e) f[e] = mul_p(f[e], u[e]);
    get_pairs<W>(w1, u);
#pragma unroll
    for (int e = 0; e < P; ++e) g[e] = mul_p(g[e], u[e]);
  }
  if (l.half) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const Pair c = pair(cs[e].x, cs[e].z), n = pair(cs[e].y, cs[e].w), m = pair(-cs[e].y, -cs[e].w);
      const Pair u = fma_p(f[e], c, mul_p(g[e], m));
      g[e] = fma_p(g[e], c, mul_p(f[e], n));
      f[e] = u;
    }
  }
  if (l.first) {
#pragma unroll
    for (int e = 0; e < P; e += 2) {
      f[e] = turn_inner(f[e], cs[e / 2].x, cs[e / 2].y);
      f[e + 1] = turn_inner(f[e + 1], cs[e / 2].z, cs[e / 2].w);
    }
  }
  if (l.second) {
#pragma unroll
    for (int e = 0; e < P; e += 2) {
      g[e] = turn_inner(g[e], cs[(P + e) / 2].x, cs[(P + e) / 2].y);
      g[e + 1] = turn_inner(g[e + 1], cs[(P + e) / 2].z, cs[(P + e) / 2].w);
    }
  }
  set_pairs<W>(p, f);
  set_pairs<W>(q, g);
}

// Where a token of a segment goes and its table row; false: it is skipped.
// With at the token's position and slot (0 where there is none).
template <class Raw>
__device__ __forceinline__ bool route(const RopeArgs &a, const RopeSeg &s, int64_t t, int64_t slot, int at, bool tell,
                                      Raw *&d, const float2 *&row) {
  d = static_cast<Raw *>(s.dst);
  row = nullptr;
  if (s.paged) {
    if (slot < 0) return false;
    if (slot >= a.num_slots) {
      if (tell) set_status(a.status, WQ_ERR_INDEX);
      return false;
    }
    // a division of 64 bits takes as long as all the rest of a lane's work
    const int64_t page = slot >> 32 ? slot / a.page_size : int64_t(uint32_t(slot) / uint32_t(a.page_size));
    d += page * s.d_page + (slot - page * a.page_size) * s.d_token;
  } else {
    d += t * s.d_token;
  }
  if (s.rot || (s.paged && a.rot)) {
    if (at < 0 || at >= a.max_pos) {
      if (tell) set_status(a.status, WQ_ERR_INDEX);
      return false;
    }
    row = reinterpret_cast<const float2 *>(a.table) + int64_t(at) * (a.rot / 2);
  }
  return true;
}

// Few tokens: a warp takes one
template <class DT>
__global__ void __launch_bounds__(256) head_norm_vec_kernel(const __grid_constant__ HeadNormArgs h,
                                                            const __grid_constant__ Cut cut) {
  using Raw = typename DT::Raw;
  constexpr int W = DT::kVec;
  using V = Vec<DT, W>;
  const RopeArgs &a = h.r;
  const int warp = threadIdx.x >> 5, own_token = warp / cut.per_token;
  const int rest = int(blockIdx.y) * 8 + warp - own_token * cut.per_token;
  const int64_t t = int64_t(blockIdx.x) * cut.tokens + own_token;
  if (t >= a.T || rest >= cut.per_token) return;  // whole warps
  const Place<W> l(h, cut, rest, 1);
  const RopeSeg &s = a.seg[l.i];
  const bool on = l.live && l.head0 < s.heads;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + l.head0 * s.s_head;
  V p, q, w0, w1;
  p.w = q.w = w0.w = w1.w = make_uint4(0, 0, 0, 0);
  if (on) p = V::load(x + l.o0);
  if (on && l.two) q = V::load(x + l.o1);
  const Raw *weight = static_cast<const Raw *>(h.weight[l.i]);
  if (weight && l.live) {
    w0 = V::load(weight + l.o0);
    if (l.two) w1 = V::load(weight + l.o1);
  }
  Raw *d;
  const float2 *row;
  if (!route<Raw>(a, s, t, s.paged ? a.slots[t] : 0, a.rot ? a.positions[t] : 0, (threadIdx.x & 31) == 0, d, row))
    return;  // the same for the whole warp
  if (h.norm[l.i]) {
    float4 cs[W / 2];
    load_turns<W>(l, row, cs);
    norm_turn<DT>(p, q, w0, w1, weight != nullptr, cs, l, h.inv_d[l.i], h.eps);
  }
  d += l.head0 * s.d_head;
  if (on) p.store(d + l.o0);
  if (on && l.two) q.store(d + l.o1);
}

// Many tokens: a warp keeps its place and walks over the tokens.  Its lanes
// copy their own vectors of the tokens to come into shared memory (no thread
// reads another's, so a thread waits for its own copies alone); position and
// slot are read two tokens ahead and the table row one, which takes their
// latencies, one after the other, out of a token's way.
constexpr int STAGES = 4;
template <class DT, int KH>
__global__ void __launch_bounds__(256, 2) head_norm_stream_kernel(const __grid_constant__ HeadNormArgs h,
                                                               const __grid_constant__ Cut cut) {
  using Raw = typename DT::Raw;
  constexpr int W = DT::kVec;
  using V = Vec<DT, W>;
  extern __shared__ uint4 ring[];  // [STAGES][2 KH][threads]
  const RopeArgs &a = h.r;
  const int warp = threadIdx.x >> 5, own_token = warp / cut.per_token;
  const int rest = int(blockIdx.y) * 8 + warp - own_token * cut.per_token;
  const int64_t t0 = int64_t(blockIdx.x) * cut.tokens + own_token, by = int64_t(gridDim.x) * cut.tokens;
  if (t0 >= a.T || rest >= cut.per_token) return;  // whole warps
  const Place<W> l(h, cut, rest, KH);
  const RopeSeg &s = a.seg[l.i];
  const Raw *x = static_cast<const Raw *>(s.src) + t0 * s.s_token + l.head0 * s.s_head;
  const Raw *none = static_cast<const Raw *>(s.src);  // of copies of nothing
  const Raw *weight = static_cast<const Raw *>(h.weight[l.i]);
  V w0, w1;
  w0.w = w1.w = make_uint4(0, 0, 0, 0);
  if (weight && l.live) {
    w0 = V::load(weight + l.o0);
    if (l.two) w1 = V::load(weight + l.o1);
  }
  bool on[KH];
#pragma unroll
  for (int k = 0; k < KH; ++k) on[k] = l.live && l.head0 + k * l.side < s.heads;
  const uint32_t mine = uint32_t(__cvta_generic_to_shared(ring + threadIdx.x)), stage = 2 * KH * blockDim.x * 16;
  int64_t t_in = t0;
  uint32_t in = 0;
  auto copy = [&]() {
    if (t_in < a.T) {
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const uint32_t to = mine + in + 2 * k * blockDim.x * 16;
        const Raw *from = x + k * l.side * s.s_head;
        cp16(to, on[k] ? from + l.o0 : none, on[k]);
        cp16(to + blockDim.x * 16, on[k] && l.two ? from + l.o1 : none, on[k] && l.two);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    x += t_in + by < a.T ? by * s.s_token : 0;
    t_in += by;
    in = in == (STAGES - 1) * stage ? 0 : in + stage;
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) copy();
  auto slot_of = [&](int64_t t) { return s.paged && t < a.T ? a.slots[t] : 0; };
  auto at_of = [&](int64_t t) { return a.rot && t < a.T ? a.positions[t] : 0; };
  const bool tell = (threadIdx.x & 31) == 0;
  int64_t slot = slot_of(t0 + by);
  int at = at_of(t0 + by);
  Raw *d;
  const float2 *row;
  float4 cs[W / 2], cs_next[W / 2];
  bool write = route<Raw>(a, s, t0, slot_of(t0), at_of(t0), tell, d, row);
  if (write && h.norm[l.i]) load_turns<W>(l, row, cs);
  uint32_t out = 0;
#pragma unroll 1
  for (int64_t t = t0; t < a.T; t += by) {
    copy();
    const int64_t slot_next = slot_of(t + 2 * by);
    const int at_next = at_of(t + 2 * by);
    Raw *d_next = nullptr;
    bool write_next = false;
    if (t + by < a.T) {
      write_next = route<Raw>(a, s, t + by, slot, at, tell, d_next, row);
      if (write_next && h.norm[l.i]) load_turns<W>(l, row, cs_next);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    if (write) {  // the same for the whole warp
      Raw *to = d + l.head0 * s.d_head;
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        if (__all_sync(0xffffffffu, !on[k])) break;
        const uint4 *from = ring + threadIdx.x + out / 16 + 2 * k * blockDim.x;
        V p{from[0]}, q{from[blockDim.x]};
        if (h.norm[l.i]) norm_turn<DT>(p, q, w0, w1, weight != nullptr, cs, l, h.inv_d[l.i], h.eps);
        if (on[k]) p.store(to + k * l.side * s.d_head + l.o0);
        if (on[k] && l.two) q.store(to + k * l.side * s.d_head + l.o1);
      }
    }
    out = out == (STAGES - 1) * stage ? 0 : out + stage;
    write = write_next;
    d = d_next;
    slot = slot_next;
    at = at_next;
#pragma unroll
    for (int e = 0; e < W / 2; ++e) cs[e] = cs_next[e];
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

template <class DT, bool STREAM>
int launch_vec(const HeadNormArgs &h, cudaStream_t st) {
  constexpr int KH = STREAM ? 2 : 1;
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
  const unsigned y = unsigned((c.per_token + 7) / 8);
  if (y > 65535) return WQ_ERR_UNSUPPORTED;
  const int threads = 32 * c.tokens * std::min(c.per_token, 8);
  const int64_t blocks = (h.r.T + c.tokens - 1) / c.tokens;
  if constexpr (STREAM) {
    auto *k = head_norm_stream_kernel<DT, KH>;
    const int smem = STAGES * 2 * KH * threads * 16;
    static OncePerDevice sized;
    if (!allow_smem(sized, k, STAGES * 2 * KH * 256 * 16)) return WQ_ERR_LAUNCH;
    const int64_t most = std::max<int64_t>(1, 2 * 152 / y);  // two blocks an SM
    k<<<dim3(unsigned(std::min(blocks, most)), y), threads, smem, st>>>(h, c);
  } else {
    head_norm_vec_kernel<DT><<<dim3(unsigned(blocks), y), threads, 0, st>>>(h, c);
  }
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
  // walks over tokens once each warp has several
  if (vec) return lanes > 2 * 2 * 152 * 256 * 3 ? launch_vec<DT, true>(h, st) : launch_vec<DT, false>(h, st);
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
