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
// read once and written once; table rows come from L2.  8191 tokens of 40 query
// heads, 8 keys and 8 values of 128 bf16 take 45.8 us, 5.1 TB/s, at 0.67 of issue.
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

// Norm and rotation of one head's two vectors, in place.  row: cos and sin of
// the token's pairs.  The weight and the rotation are taken before the norm's
// factor, which all of them wait for the sum of squares for.
template <class DT, int W = DT::kVec>
__device__ __forceinline__ void norm_turn(Vec<DT, W> &p, Vec<DT, W> &q, const Vec<DT, W> &w0, const Vec<DT, W> &w1,
                                          bool weighted, const float2 *row, const Place<W> &l, float inv_d, float eps) {
  float f[W], g[W], sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  p.get(f);
  q.get(g);
#pragma unroll
  for (int e = 0; e < W; ++e) {
    sum[e & 1] = __fmaf_rn(f[e], f[e], sum[e & 1]);
    sum[2 + (e & 1)] = __fmaf_rn(g[e], g[e], sum[2 + (e & 1)]);
  }
  const float all = head_sum(__fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])), l.lanes, l.piece, l.top);
  if (weighted) {
    float u[W];
    w0.get(u);
#pragma unroll
    for (int e = 0; e < W; ++e) f[e] = __fmul_rn(f[e], u[e]);
    w1.get(u);
#pragma unroll
    for (int e = 0; e < W; ++e) g[e] = __fmul_rn(g[e], u[e]);
  }
  if (l.half) {
    const float4 *cs = reinterpret_cast<const float4 *>(row + l.o0);
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float4 t = cs[e / 2];
      turn(f[e], g[e], t.x, t.y);
      turn(f[e + 1], g[e + 1], t.z, t.w);
    }
  }
  if (l.first) {
    const float4 *cs = reinterpret_cast<const float4 *>(row + l.o0 / 2);
#pragma unroll
    for (int e = 0; e < W; e += 4) {
      const float4 t = cs[e / 4];
      turn(f[e], f[e + 1], t.x, t.y);
      turn(f[e + 2], f[e + 3], t.z, t.w);
    }
  }
  if (l.second) {
    const float4 *cs = reinterpret_cast<const float4 *>(row + l.o1 / 2);
#pragma unroll
    for (int e = 0; e < W; e += 4) {
      const float4 t = cs[e / 4];
      turn(g[e], g[e + 1], t.x, t.y);
      turn(g[e + 2], g[e + 3], t.z, t.w);
    }
  }
  const float r = rsqrtf(__fmaf_rn(all, inv_d, eps));
#pragma unroll
  for (int e = 0; e < W; ++e) f[e] = __fmul_rn(f[e], r), g[e] = __fmul_rn(g[e], r);
  p.set(f);
  q.set(g);
}

// Offset of a token of a segment from its destination's start, and its table
// row, -1 where there is none; an offset of -1: it is skipped.
__device__ __forceinline__ void route(const RopeArgs &a, const RopeSeg &s, int64_t t, bool tell, int64_t &off, int &row) {
  const int64_t slot = s.paged ? a.slots[t] : 0;
  const bool turned = s.rot || (s.paged && a.rot);
  row = turned ? a.positions[t] : -1;
  off = -1;
  if (slot < 0) return;
  if (slot >= a.num_slots && s.paged) {
    if (tell) set_status(a.status, WQ_ERR_INDEX);
    return;
  }
  if (turned && unsigned(row) >= unsigned(a.max_pos)) {
    if (tell) set_status(a.status, WQ_ERR_INDEX);
    return;
  }
  if (!s.paged) {
    off = t * s.d_token;
    return;
  }
  // a division of 64 bits takes as long as all the rest of a lane's work
  const int64_t page = slot >> 32 ? slot / a.page_size : int64_t(uint32_t(slot) / uint32_t(a.page_size));
  off = page * s.d_page + (slot - page * a.page_size) * s.d_token;
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
  int64_t off;
  int row;
  route(a, s, t, (threadIdx.x & 31) == 0, off, row);
  if (off < 0) return;  // the same for the whole warp
  if (h.norm[l.i])
    norm_turn<DT>(p, q, w0, w1, weight != nullptr,
                  reinterpret_cast<const float2 *>(a.table) + int64_t(max(row, 0)) * (a.rot / 2), l, h.inv_d[l.i], h.eps);
  Raw *d = static_cast<Raw *>(s.dst) + off + l.head0 * s.d_head;
  if (on) p.store(d + l.o0);
  if (on && l.two) q.store(d + l.o1);
}

// Many tokens: a warp keeps its place and walks over the tokens.  Its lanes
// copy their own vectors of the tokens to come, and the tokens' table rows
// together, into shared memory.  Where 32 tokens go and which rows they take is
// found by a lane each, so that neither the chain of loads (slot or position,
// page or row) nor the divisions stand in a token's way.  (8191 tokens: a warp a
// token 83 us, walking with slot, position and row one token ahead 59, so 45.)
constexpr int STAGES = 3;
template <class DT, int KH>
__global__ void __launch_bounds__(256, 3) head_norm_stream_kernel(const __grid_constant__ HeadNormArgs h,
                                                                  const __grid_constant__ Cut cut) {
  using Raw = typename DT::Raw;
  constexpr int W = DT::kVec;
  using V = Vec<DT, W>;
  extern __shared__ uint4 ring[];  // [STAGES][2 KH][threads], then [warps][STAGES] table rows
  const RopeArgs &a = h.r;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, own_token = warp / cut.per_token;
  const int rest = int(blockIdx.y) * 8 + warp - own_token * cut.per_token;
  const int64_t t0 = int64_t(blockIdx.x) * cut.tokens + own_token, by = int64_t(gridDim.x) * cut.tokens;
  if (t0 >= a.T || rest >= cut.per_token) return;  // whole warps
  const Place<W> l(h, cut, rest, KH);
  const RopeSeg &s = a.seg[l.i];
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
  const int threads = int(blockDim.x), pieces = h.norm[l.i] ? s.rot / 4 : 0;  // of a table row
  uint4 *rows = ring + STAGES * 2 * KH * threads + warp * STAGES * (a.rot / 4);
  const Raw *src = static_cast<const Raw *>(s.src);
  auto to_smem = [](const uint4 *p) { return uint32_t(__cvta_generic_to_shared(p)); };
#pragma unroll 1
  for (int64_t first = t0; first < a.T; first += 32 * by) {
    // lane j: the j-th token from here on
    const int64_t ahead = (a.T - first + by - 1) / by;
    const int n = int(ahead < 32 ? ahead : 32);
    int64_t off = -1;
    int row = -1;
    if (lane < n) route(a, s, first + lane * by, true, off, row);
    int in = 0;
    auto copy = [&](int k) {
      if (k < n) {
        const int r = __shfl_sync(0xffffffffu, row, k);
        const Raw *x = src + (first + k * by) * s.s_token + l.head0 * s.s_head;
        uint4 *to = ring + in * 2 * KH * threads + threadIdx.x;
#pragma unroll
        for (int e = 0; e < KH; ++e) {
          if (on[e]) {
            cp16(to_smem(to + 2 * e * threads), x + e * l.side * s.s_head + l.o0, true);
            if (l.two) cp16(to_smem(to + (2 * e + 1) * threads), x + e * l.side * s.s_head + l.o1, true);
          }
        }
        if (unsigned(r) < unsigned(a.max_pos)) {
          const float4 *from = reinterpret_cast<const float4 *>(a.table) + int64_t(r) * (a.rot / 4);
          for (int e = lane; e < pieces; e += 32) cp16(to_smem(rows + in * (a.rot / 4) + e), from + e, true);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      in = in == STAGES - 1 ? 0 : in + 1;
    };
    __syncwarp();
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy(k);
    int out = 0;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      __syncwarp();  // the row that the next copies replace has been read
      copy(k + STAGES - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      __syncwarp();
      const int64_t at = __shfl_sync(0xffffffffu, off, k);
      if (at >= 0) {
        Raw *to = static_cast<Raw *>(s.dst) + at + l.head0 * s.d_head;
        const uint4 *from = ring + out * 2 * KH * threads + threadIdx.x;
        const float2 *turns = reinterpret_cast<const float2 *>(rows + out * (a.rot / 4));
#pragma unroll
        for (int e = 0; e < KH; ++e) {
          if (__all_sync(0xffffffffu, !on[e])) break;
          V p, q;
          p.w = q.w = make_uint4(0, 0, 0, 0);
          if (on[e]) p.w = from[2 * e * threads];
          if (on[e] && l.two) q.w = from[(2 * e + 1) * threads];
          if (h.norm[l.i]) norm_turn<DT>(p, q, w0, w1, weight != nullptr, turns, l, h.inv_d[l.i], h.eps);
          if (on[e]) p.store(to + e * l.side * s.d_head + l.o0);
          if (on[e] && l.two) q.store(to + e * l.side * s.d_head + l.o1);
        }
      }
      out = out == STAGES - 1 ? 0 : out + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
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
    const int smem = STAGES * (2 * KH * threads * 16 + threads / 32 * h.r.rot * 4);
    static OncePerDevice sized;
    if (!allow_smem(sized, k, STAGES * (2 * KH * 256 * 16 + 8 * 512 * 4))) return WQ_ERR_LAUNCH;
    const int64_t most = std::max<int64_t>(1, 3 * 152 / y);  // three blocks an SM
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
  // Walks over tokens once each of three blocks an SM has several: 700,000 lanes.
  // Heads of 128, us a warp a token and walking: 40 heads bf16, 1024 tokens (328,000
  // lanes) 7.8 and 8.1, 2048 (655,000) 12.5 and 11.9, 4096 23 and 20, 16384 94 and
  // 72; float32, 1024 tokens (655,000) 9.9 and 10.7, 2048 18.1 and 17.7, 8192 73 and
  // 64; 8 heads bf16, 2048 tokens (131,000) 4.2 and 4.8, 16384 (1,049,000) 17.2 and 15.6.
  if (vec) return lanes > 2 * 3 * 152 * 256 * 3 ? launch_vec<DT, true>(h, st) : launch_vec<DT, false>(h, st);
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
