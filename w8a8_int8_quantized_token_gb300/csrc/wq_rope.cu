// Rotary positions and the rotated append to a paged cache.
//
// One launch walks up to three tensors of heads (queries, keys, values).  The
// unit of a thread is 16 elements of a head: 8 pairs (two 16-byte vectors half
// a rotation apart in the half layout, 16 consecutive elements in the
// interleaved one), or 16 elements to copy; with many tokens a thread takes
// the same unit of up to four heads, whose loads are in flight together and
// which share the unit's part of the table row.  Bound by HBM: every element
// read once and written once; the table rows come from L2.  4096 tokens x 128
// heads x 64 bf16 take 31 us, 4.4 TB/s.
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

// Table row of token t, nullptr if its position is outside the table
__device__ __forceinline__ const float2 *row_of(const RopeArgs &a, int64_t t, bool tell) {
  const int p = a.positions[t];
  if (p < 0 || p >= a.max_pos) {
    if (tell) set_status(a.status, WQ_ERR_INDEX);
    return nullptr;
  }
  return reinterpret_cast<const float2 *>(a.table) + int64_t(p) * (a.rot / 2);
}

__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
  const float u = __fmaf_rn(x, c, -__fmul_rn(y, s));
  y = __fmaf_rn(y, c, __fmul_rn(x, s));
  x = u;
}

// Units of one head: rot / 16 rotated ones, then the rest in copies of 16
__host__ __device__ inline int units_of(const RopeSeg &s) {
  return s.rot / 16 + (s.D - s.rot / 16 * 16 + 15) / 16;
}

// Threads that share a segment's token: a unit of KH heads each
template <int KH>
__host__ __device__ inline int threads_of(const RopeSeg &s) {
  return (s.heads + KH - 1) / KH * units_of(s);
}

// A thread's token and its place among the token's threads: blocks of whole
// tokens, or (y) a token's threads in blocks of 256
__device__ __forceinline__ bool place_of(const RopeArgs &a, int per_token, int64_t &t, int &rest) {
  if (per_token >= 256) {
    t = blockIdx.x;
    rest = int(blockIdx.y * 256 + threadIdx.x);
    return rest < per_token;
  }
  const int tokens = 256 / per_token, own = int(threadIdx.x) / per_token;
  t = int64_t(blockIdx.x) * tokens + own;
  rest = int(threadIdx.x) - own * per_token;
  return own < tokens && t < a.T;
}
inline dim3 grid_of(const RopeArgs &a, int per_token) {
  const int tokens = per_token >= 256 ? 1 : 256 / per_token;
  return dim3(unsigned((a.T + tokens - 1) / tokens), unsigned(per_token >= 256 ? (per_token + 255) / 256 : 1));
}

template <class DT, int KH>
__global__ void __launch_bounds__(256) rope_vec_kernel(const RopeArgs a, int per_token) {
  using Raw = typename DT::Raw;
  using V = Vec<DT, 8>;
  int64_t t;
  int rest;
  if (!place_of(a, per_token, t, rest)) return;
  int i = 0;
  while (rest >= threads_of<KH>(a.seg[i])) rest -= threads_of<KH>(a.seg[i]), ++i;
  const RopeSeg &s = a.seg[i];
  const int units = units_of(s), groups = (s.heads + KH - 1) / KH;
  const int head0 = rest / units, piece = rest - head0 * units;  // heads head0 + k * groups
  Raw *d = dst_of<Raw>(a, s, t, rest == 0);
  if (!d) return;
  const float2 *row = nullptr;
  if ((s.rot || (s.paged && a.rot)) && !(row = row_of(a, t, rest == 0))) return;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token;
  const bool half = piece < s.rot / 16 && a.layout == WQ_ROPE_HALF;
  const int o0 = half ? piece * 8 : piece * 16, o1 = half ? o0 + s.rot / 2 : o0 + 8;
  const bool two = o1 < s.D;
  // pairs of the first and of the second vector that turn
  const int first = half ? 8 : (a.layout == WQ_ROPE_INTERLEAVED && o0 < s.rot ? 4 : 0);
  const int second = !half && a.layout == WQ_ROPE_INTERLEAVED && o1 < s.rot ? 4 : 0;
  V p[KH], q[KH];
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int head = head0 + k * groups;
    if (head >= s.heads) break;
    p[k] = V::load(x + head * s.s_head + o0);
    if (two) q[k] = V::load(x + head * s.s_head + o1);
  }
  float c[8], n[8];  // cos and sin of the unit's pairs
  if (first) {
    const float2 *r = row + (half ? o0 : o0 / 2);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      if (e < 4 || half || second) {
        const float4 w = *reinterpret_cast<const float4 *>(r + e);
        c[e] = w.x;
        n[e] = w.y * a.sign;
        c[e + 1] = w.z;
        n[e + 1] = w.w * a.sign;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int head = head0 + k * groups;
    if (head >= s.heads) break;
    if (first) {
      float f[8], g[8];
      p[k].get(f);
      q[k].get(g);
      if (half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn(f[e], g[e], c[e], n[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) turn(f[2 * e], f[2 * e + 1], c[e], n[e]);
        if (second) {
#pragma unroll
          for (int e = 0; e < 4; ++e) turn(g[2 * e], g[2 * e + 1], c[4 + e], n[4 + e]);
        }
      }
      p[k].set(f);
      if (half || second) q[k].set(g);
    }
    p[k].store(d + head * s.d_head + o0);
    if (two) q[k].store(d + head * s.d_head + o1);
  }
}

// Any size, pitch and alignment: a thread per pair or copied element
template <class DT>
__global__ void __launch_bounds__(256) rope_any_kernel(const RopeArgs a, int per_token) {
  using Raw = typename DT::Raw;
  int64_t t;
  int rest;
  if (!place_of(a, per_token, t, rest)) return;
  int i = 0;
  while (rest >= a.seg[i].heads * (a.seg[i].D - a.seg[i].rot / 2))
    rest -= a.seg[i].heads * (a.seg[i].D - a.seg[i].rot / 2), ++i;
  const RopeSeg &s = a.seg[i];
  const int units = s.D - s.rot / 2, head = rest / units, piece = rest - head * units;
  Raw *d = dst_of<Raw>(a, s, t, rest == 0);
  if (!d) return;
  const float2 *row = nullptr;
  if ((s.rot || (s.paged && a.rot)) && !(row = row_of(a, t, rest == 0))) return;
  d += head * s.d_head;
  const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + head * s.s_head;
  if (piece >= s.rot / 2) {
    d[piece + s.rot / 2] = x[piece + s.rot / 2];
    return;
  }
  const int o0 = a.layout == WQ_ROPE_HALF ? piece : 2 * piece;
  const int o1 = a.layout == WQ_ROPE_HALF ? piece + s.rot / 2 : o0 + 1;
  float f = DT::to_f(x[o0]), g = DT::to_f(x[o1]);
  turn(f, g, row[piece].x, row[piece].y * a.sign);
  d[o0] = DT::from_f(f);
  d[o1] = DT::from_f(g);
}

// Angles in float64: a float32 angle is off by 2^-8 at position 65536.
// Runs once when a program starts.
__global__ void rope_table_kernel(float2 *table, int64_t n, int half, double log_base, int yarn,
                                  double factor, double lo, double hi, double m) {
  for (int64_t u = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; u < n;
       u += int64_t(gridDim.x) * blockDim.x) {
    const int64_t p = u / half;
    const int i = int(u - p * half);
    double f = exp(-log_base * i / half);
    if (yarn) {
      const double keep = 1.0 - fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
      f = f * (keep + (1.0 - keep) / factor);
    } else {
      f = f / factor;
    }
    double s, c;
    sincos(double(p) * f, &s, &c);
    table[u] = make_float2(float(m * c), float(m * s));
  }
}

template <class DT, int KH>
int launch_vec(const RopeArgs &a, cudaStream_t st) {
  int per_token = 0;
  for (int i = 0; i < a.nseg; ++i) per_token += threads_of<KH>(a.seg[i]);
  if (per_token == 0) return WQ_OK;
  const dim3 grid = grid_of(a, per_token);
  if (grid.y > 65535) return WQ_ERR_UNSUPPORTED;
  rope_vec_kernel<DT, KH><<<grid, 256, 0, st>>>(a, per_token);
  return launched(1);
}

template <class DT>
int launch_t(const RopeArgs &a, bool vec, cudaStream_t st) {
  if constexpr (DT::kVec == 8) {
    // four heads a thread once that leaves each SM a few blocks
    int64_t units = 0;
    for (int i = 0; i < a.nseg; ++i) units += a.T * a.seg[i].heads * units_of(a.seg[i]);
    if (vec) return units > 4 * 256 * 152 * 4 ? launch_vec<DT, 4>(a, st) : launch_vec<DT, 1>(a, st);
  }
  const int per_token = int(rope_pair_threads(a));  // at most kRopeMostThreads
  if (per_token == 0) return WQ_OK;
  const dim3 grid = grid_of(a, per_token);
  rope_any_kernel<DT><<<grid, 256, 0, st>>>(a, per_token);
  return launched(1);
}

}  // namespace

int launch_rope(const RopeArgs &a, int dtype, bool vec, cudaStream_t st) {
  switch (dtype) {
    case WQ_DT_BF16: return launch_t<Bf16>(a, vec, st);
    case WQ_DT_F16: return launch_t<F16>(a, vec, st);
    default: return launch_t<F32>(a, false, st);
  }
}

int launch_rope_table(float *table, int64_t max_pos, int rot, double base, int scaling,
                      double factor, double trained, double beta_fast, double beta_slow,
                      double mscale, cudaStream_t st) {
  const int half = rot / 2;
  double log_base = log(base), lo = 0.0, hi = 1.0, m = 1.0, div = 1.0;
  if (scaling == WQ_ROPE_LINEAR) div = factor;
  if (scaling == WQ_ROPE_NTK) log_base += log(factor) * rot / (rot - 2.0);
  if (scaling == WQ_ROPE_YARN) {
    // the pair whose wave length fits n turns into the trained context
    auto pair_of = [&](double n) {
      return rot * log(trained / (n * 2.0 * 3.14159265358979323846)) / (2.0 * log_base);
    };
    lo = fmax(floor(pair_of(beta_fast)), 0.0);
    hi = fmin(ceil(pair_of(beta_slow)), rot - 1.0);
    if (lo == hi) hi += 0.001;
    m = mscale > 0.0 ? mscale : (factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0);
    div = factor;
  }
  const int64_t n = max_pos * half, blocks = (n + 255) / 256;
  rope_table_kernel<<<unsigned(blocks < 65535 ? blocks : 65535), 256, 0, st>>>(
      reinterpret_cast<float2 *>(table), n, half, log_base, scaling == WQ_ROPE_YARN, div, lo, hi, m);
  return launched(1);
}

}  // namespace wq
