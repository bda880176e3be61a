// Rotary positions and the rotated append to a paged cache.
//
// One launch walks up to three tensors of heads (queries, keys, values).  The
// unit of a thread is 16 elements of one head: 8 pairs (two 16-byte vectors
// half a rotation apart in the half layout, 16 consecutive elements in the
// interleaved one), or 16 elements to copy.  Bound by HBM: every element read
// once and written once; the table rows come from L2.
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

__device__ __forceinline__ void turn(float &x, float &y, float2 cs, float sign) {
  const float s = __fmul_rn(cs.y, sign);
  const float u = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, s));
  x = u;
}

// Units of one head: rot / 16 rotated ones, then the rest in copies of 16
__host__ __device__ inline int units_of(const RopeSeg &s) {
  return s.rot / 16 + (s.D - s.rot / 16 * 16 + 15) / 16;
}

template <class DT>
__global__ void rope_vec_kernel(const RopeArgs a, int per_token) {
  using Raw = typename DT::Raw;
  using V = Vec<DT, 8>;
  const int64_t n = a.T * per_token;
  for (int64_t u = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; u < n;
       u += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = u / per_token;
    int rest = int(u - t * per_token), i = 0;
    while (rest >= a.seg[i].heads * units_of(a.seg[i])) rest -= a.seg[i].heads * units_of(a.seg[i]), ++i;
    const RopeSeg &s = a.seg[i];
    const int units = units_of(s), head = rest / units, piece = rest - head * units;
    Raw *d = dst_of<Raw>(a, s, t, rest == 0);
    if (!d) continue;
    const float2 *row = nullptr;
    if ((s.rot || (s.paged && a.rot)) && !(row = row_of(a, t, rest == 0))) continue;
    d += head * s.d_head;
    const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + head * s.s_head;
    const int nrot = s.rot / 16;
    if (piece < nrot && a.layout == WQ_ROPE_HALF) {
      const int o0 = piece * 8, o1 = o0 + s.rot / 2;
      V p = V::load(x + o0), q = V::load(x + o1);
      float f[8], g[8];
      p.get(f);
      q.get(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) turn(f[e], g[e], row[o0 + e], a.sign);
      p.set(f);
      q.set(g);
      p.store(d + o0);
      q.store(d + o1);
      continue;
    }
    const int o0 = piece * 16;  // 16 consecutive elements, rotated below rot
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int o = o0 + 8 * v;
      if (o >= s.D) break;
      V p = V::load(x + o);
      if (a.layout == WQ_ROPE_INTERLEAVED && o < s.rot) {
        float f[8];
        p.get(f);
#pragma unroll
        for (int e = 0; e < 8; e += 2) turn(f[e], f[e + 1], row[(o + e) / 2], a.sign);
        p.set(f);
      }
      p.store(d + o);
    }
  }
}

// Any size, pitch and alignment: a thread per pair or copied element
template <class DT>
__global__ void rope_any_kernel(const RopeArgs a, int per_token) {
  using Raw = typename DT::Raw;
  const int64_t n = a.T * per_token;
  for (int64_t u = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; u < n;
       u += int64_t(gridDim.x) * blockDim.x) {
    const int64_t t = u / per_token;
    int rest = int(u - t * per_token), i = 0;
    while (rest >= a.seg[i].heads * (a.seg[i].D - a.seg[i].rot / 2))
      rest -= a.seg[i].heads * (a.seg[i].D - a.seg[i].rot / 2), ++i;
    const RopeSeg &s = a.seg[i];
    const int units = s.D - s.rot / 2, head = rest / units, piece = rest - head * units;
    Raw *d = dst_of<Raw>(a, s, t, rest == 0);
    if (!d) continue;
    const float2 *row = nullptr;
    if ((s.rot || (s.paged && a.rot)) && !(row = row_of(a, t, rest == 0))) continue;
    d += head * s.d_head;
    const Raw *x = static_cast<const Raw *>(s.src) + t * s.s_token + head * s.s_head;
    if (piece >= s.rot / 2) {
      d[piece + s.rot / 2] = x[piece + s.rot / 2];
      continue;
    }
    const int o0 = a.layout == WQ_ROPE_HALF ? piece : 2 * piece;
    const int o1 = a.layout == WQ_ROPE_HALF ? piece + s.rot / 2 : o0 + 1;
    float f = DT::to_f(x[o0]), g = DT::to_f(x[o1]);
    turn(f, g, row[piece], a.sign);
    d[o0] = DT::from_f(f);
    d[o1] = DT::from_f(g);
  }
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

template <class DT>
int launch_t(const RopeArgs &a, bool vec, cudaStream_t st) {
  int per_token = 0;
  for (int i = 0; i < a.nseg; ++i)
    per_token += a.seg[i].heads * (vec ? units_of(a.seg[i]) : a.seg[i].D - a.seg[i].rot / 2);
  if (per_token == 0) return WQ_OK;
  const int64_t blocks = (a.T * per_token + 255) / 256;
  const unsigned grid = unsigned(blocks < (1 << 20) ? blocks : (1 << 20));
  if (vec) {
    if constexpr (DT::kVec == 8) rope_vec_kernel<DT><<<grid, 256, 0, st>>>(a, per_token);
  } else {
    rope_any_kernel<DT><<<grid, 256, 0, st>>>(a, per_token);
  }
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
