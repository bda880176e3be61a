// Eviction from a paged cache by accumulated attention weight.
//
// Of a sequence's n > budget keys, head by head, the first and the most recent
// ones stay, and the heaviest of those between.  Two kernels:
//
// evict_select_kernel, a block per (sequence, head): the weights' bits are
// mapped to unsigned keys of the same order, and the key of the last one that
// stays is found digit by digit from the top (11, 11 and 10 bits: a histogram
// in shared memory and a scan over its bins for each).  Then every warp counts
// the larger and the equal keys of its own stretch, a scan over the warps gives
// each its place, and the places that stay are written in order; of equal keys
// the first stay.  Counts do not depend on the order of the atomics that take
// them.
//
// evict_move_kernel packs the rows that stay, in their order.  A row goes to a
// place at or before its own, so in place no row may be written before all
// rows at or before its place are read.  A block therefore owns some columns of
// all rows of a (sequence, head) and walks them in order: it reads a stretch of
// rows, waits for all its threads, and writes it, with the next stretch's reads
// in flight; later stretches lie behind everything that it writes.  Columns of
// a row, keys, values and weights are independent and go to different blocks.
// Into other pages any block may take any rows.  Bound by HBM: rows that move
// are read once and written once.
#include <algorithm>

#include "wq_attn.cuh"
#include "wq_serve.cuh"

namespace wq {
namespace {

using attn::launch_chained;
using attn::start_next_kernel;
using attn::wait_last_kernel;

constexpr int NT = 1024, NW = NT / 32;  // threads, warps of the selection
constexpr int BINS = 2048;

// Unsigned key in the order of the weights: -0 as 0, NaN below everything
__device__ __forceinline__ uint32_t key_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Keys of sequence b
__device__ __forceinline__ int length_of(const EvictArgs &a, int b) {
  return min(max(a.key_len[b], 0), a.max_len);
}

// Inclusive sum over the block's threads, and its total
__device__ __forceinline__ int block_scan(int v, int *part, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  __syncthreads();
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int p = lane < NW ? part[lane] : 0;
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xffffffffu, p, o);
    if (lane >= o) p += w;
  }
  total = __shfl_sync(0xffffffffu, p, 31);
  const int before = __shfl_sync(0xffffffffu, p, max(warp - 1, 0));
  return v + (warp ? before : 0);
}

// STAGED: the weights between the first and the recent keys fit shared memory
template <bool STAGED>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictArgs a) {
  extern __shared__ float staged[];
  __shared__ int hist[BINS];
  __shared__ int part[NW], found[2];
  const int b = int(blockIdx.x) / a.heads, h = int(blockIdx.x) - b * a.heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  start_next_kernel();
  const int n = length_of(a, b), fresh = min(n, a.budget);
  if (h == 0 && threadIdx.x == 0) {
    a.new_len[b] = fresh;
    if (n != a.key_len[b]) set_status(a.status, WQ_ERR_INDEX);
  }
  const float *w = a.w + b * a.w_seq + h * a.w_head;
  int32_t *kept = a.kept + (int64_t(b) * a.heads + h) * a.budget;
  int2 *map = a.map + (int64_t(b) * a.heads + h) * a.budget;
  // key i goes to place j
  const bool moves = !a.in_place || n > a.budget;
  auto emit = [&](int j, int i) {
    kept[j] = i;
    if (moves) {
      const int at = i / a.page_size, page = a.page_table[b * a.ld_table + at];
      const bool good = unsigned(page) < unsigned(a.num_pages);
      if (!good) set_status(a.status, WQ_ERR_INDEX);
      map[j] = make_int2(good ? page : -1, i - at * a.page_size);
    }
  };
  for (int j = fresh + threadIdx.x; j < a.budget; j += NT) kept[j] = -1;
  if (n <= a.budget) {
    for (int j = threadIdx.x; j < n; j += NT) emit(j, j);
    return;
  }
  const int lo = a.first, hi = n - a.recent, mid = hi - lo;
  for (int j = threadIdx.x; j < lo; j += NT) emit(j, j);
  for (int j = threadIdx.x; j < a.recent; j += NT) emit(a.budget - a.recent + j, hi + j);
  int need = a.budget - a.first - a.recent;  // of the mid keys, fewer than all
  if (need == 0) return;
  auto at = [&](int i) { return key_of(STAGED ? staged[i] : w[lo + i]); };
  uint32_t prefix = 0;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
    for (int i = threadIdx.x; i < BINS; i += NT) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < mid; i += NT) {
      uint32_t k;
      if (STAGED && digit == 0) {
        const float f = w[lo + i];
        staged[i] = f;
        k = key_of(f);
      } else {
        k = at(i);
      }
      if (digit == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
    }
    __syncthreads();
    // bins from the top: thread t has the t-th pair
    const int top = BINS - 1 - 2 * int(threadIdx.x), h1 = hist[top], h0 = hist[top - 1];
    int total;
    const int upto = block_scan(h0 + h1, part, total);
    const int above = upto - h0 - h1;
    if (above < need && need <= upto) {  // one thread
      const bool upper = need <= above + h1;
      found[0] = upper ? top : top - 1;
      found[1] = need - (upper ? above : above + h1);
    }
    __syncthreads();
    prefix = digit == 0 ? uint32_t(found[0]) : (prefix << bits) | uint32_t(found[0]);
    need = found[1];  // of the keys that begin with prefix
  }
  // keys above `prefix` stay, and the first `need` of those equal to it
  const int stretch = ((mid + NW - 1) / NW + 31) / 32 * 32;
  const int s0 = min(warp * stretch, mid), s1 = min(s0 + stretch, mid);
  int more = 0, same = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    const uint32_t k = at(i);
    more += k > prefix;
    same += k == prefix;
  }
  for (int o = 16; o > 0; o >>= 1) {
    more += __shfl_xor_sync(0xffffffffu, more, o);
    same += __shfl_xor_sync(0xffffffffu, same, o);
  }
  __syncthreads();
  if (lane == 0) hist[warp] = more, hist[NW + warp] = same;
  __syncthreads();
  int j = lo, equal = 0;
  for (int v = 0; v < warp; ++v) j += hist[v], equal += hist[NW + v];
  j += min(equal, need);
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < s1 ? at(i) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, i < s1 && k == prefix), below = (1u << lane) - 1u;
    const bool stays = i < s1 && (k > prefix || (k == prefix && equal + __popc(eq & below) < need));
    const uint32_t st = __ballot_sync(0xffffffffu, stays);
    if (stays) emit(j + __popc(st & below), lo + i);
    j += __popc(st);
    equal += __popc(eq);
  }
}

// One tensor's columns that a block moves
template <class V>
__device__ __forceinline__ void move_rows(const EvictArgs &a, const V *src, V *dst, int64_t s_page, int64_t s_row,
                                          int64_t d_page, int64_t d_row, int c0, int cols, int b, int h, int rows,
                                          int rb) {
  constexpr int U = 4;
  const int side = 256 / cols, row = int(threadIdx.x) / cols, col = c0 + int(threadIdx.x) - row * cols;
  const bool live = row < side;
  const int R = side * U;
  const int2 *map = a.map + (int64_t(b) * a.heads + h) * a.budget;
  const int32_t *kept = a.kept + (int64_t(b) * a.heads + h) * a.budget;
  const int32_t *out = a.out_table + b * a.ld_out;
  V v[U], x[U];
  bool on[U], nx[U];
  auto load = [&](int j0, V(&to)[U], bool(&is)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * side + row;
      is[u] = false;
      if (!live || j >= rows) continue;
      const int2 m = map[j];
      is[u] = m.x >= 0 && !(a.in_place && kept[j] == j);
      if (is[u]) to[u] = src[m.x * s_page + m.y * s_row + col];
    }
  };
  const int step = R * a.row_blocks;
  load(rb * R, v, on);
  for (int j0 = rb * R; j0 < rows; j0 += step) {
    load(j0 + step, x, nx);
    if (a.in_place) __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (on[u]) {
        const int j = j0 + u * side + row, at = j / a.page_size, page = out[at];
        if (unsigned(page) < unsigned(a.num_pages)) dst[page * d_page + (j - at * a.page_size) * d_row + col] = v[u];
        else set_status(a.status, WQ_ERR_INDEX);
      }
      on[u] = nx[u];
      v[u] = x[u];
    }
  }
}

template <class V>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  constexpr int E = sizeof(V) / 2;  // elements of a vector
  const int bh = int(blockIdx.x / unsigned(a.row_blocks)), rb = int(blockIdx.x % unsigned(a.row_blocks));
  const int b = bh / a.heads, h = bh - b * a.heads;
  const int n = length_of(a, b), rows = min(n, a.budget);
  wait_last_kernel();  // in every block: what follows may rely on the selection too
  if (a.in_place && n <= a.budget && a.w_out == a.w) return;
  int part = int(blockIdx.y);
  if (part == 0) {  // weights
    const int blocks = a.w_out == a.w ? 1 : a.row_blocks;  // one walk in place
    if (rb >= blocks) return;
    const float *w = a.w + b * a.w_seq + h * a.w_head;
    float *to = a.w_out + b * a.o_seq + h * a.o_head;
    const int32_t *kept = a.kept + (int64_t(b) * a.heads + h) * a.budget;
    constexpr int U = 4;
    float v[U], x[U];
    const int step = 256 * U * blocks;
    auto load = [&](int j0, float(&t)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * 256 + int(threadIdx.x);
        if (j < rows) t[u] = w[kept[j]];
      }
    };
    load(rb * 256 * U, v);
    for (int j0 = rb * 256 * U; j0 < rows; j0 += step) {
      load(j0 + step, x);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = j0 + u * 256 + int(threadIdx.x);
        if (j < rows) to[j] = v[u];
        v[u] = x[u];
      }
    }
    return;
  }
  if (a.in_place && n <= a.budget) return;
  --part;
  if (part < a.k_parts) {
    const int per = (a.dk / E + a.k_parts - 1) / a.k_parts, c0 = part * per, cols = min(per, a.dk / E - c0);
    if (cols > 0)
      move_rows<V>(a, reinterpret_cast<const V *>(a.k + h * a.k_head), reinterpret_cast<V *>(a.k + h * a.k_head),
                   a.k_page / E, a.k_token / E, a.k_page / E, a.k_token / E, c0, cols, b, h, rows, rb);
  } else {
    part -= a.k_parts;
    const int per = (a.dv / E + a.v_parts - 1) / a.v_parts, c0 = part * per, cols = min(per, a.dv / E - c0);
    if (cols > 0)
      move_rows<V>(a, reinterpret_cast<const V *>(a.v + h * a.v_head), reinterpret_cast<V *>(a.v + h * a.v_head),
                   a.v_page / E, a.v_token / E, a.v_page / E, a.v_token / E, c0, cols, b, h, rows, rb);
  }
}

template <class V>
int launch_move(EvictArgs a, cudaStream_t st) {
  constexpr int E = sizeof(V) / 2;
  const int64_t bh = int64_t(a.B) * a.heads;
  // Columns in place: four blocks for keys and four for values at least, since
  // most sequences of a batch may have nothing to move; 32 bytes or more each.
  auto parts = [&](int cols) {
    const int64_t least = (cols + 255) / 256, most = std::max<int64_t>(least, cols * int64_t(sizeof(V)) / 32);
    return int(a.in_place ? std::min(std::max<int64_t>({least, 4, 2432 / bh}), most) : least);
  };
  a.k_parts = parts(a.dk / E);
  a.v_parts = parts(a.dv / E);
  // Into other pages: rows of a (sequence, head) over several blocks
  const int64_t side = std::max(1, 256 / std::max(std::min(a.dk, a.dv) / E, 1)) * 4;
  a.row_blocks = int(a.in_place ? 1 : std::min((a.budget + side - 1) / side, std::max<int64_t>(1, 4864 / (2 * bh))));
  if (bh * a.row_blocks >= (int64_t(1) << 31) || a.k_parts + a.v_parts >= 65535) return WQ_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(bh * a.row_blocks), unsigned(1 + a.k_parts + a.v_parts));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_move_kernel<V>, a) != cudaSuccess) return WQ_ERR_LAUNCH;
  return launched(1);
}

constexpr int kStaged = 48 * 1024;  // weights that shared memory holds

}  // namespace

int launch_evict(const EvictArgs &a, bool vec, cudaStream_t st) {
  const int64_t bh = int64_t(a.B) * a.heads;
  if (bh >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  if (a.max_len <= kStaged) {
    static OncePerDevice sized;
    if (!allow_smem(sized, evict_select_kernel<true>, kStaged * 4)) return WQ_ERR_LAUNCH;
    evict_select_kernel<true><<<unsigned(bh), NT, size_t(a.max_len) * 4, st>>>(a);
  } else {
    evict_select_kernel<false><<<unsigned(bh), NT, 0, st>>>(a);
  }
  const int rc = launched(1);
  if (rc != WQ_OK) return rc;
  return vec ? launch_move<uint4>(a, st) : launch_move<uint16_t>(a, st);
}

}  // namespace wq
