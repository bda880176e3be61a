// Eviction from a paged cache by accumulated attention weight.
//
// Of a sequence's n > budget keys, head by head, the first and the most recent
// ones stay, and the heaviest of those between.  Two kernels:
//
// evict_select_kernel, a cluster of blocks per (sequence, head), each with a
// stretch of the keys: the weights' bits are mapped to unsigned keys of the
// same order, and the key of the last one that stays is found digit by digit
// from the top.  A digit is a histogram in shared memory, whose bins are added
// over the cluster, and a scan over them.  As soon as few keys share the digits
// found so far, which is mostly after the first one, every block gathers them and
// goes on by itself, without the cluster's barriers, and ranks the last ones
// against one another.  Then every warp counts the larger and the equal
// keys of its own part, the counts before it give each its place, and the
// places that stay are written in order; of equal keys the first stay.  Neither
// counts nor ranks depend on the order of the atomics that take them.  Bound by
// latency: about ten steps with a barrier each (the cluster's between some).
// Both kernels take 22 us for 8 heads of 32768 keys, a block for 4096 of them
// (25 with the last 512 keys ranked and a second digit over the cluster before).
//
// evict_move_kernel packs the rows that stay, in their order.  A row goes to a
// place at or before its own, so in place no row may be written before all
// rows at or before its place are read.  A block therefore owns some columns of
// all rows of a (sequence, head) and walks them in order: it reads a stretch of
// rows, waits for all its threads, and writes it; later stretches lie behind
// everything that it writes.  Columns of a row, keys, values and weights are
// independent and go to different blocks.  Into other pages any block may take
// any rows.  Bound by HBM: rows that move are read once and written once; 8 heads
// of 4096 rows (17 MB read, 17 written) take 11 us with cold caches.  In place a
// block has 32 bytes of a row, which lets it read 1024 rows before it waits, and
// blocks may be left with a second walk while the others are done: 4 sequences of 8
// heads are 512 walks for 456 blocks (2 of 8 heads of 1900 rows, 16 MB read, take 15
// us).  All of 64 sequences that give 148 of 2048 keys back take 256 us with their
// selection (up to 996 MB, 3.9 TB/s).
#include <algorithm>

#include "wq_attn.cuh"
#include "wq_serve.cuh"
#include "wq_tc.cuh"

namespace wq {
namespace {

using attn::launch_chained;
using attn::start_next_kernel;
using attn::wait_last_kernel;

constexpr int NT = 512, NW = NT / 32;  // threads, warps of the selection
constexpr int BINS = 2048;
constexpr int FEW = 2048;              // keys that a block gathers
constexpr int LAST = 128;              // keys that are ranked against one another
constexpr int MOST_BLOCKS = 8;         // of a cluster

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

template <class T>
__device__ __forceinline__ const T *of_block(const T *p, int rank) {
  T *r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return r;
}

struct Shared {
  int hist[2][BINS];     // of digits in turn: a block may be a digit ahead of one that reads its bins
  uint32_t few[FEW];     // the block's keys with the digits found
  uint32_t all[FEW];     // the cluster's
  int2 counts;           // the block's larger keys, equal keys
  int part[NW], part2[NW];
  int taken, last, left, digit, need;
};
constexpr int STAGE_BYTES = 192 * 1024;  // of weights in shared memory, at most
static_assert(STAGE_BYTES + sizeof(Shared) <= 232448, "shared memory plan");

// STAGED: a block's stretch of the weights between the first and the recent
// keys fits shared memory
template <bool STAGED>
__global__ void __launch_bounds__(NT, 2) evict_select_kernel(const EvictArgs a, int C) {
  extern __shared__ float staged[];
  __shared__ Shared sm;
  const int cluster = int(blockIdx.x) / C, rank = int(blockIdx.x) - cluster * C;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (cluster == 0) {  // the sequences with rows to move, for the other kernel
    if (rank > 0) return;
    int count = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
      const int q = b0 + int(threadIdx.x), len = q < a.B ? length_of(a, q) : 0;
      const bool moves = a.in_place ? len > a.budget : len > 0;
      int total;
      const int upto = block_scan(int(moves), sm.part, total);
      if (moves) a.moving[count + upto] = q;
      count += total;
    }
    if (threadIdx.x == 0) a.moving[0] = count;
    return;
  }
  const int b = (cluster - 1) / a.heads, h = cluster - 1 - b * a.heads;
  const int n = length_of(a, b), fresh = min(n, a.budget);
  if (h == 0 && rank == 0 && threadIdx.x == 0) {
    a.new_len[b] = fresh;
    if (n != a.key_len[b]) set_status(a.status, WQ_ERR_INDEX);
  }
  const float *w = a.w + b * a.w_seq + h * a.w_head;
  const float *w_row = w;
  float *w_out = a.w_out == a.w ? nullptr : a.w_out + b * a.o_seq + h * a.o_head;
  int32_t *kept = a.kept + (int64_t(b) * a.heads + h) * a.budget;
  // What the other kernel needs to move key i to place j: pages and places,
  // found here once and not by every thread that has a piece of the row
  int4 *ways = a.ways + (int64_t(b) * a.heads + h) * a.budget;
  const int32_t *in = a.page_table + b * a.ld_table, *out = a.out_table + b * a.ld_out;
  auto find_way = [&](int j, int i) {
    const int p = i / a.page_size, q = j / a.page_size, from = in[p], to = out[q];
    const bool good = unsigned(from) < unsigned(a.num_pages) && unsigned(to) < unsigned(a.num_pages);
    if (!good) set_status(a.status, WQ_ERR_INDEX);
    const bool stands = a.in_place && i == j;  // its page is looked at all the same
    ways[j] = make_int4(good && !stands ? from : -1, i - p * a.page_size, to, j - q * a.page_size);
  };
  // key i goes to place j
  const bool moves = !a.in_place || n > a.budget;
  auto emit = [&](int j, int i) {
    kept[j] = i;
    if (w_out) w_out[j] = w_row[i];
    if (moves) find_way(j, i);
  };
  // the cluster's threads share what needs no order
  const int all0 = rank * NT + int(threadIdx.x), all = C * NT;
  for (int j = fresh + all0; j < a.budget; j += all) kept[j] = -1;
  if (n <= a.budget) {
    for (int j = all0; j < n; j += all) emit(j, j);
    if (!moves && h == 0) {  // nothing looks at its pages
      for (int p = all0; p < (n + a.page_size - 1) / a.page_size; p += all)
        if (unsigned(in[p]) >= unsigned(a.num_pages)) set_status(a.status, WQ_ERR_INDEX);
    }
    return;  // the whole cluster
  }
  const int first = a.first, mid = n - a.recent - first;
  for (int j = all0; j < first; j += all) emit(j, j);
  for (int j = all0; j < a.recent; j += all) emit(a.budget - a.recent + j, n - a.recent + j);
  int need = a.budget - first - a.recent;  // of the mid keys, fewer than all
  if (need == 0) return;
  // this block's stretch
  const int per = (mid + C - 1) / C, lo = min(rank * per, mid), size = min(per, mid - lo);
  w += first + lo;
  auto at = [&](int i) { return key_of(STAGED ? staged[i] : w[i]); };
  auto together = [&]() {  // all blocks of the cluster, or this one
    if (C > 1) tc::cluster_sync();
    else __syncthreads();
  };
  uint32_t prefix = 0;
  int left = mid;  // keys that begin with prefix
  int bits_left = 32;
  auto begins = [&](uint32_t k) { return bits_left == 32 || (k >> bits_left) == prefix; };
  // One digit more, of `bits` bits: c has this thread's four bins, from the top
  const int top = BINS - 4 - 4 * int(threadIdx.x);
  auto pick = [&](const int4 &c, int bits) {
    const int own = c.x + c.y + c.z + c.w;
    int total;
    const int upto = block_scan(own, sm.part, total);
    int above = upto - own;
    if (above < need && need <= upto) {  // one thread
      int d = top + 3, in = c.w;
      if (above + in < need) above += in, --d, in = c.z;
      if (above + in < need) above += in, --d, in = c.y;
      if (above + in < need) above += in, --d, in = c.x;
      sm.digit = d;
      sm.need = need - above;
      sm.left = in;
    }
    __syncthreads();
    prefix = (prefix << bits) | uint32_t(sm.digit);
    need = sm.need;  // of the keys that begin with prefix
    left = sm.left;
    bits_left -= bits;
    __syncthreads();
  };
  const int few = C > 1 ? FEW : FEW / 4;  // a digit costs a block alone no more than gathering does
  const bool digits = left > few;
  {
    constexpr int U = 8;
    float f[U];
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * NT < size) f[u] = w[i0 + u * NT];
    };
    if (STAGED || digits) load(threadIdx.x);
    for (int i = threadIdx.x; i < 2 * BINS; i += NT) sm.hist[0][i] = 0;
    if (threadIdx.x == 0) sm.taken = sm.last = 0;
    __syncthreads();
    if (STAGED || digits) {
      for (int i0 = threadIdx.x; i0 < size; i0 += U * NT) {
        if (i0 != int(threadIdx.x)) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (i0 + u * NT >= size) break;
          if (STAGED) staged[i0 + u * NT] = f[u];
          if (digits) atomicAdd(&sm.hist[0][key_of(f[u]) >> 21], 1);
        }
      }
    }
  }
#pragma unroll 1
  for (int digit = 0; digit < 3 && left > few; ++digit) {
    const int bits = digit == 2 ? 10 : 11, shift = bits_left - bits;
    int *hist = sm.hist[digit & 1];
    if (digit == 2) {  // the first digit's bins: all have read them before the second's were together
      for (int i = threadIdx.x; i < BINS; i += NT) hist[i] = 0;
      __syncthreads();
    }
    if (digit > 0) {
#pragma unroll 4
      for (int i = threadIdx.x; i < size; i += NT) {
        const uint32_t k = at(i);
        if (begins(k)) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
    }
    together();
    int4 c = *reinterpret_cast<const int4 *>(&hist[top]);
    if (C > 1) {
      int4 v[MOST_BLOCKS];
#pragma unroll
      for (int r = 1; r < MOST_BLOCKS; ++r)
        if (r < C) v[r] = *reinterpret_cast<const int4 *>(of_block(&hist[top], (rank + r) & (C - 1)));
#pragma unroll
      for (int r = 1; r < MOST_BLOCKS; ++r) {
        if (r >= C) break;
        c.x += v[r].x;
        c.y += v[r].y;
        c.z += v[r].z;
        c.w += v[r].w;
      }
    }
    pick(c, bits);
  }
  if (bits_left > 0) {
    // few are left: every block takes them all (a thread's own keys are staged by itself)
    for (int i0 = warp * 32; i0 < size; i0 += NT) {
      const int i = i0 + lane;
      const uint32_t k = i < size ? at(i) : 0u;
      const bool take = i < size && begins(k);
      const uint32_t m = __ballot_sync(0xffffffffu, take);
      int from = 0;
      if (lane == 0 && m) from = atomicAdd(&sm.taken, __popc(m));
      from = __shfl_sync(0xffffffffu, from, 0);
      if (take) sm.few[from + __popc(m & ((1u << lane) - 1u))] = k;
    }
    together();
    if (left > LAST) {  // none reads another block's bins any more
      for (int i = threadIdx.x; i < BINS; i += NT) sm.hist[0][i] = 0;
    }
    const uint32_t *keys = C > 1 ? sm.all : sm.few;
    const int all_left = left;
    if (C > 1) {
      int c[MOST_BLOCKS];
#pragma unroll
      for (int r = 0; r < MOST_BLOCKS; ++r) c[r] = r < C ? *of_block(&sm.taken, r) : 0;
      for (int i = threadIdx.x; i < left; i += NT) {
        int r = 0, j = i;
#pragma unroll
        for (int q = 0; q < MOST_BLOCKS - 1; ++q)
          if (r == q && j >= c[q]) j -= c[q], ++r;
        sm.all[i] = *of_block(&sm.few[j], r);
      }
    }
    if (C > 1 || left > LAST) __syncthreads();
#pragma unroll 1
    while (left > LAST && bits_left > 0) {
      const int bits = min(bits_left, 11), shift = bits_left - bits;
      for (int i = threadIdx.x; i < all_left; i += NT) {
        const uint32_t k = keys[i];
        if (begins(k)) atomicAdd(&sm.hist[0][(k >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      int4 *own = reinterpret_cast<int4 *>(&sm.hist[0][top]);
      const int4 c = *own;
      *own = make_int4(0, 0, 0, 0);
      pick(c, bits);
    }
    if (bits_left > 0) {
      if (left < all_left) {
        uint32_t *last = reinterpret_cast<uint32_t *>(sm.hist[1]);
        for (int i = threadIdx.x; i < all_left; i += NT) {
          const uint32_t k = keys[i];
          if (begins(k)) last[atomicAdd(&sm.last, 1)] = k;
        }
        keys = last;
        __syncthreads();
      }
      // the key that is the need-th from the top
      if (int(threadIdx.x) < left) {
        const uint32_t x = keys[threadIdx.x];
        int larger = 0, same = 0;
        for (int j = 0; j < left; ++j) {
          const uint32_t y = keys[j];
          larger += y > x;
          same += y == x;
        }
        if (larger < need && need <= larger + same) {  // equal ones write the same
          sm.digit = int(x);
          sm.need = need - larger;
        }
      }
      __syncthreads();
      prefix = uint32_t(sm.digit);
      need = sm.need;  // of the keys equal to prefix
    }
  }
  // The moving kernel's blocks come in from here on.  Earlier, they take the
  // place of blocks with work still to do (64 sequences 26.0 us, so 24.5).
  start_next_kernel();
  // keys above `prefix` stay, and the first `need` of those equal to it
  const int stretch = ((size + NW - 1) / NW + 31) / 32 * 32;
  const int s0 = min(warp * stretch, size), s1 = min(s0 + stretch, size);
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
  if (lane == 0) sm.part[warp] = more, sm.part2[warp] = same;
  __syncthreads();
  if (warp == 0) {
    int m = lane < NW ? sm.part[lane] : 0, e = lane < NW ? sm.part2[lane] : 0;
    for (int o = 16; o > 0; o >>= 1) {
      m += __shfl_xor_sync(0xffffffffu, m, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    if (lane == 0) sm.counts = make_int2(m, e);
  }
  together();
  int j = first, equal = 0;
  if (rank > 0) {
    int2 c[MOST_BLOCKS];
#pragma unroll
    for (int r = 0; r < MOST_BLOCKS; ++r) c[r] = r < rank ? *of_block(&sm.counts, r) : make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < MOST_BLOCKS; ++r) j += c[r].x, equal += c[r].y;
  }
  for (int v = 0; v < warp; ++v) j += sm.part[v], equal += sm.part2[v];
  j += min(equal, need);
  for (int i0 = s0; i0 < s1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < s1 ? at(i) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, i < s1 && k == prefix), below = (1u << lane) - 1u;
    const bool stays = i < s1 && (k > prefix || (k == prefix && equal + __popc(eq & below) < need));
    const uint32_t st = __ballot_sync(0xffffffffu, stays);
    if (stays) {
      const int to = j + __popc(st & below);
      kept[to] = first + lo + i;
      if (w_out) w_out[to] = STAGED ? staged[i] : w[i];
    }
    j += __popc(st);
    equal += __popc(eq);
  }
  together();  // none looks at another block any more, and all have written their places
#pragma unroll 4
  for (int q = first + all0; q < a.budget - a.recent; q += all) find_way(q, __ldcg(kept + q));
}

constexpr int MT = 256, MU = 8;  // threads of a moving block, rows of a thread a stretch

// Columns c0 .. c0 + cols of one tensor's rows of a (sequence, head)
template <class V>
__device__ __forceinline__ void move_rows(const EvictArgs &a, V *cache, int64_t pitch_page, int64_t pitch_row, int c0,
                                          int cols, int b, int h, int rows, int rb) {
  const int side = MT / cols, row = int(threadIdx.x) / cols;
  const bool live = row < side;
  const int4 *ways = a.ways + (int64_t(b) * a.heads + h) * a.budget;
  const int R = side * MU;
  cache += c0 + int(threadIdx.x) - row * cols;
  for (int j0 = rb * R; j0 < rows; j0 += R * a.row_blocks) {
    int4 way[MU];
    V v[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      const int j = j0 + u * side + row;
      way[u].x = -1;
      if (live && j < rows) way[u] = ways[j];
    }
#pragma unroll
    for (int u = 0; u < MU; ++u)
      if (way[u].x >= 0) v[u] = cache[way[u].x * pitch_page + way[u].y * pitch_row];
    if (a.in_place) __syncthreads();
#pragma unroll
    for (int u = 0; u < MU; ++u)
      if (way[u].x >= 0) cache[way[u].z * pitch_page + way[u].w * pitch_row] = v[u];
  }
}

// Weights in place, in one walk
__device__ __forceinline__ void move_weights(const EvictArgs &a, int b, int h, int rows) {
  float *w = a.w_out + b * a.w_seq + h * a.w_head;
  const int32_t *kept = a.kept + (int64_t(b) * a.heads + h) * a.budget;
  for (int j0 = 0; j0 < rows; j0 += MT * MU) {
    float v[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      const int j = j0 + u * MT + int(threadIdx.x);
      if (j < rows) v[u] = w[kept[j]];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      const int j = j0 + u * MT + int(threadIdx.x);
      if (j < rows) w[j] = v[u];
    }
  }
}

// Blocks that walk over the items of the sequences with rows to move
template <class V>
__global__ void __launch_bounds__(MT, 3) evict_move_kernel(const EvictArgs a) {
  constexpr int E = sizeof(V) / 2;  // elements of a vector
  wait_last_kernel();  // in every block: what follows may rely on the selection too
  const int per_head = (a.k_parts + a.v_parts) * a.row_blocks + int(a.w_out == a.w);
  const int64_t items = int64_t(a.moving[0]) * a.heads * per_head;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t bh = it / per_head;
    int part = int(it - bh * per_head);
    const int b = a.moving[1 + bh / a.heads], h = int(bh % a.heads), rows = min(length_of(a, b), a.budget);
    if (part == (a.k_parts + a.v_parts) * a.row_blocks) {
      move_weights(a, b, h, rows);
      continue;
    }
    const int rb = part % a.row_blocks;
    part /= a.row_blocks;
    const bool keys = part < a.k_parts;
    if (!keys) part -= a.k_parts;
    const int all = (keys ? a.dk : a.dv) / E, parts = keys ? a.k_parts : a.v_parts;
    const int per = (all + parts - 1) / parts, c0 = part * per, cols = min(per, all - c0);
    if (cols <= 0) continue;
    uint16_t *cache = keys ? a.k + h * a.k_head : a.v + h * a.v_head;
    move_rows<V>(a, reinterpret_cast<V *>(cache), (keys ? a.k_page : a.v_page) / E, (keys ? a.k_token : a.v_token) / E,
                 c0, cols, b, h, rows, rb);
  }
}

template <class V>
int launch_move(EvictArgs a, cudaStream_t st) {
  constexpr int E = sizeof(V) / 2;
  const int64_t bh = int64_t(a.B) * a.heads;
  // In place: columns of 32 bytes a block.  Into other pages: whole rows, those
  // of a (sequence, head) over several blocks.
  auto parts = [&](int cols) {
    const int least = (cols + MT - 1) / MT;
    return a.in_place ? std::max(least, cols * int(sizeof(V)) / 32) : least;
  };
  a.k_parts = parts(a.dk / E);
  a.v_parts = parts(a.dv / E);
  const int R = std::max(1, MT / std::max((a.dv ? std::min(a.dk, a.dv) : a.dk) / E, 1)) * MU;
  a.row_blocks = a.in_place ? 1 : (a.budget + R - 1) / R;
  if (int64_t(a.k_parts + a.v_parts) * a.row_blocks >= (int64_t(1) << 30)) return WQ_ERR_UNSUPPORTED;
  const int64_t items = bh * (int64_t(a.k_parts + a.v_parts) * a.row_blocks + 1);
  return launch_chained(evict_move_kernel<V>, unsigned(std::min<int64_t>(items, 3 * 152)), MT, 0, true, st, a);
}

template <bool STAGED>
int launch_select(const EvictArgs &a, int C, int smem, cudaStream_t st) {
  auto *k = evict_select_kernel<STAGED>;
  static OncePerDevice sized;
  if (!allow_smem(sized, k, STAGED ? STAGE_BYTES : 1024)) return WQ_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned((int64_t(a.B) * a.heads + 1) * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = unsigned(C);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, k, a, C) != cudaSuccess) return WQ_ERR_LAUNCH;
  return launched(1);
}

}  // namespace

int launch_evict(const EvictArgs &a, bool vec, cudaStream_t st) {
  // Blocks of a (sequence, head): enough for about 4096 keys each, while there
  // are SMs for them
  const int64_t bh = int64_t(a.B) * a.heads;
  int C = 1;
  while (C < MOST_BLOCKS && a.max_len > 4096 * C && 2 * C * bh <= 152) C *= 2;
  if ((bh + 1) * C >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  const int64_t stretch = (int64_t(a.max_len) + C - 1) / C * 4;
  const int rc = stretch <= STAGE_BYTES ? launch_select<true>(a, C, int(stretch), st) : launch_select<false>(a, C, 0, st);
  if (rc != WQ_OK) return rc;
  return vec ? launch_move<uint4>(a, st) : launch_move<uint16_t>(a, st);
}

}  // namespace wq
