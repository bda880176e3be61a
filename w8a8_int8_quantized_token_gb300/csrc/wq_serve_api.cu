// C ABI of the serving operators around the MoE layer: host-side argument
// checks.  Contracts are in include/wq.h.
#include <algorithm>
#include <cmath>

#include "wq_serve.cuh"

using namespace wq;

namespace {

inline bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

bool cache_ok(const wq_paged_cache *c) {
  return c && c->heads >= 1 && c->page_size >= 1 && c->num_pages >= 0 && c->dk >= 1 && c->dv >= 1 &&
         (c->dtype == WQ_DT_BF16 || c->dtype == WQ_DT_F16) && c->k_page >= 0 && c->k_head >= 0 &&
         c->k_token >= 0 && c->v_page >= 0 && c->v_head >= 0 && c->v_token >= 0 &&
         c->num_pages < (int64_t(1) << 31);
}

// Rotary segments that the vector kernel may take
bool rope_vec_ok(const RopeArgs &a, int dtype) {
  if (dtype == WQ_DT_F32) return false;
  if (a.rot % (a.layout == WQ_ROPE_HALF ? 16 : 8) || !al(a.table, 16)) return false;
  for (int i = 0; i < a.nseg; ++i) {
    const RopeSeg &s = a.seg[i];
    if (s.D % 8 || s.s_token % 8 || s.s_head % 8 || s.d_token % 8 || s.d_head % 8 || s.d_page % 8 ||
        !al(s.src, 16) || !al(s.dst, 16))
      return false;
  }
  return true;
}

// Head norms that the vector kernel may take: float tensors too, and weights
// that start on 16 bytes
bool head_norm_vec_ok(const HeadNormArgs &h, int dtype) {
  const RopeArgs &a = h.r;
  const int n = dtype == WQ_DT_F32 ? 4 : 8;
  if (a.rot % (a.layout == WQ_ROPE_HALF ? 2 * n : n) || !al(a.table, 16)) return false;
  for (int i = 0; i < a.nseg; ++i) {
    const RopeSeg &s = a.seg[i];
    if (s.D % n || s.s_token % n || s.s_head % n || s.d_token % n || s.d_head % n || s.d_page % n ||
        !al(s.src, 16) || !al(s.dst, 16) || !al(h.weight[i], 16))
      return false;
  }
  return true;
}

int fill_attention(AttnArgs &a, int64_t T, int B, int max_q, int q_heads, const wq_paged_cache *c,
                   int64_t prefix_len, int64_t max_suffix) {
  if (T < 0 || B < 0 || max_q < 0 || q_heads < 1 || prefix_len < 0 || max_suffix < 0 || !cache_ok(c))
    return WQ_ERR_INVALID_ARG;
  if (q_heads % c->heads) return WQ_ERR_INVALID_ARG;
  if (T >= (1 << 24) || B >= (1 << 24) || prefix_len >= (int64_t(1) << 30) ||
      max_suffix >= (int64_t(1) << 30) || q_heads > (1 << 16) || q_heads / c->heads > 128)
    return WQ_ERR_UNSUPPORTED;
  if (c->dk % 8 || c->dv % 8 || c->dk > 128 || c->dv > 128) return WQ_ERR_UNSUPPORTED;
  if (c->k_page % 8 || c->k_head % 8 || c->k_token % 8 || c->v_page % 8 || c->v_head % 8 ||
      c->v_token % 8)
    return WQ_ERR_UNSUPPORTED;
  a = AttnArgs{};
  a.T = int(T);
  a.B = B;
  a.max_q = int(max_q < T ? max_q : T);
  a.Hq = q_heads;
  a.Hkv = c->heads;
  a.G = q_heads / c->heads;
  a.k = static_cast<const uint16_t *>(c->k);
  a.v = static_cast<const uint16_t *>(c->v);
  a.k_page = c->k_page;
  a.k_head = c->k_head;
  a.k_token = c->k_token;
  a.v_page = c->v_page;
  a.v_head = c->v_head;
  a.v_token = c->v_token;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.dk = c->dk;
  a.dv = c->dv;
  a.P = int(prefix_len);
  a.max_suffix = B > 0 ? int(max_suffix) : 0;
  plan_attention(a);
  return WQ_OK;
}

// Whether rows of n elements at b * seq + h * head, b < B and h < heads, share none
bool rows_apart(int64_t B, int64_t seq, int64_t heads, int64_t head, int64_t n) {
  if (heads == 1) return B == 1 || seq >= n;
  if (B == 1) return head >= n;
  return head <= seq ? head >= n && seq >= (heads - 1) * head + n : seq >= n && head >= (B - 1) * seq + n;
}

int fill_weights(WeightArgs &a, int64_t T, int B, int max_q, int q_heads, const wq_paged_cache *c,
                 int64_t max_len) {
  if (T < 0 || B < 0 || max_q < 0 || q_heads < 1 || max_len < 0 || !cache_ok(c) || q_heads % c->heads)
    return WQ_ERR_INVALID_ARG;
  if (T >= (1 << 24) || B >= (1 << 24) || max_len >= (int64_t(1) << 30) || q_heads > (1 << 16) ||
      q_heads / c->heads > 128 || c->dk % 8 || c->dk > 128 || c->k_page % 8 || c->k_head % 8 ||
      c->k_token % 8)
    return WQ_ERR_UNSUPPORTED;
  a = WeightArgs{};
  a.T = int(T);
  a.B = B;
  a.max_q = int(max_q < T ? max_q : T);
  a.Hq = q_heads;
  a.heads = c->heads;
  a.G = q_heads / c->heads;
  a.k = static_cast<const uint16_t *>(c->k);
  a.k_page = c->k_page;
  a.k_head = c->k_head;
  a.k_token = c->k_token;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.dk = c->dk;
  a.max_len = int(max_len);
  plan_weights(a);
  return WQ_OK;
}

}  // namespace

extern "C" {

int wq_block_norm(const void *block, int64_t ldb, const void *residual, int64_t ldr,
                  const void *gate, int64_t ldg, float scale, int post, const void *post_weight,
                  const void *post_bias, int pre, const void *pre_weight, const void *pre_bias,
                  float eps, int64_t T, int64_t H, int dtype, void *x_out, int64_t ldx, void *y,
                  int64_t ldy, wq_stream_t stream) {
  if (T < 0 || H < 0 || dtype < WQ_DT_BF16 || dtype > WQ_DT_F32 || post < WQ_NORM_NONE ||
      post > WQ_NORM_LAYER || pre < WQ_NORM_NONE || pre > WQ_NORM_LAYER || !(eps >= 0.0f))
    return WQ_ERR_INVALID_ARG;
  if (T == 0) return WQ_OK;
  if (!block || (!x_out && !y) || H < 1) return WQ_ERR_INVALID_ARG;
  if (ldb < H || (residual && ldr < H) || (gate && ldg != 0 && ldg < H) || (x_out && ldx < H) ||
      (y && ldy < H))
    return WQ_ERR_INVALID_ARG;
  if (H > 32768 || T >= (int64_t(1) << 31)) return WQ_ERR_UNSUPPORTED;
  const unsigned esz = dtype == WQ_DT_F32 ? 4 : 2, n = 16 / esz;
  const void *ptrs[] = {block, residual, gate, post_weight, post_bias, pre_weight, pre_bias, x_out, y};
  const int64_t pitch[] = {ldb, ldr, ldg, 0, 0, 0, 0, ldx, ldy};
  bool vec = H % n == 0, shift = true;
  for (int i = 0; i < 9; ++i) {
    if (!ptrs[i]) continue;
    if (!al(ptrs[i], esz)) return WQ_ERR_UNSUPPORTED;
    vec = vec && al(ptrs[i], 16) && pitch[i] % n == 0;
    // rows that start alike against 16-byte boundaries (one row for all, and
    // weights, are read element by element there)
    const bool rows = i < 3 ? !(i == 2 && ldg == 0) : i > 6;
    if (rows)
      shift = shift && reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == reinterpret_cast<uintptr_t>(block) % 16 &&
              pitch[i] % n == ldb % n;
  }
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  const BlockNormArgs a{block, residual, gate, post_weight, post_bias, pre_weight, pre_bias,
                        ldb,   ldr,      ldg,  ldx,         ldy,       scale,      eps,
                        post,  pre,      T,    int(H),      x_out,     y,          vec ? 0 : shift ? 1 : 2};
  return launch_block_norm(a, dtype, stream);
}

int wq_rope_table(float *table, int64_t max_pos, int rot, double base, int scaling, double factor,
                  double trained, double beta_fast, double beta_slow, double mscale,
                  wq_stream_t stream) {
  if (max_pos < 0 || rot < 2 || rot % 2 || scaling < WQ_ROPE_PLAIN || scaling > WQ_ROPE_YARN ||
      !(base > 1.0) || !(factor >= 1.0) || !(mscale >= 0.0) || !(base < 1e300) || !(factor < 1e300))
    return WQ_ERR_INVALID_ARG;
  if (scaling == WQ_ROPE_NTK && rot == 2) return WQ_ERR_INVALID_ARG;
  if (scaling == WQ_ROPE_YARN && (!(trained >= 1.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow)))
    return WQ_ERR_INVALID_ARG;
  if (max_pos == 0) return WQ_OK;
  if (!table) return WQ_ERR_INVALID_ARG;
  if (rot > 1024 || max_pos >= (int64_t(1) << 31) || !al(table, 8)) return WQ_ERR_UNSUPPORTED;
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  return launch_rope_table(table, max_pos, rot, base, scaling, factor, trained, beta_fast, beta_slow,
                           mscale, stream);
}

int wq_rope(const void *x, int64_t x_token, int64_t x_head, const int32_t *positions,
            const float *table, int64_t max_pos, int64_t T, int heads, int D, int rot, int layout,
            int inverse, int dtype, void *out, int64_t o_token, int64_t o_head, int32_t *status,
            wq_stream_t stream) {
  if (T < 0 || heads < 0 || D < 0 || max_pos < 0 || dtype < WQ_DT_BF16 || dtype > WQ_DT_F32 ||
      layout < WQ_ROPE_HALF || layout > WQ_ROPE_INTERLEAVED || x_token < 0 || x_head < 0 ||
      o_token < 0 || o_head < 0 || (inverse != 0 && inverse != 1))
    return WQ_ERR_INVALID_ARG;
  if (T == 0 || heads == 0) return WQ_OK;
  if (rot < 2 || rot % 2 || rot > D || !x || !out || !positions || !table) return WQ_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 31) || heads > (1 << 16) || D > (1 << 14) || !al(table, 8) ||
      !al(x, dtype == WQ_DT_F32 ? 4 : 2) || !al(out, dtype == WQ_DT_F32 ? 4 : 2))
    return WQ_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.seg[0] = {x, out, x_token, x_head, o_token, o_head, 0, heads, D, rot, false};
  a.nseg = 1;
  a.positions = positions;
  a.table = table;
  a.max_pos = max_pos;
  a.T = T;
  a.rot = rot;
  a.layout = layout;
  a.sign = inverse ? -1.0f : 1.0f;
  a.status = status;
  const bool vec = rope_vec_ok(a, dtype);
  if (!vec && rope_pair_threads(a) > kRopeMostThreads) return WQ_ERR_UNSUPPORTED;
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  return launch_rope(a, dtype, vec, stream);
}

int wq_rope_append_paged(const void *q, int64_t q_token, int64_t q_head, int q_heads,
                         const void *k_new, int64_t kn_token, int64_t kn_head, const void *v_new,
                         int64_t vn_token, int64_t vn_head, const int32_t *positions,
                         const int64_t *slots, const float *table, int64_t max_pos, int64_t T,
                         int rot, int layout, const wq_paged_cache *cache, void *q_out,
                         int64_t qo_token, int64_t qo_head, int32_t *status, wq_stream_t stream) {
  if (T < 0 || q_heads < 0 || rot < 0 || rot % 2 || max_pos < 0 || layout < WQ_ROPE_HALF ||
      layout > WQ_ROPE_INTERLEAVED || !cache_ok(cache) || q_token < 0 || q_head < 0 || kn_token < 0 ||
      kn_head < 0 || vn_token < 0 || vn_head < 0 || qo_token < 0 || qo_head < 0 || rot > cache->dk)
    return WQ_ERR_INVALID_ARG;
  if (T == 0) return WQ_OK;
  if (!k_new || !v_new || !slots || !cache->k || !cache->v || (rot && (!positions || !table)) ||
      (q && (!q_out || q_heads < 1)))
    return WQ_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 31) || cache->heads > (1 << 16) || q_heads > (1 << 16) ||
      cache->dk > (1 << 14) || cache->dv > (1 << 14) || !al(table, 8))
    return WQ_ERR_UNSUPPORTED;
  for (const void *p : {q, static_cast<const void *>(q_out), k_new, v_new,
                        static_cast<const void *>(cache->k), static_cast<const void *>(cache->v)})
    if (!al(p, 2)) return WQ_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.seg[0] = {k_new, cache->k, kn_token, kn_head, cache->k_token, cache->k_head, cache->k_page,
              cache->heads, cache->dk, rot, true};
  a.seg[1] = {v_new, cache->v, vn_token, vn_head, cache->v_token, cache->v_head, cache->v_page,
              cache->heads, cache->dv, 0, true};
  if (q) a.seg[2] = {q, q_out, q_token, q_head, qo_token, qo_head, 0, q_heads, cache->dk, rot, false};
  a.nseg = q ? 3 : 2;
  a.positions = positions;
  a.slots = slots;
  a.table = table;
  a.max_pos = max_pos;
  a.T = T;
  a.num_slots = cache->num_pages * cache->page_size;
  a.page_size = cache->page_size;
  a.rot = rot;
  a.layout = layout;
  a.sign = 1.0f;
  a.status = status;
  const bool vec = rope_vec_ok(a, cache->dtype);
  if (!vec && rope_pair_threads(a) > kRopeMostThreads) return WQ_ERR_UNSUPPORTED;
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  return launch_rope(a, cache->dtype, vec, stream);
}

int wq_head_norm_rope(const void *x, int64_t x_token, int64_t x_head, const void *weight, float eps,
                      const int32_t *positions, const float *table, int64_t max_pos, int64_t T,
                      int heads, int D, int rot, int layout, int dtype, void *out, int64_t o_token,
                      int64_t o_head, int32_t *status, wq_stream_t stream) {
  if (T < 0 || heads < 0 || D < 0 || max_pos < 0 || dtype < WQ_DT_BF16 || dtype > WQ_DT_F32 ||
      layout < WQ_ROPE_HALF || layout > WQ_ROPE_INTERLEAVED || x_token < 0 || x_head < 0 ||
      o_token < 0 || o_head < 0 || !(eps >= 0.0f))
    return WQ_ERR_INVALID_ARG;
  if (T == 0 || heads == 0) return WQ_OK;
  if (D < 1 || rot < 0 || rot % 2 || rot > D || !x || !out || (rot && (!positions || !table)))
    return WQ_ERR_INVALID_ARG;
  const unsigned esz = dtype == WQ_DT_F32 ? 4 : 2;
  if (T >= (int64_t(1) << 31) || heads > (1 << 16) || D > (1 << 14) || !al(table, 8) || !al(x, esz) ||
      !al(out, esz) || !al(weight, esz))
    return WQ_ERR_UNSUPPORTED;
  HeadNormArgs h{};
  RopeArgs &a = h.r;
  a.seg[0] = {x, out, x_token, x_head, o_token, o_head, 0, heads, D, rot, false};
  a.nseg = 1;
  a.positions = positions;
  a.table = table;
  a.max_pos = max_pos;
  a.T = T;
  a.rot = rot;
  a.layout = layout;
  a.status = status;
  h.weight[0] = weight;
  h.norm[0] = true;
  h.inv_d[0] = 1.0f / float(D);
  h.eps = eps;
  const bool vec = head_norm_vec_ok(h, dtype);
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  return launch_head_norm(h, dtype, vec, stream);
}

int wq_head_norm_rope_append_paged(const void *q, int64_t q_token, int64_t q_head, int q_heads,
                                   const void *q_weight, const void *k_new, int64_t kn_token,
                                   int64_t kn_head, const void *k_weight, const void *v_new,
                                   int64_t vn_token, int64_t vn_head, float eps,
                                   const int32_t *positions, const int64_t *slots,
                                   const float *table, int64_t max_pos, int64_t T, int rot,
                                   int layout, const wq_paged_cache *cache, void *q_out,
                                   int64_t qo_token, int64_t qo_head, int32_t *status,
                                   wq_stream_t stream) {
  if (T < 0 || q_heads < 0 || rot < 0 || rot % 2 || max_pos < 0 || layout < WQ_ROPE_HALF ||
      layout > WQ_ROPE_INTERLEAVED || !cache_ok(cache) || q_token < 0 || q_head < 0 || kn_token < 0 ||
      kn_head < 0 || vn_token < 0 || vn_head < 0 || qo_token < 0 || qo_head < 0 || rot > cache->dk ||
      !(eps >= 0.0f))
    return WQ_ERR_INVALID_ARG;
  if (T == 0) return WQ_OK;
  if (!k_new || !v_new || !slots || !cache->k || !cache->v || (rot && (!positions || !table)) ||
      (q && (!q_out || q_heads < 1)))
    return WQ_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 31) || cache->heads > (1 << 16) || q_heads > (1 << 16) ||
      cache->dk > (1 << 14) || cache->dv > (1 << 14) || !al(table, 8))
    return WQ_ERR_UNSUPPORTED;
  for (const void *p : {q, static_cast<const void *>(q_out), k_new, v_new, q_weight, k_weight,
                        static_cast<const void *>(cache->k), static_cast<const void *>(cache->v)})
    if (!al(p, 2)) return WQ_ERR_UNSUPPORTED;
  HeadNormArgs h{};
  RopeArgs &a = h.r;
  a.seg[0] = {k_new, cache->k, kn_token, kn_head, cache->k_token, cache->k_head, cache->k_page,
              cache->heads, cache->dk, rot, true};
  a.seg[1] = {v_new, cache->v, vn_token, vn_head, cache->v_token, cache->v_head, cache->v_page,
              cache->heads, cache->dv, 0, true};
  if (q) a.seg[2] = {q, q_out, q_token, q_head, qo_token, qo_head, 0, q_heads, cache->dk, rot, false};
  a.nseg = q ? 3 : 2;
  a.positions = positions;
  a.slots = slots;
  a.table = table;
  a.max_pos = max_pos;
  a.T = T;
  a.num_slots = cache->num_pages * cache->page_size;
  a.page_size = cache->page_size;
  a.rot = rot;
  a.layout = layout;
  a.status = status;
  h.weight[0] = k_weight;
  h.weight[2] = q ? q_weight : nullptr;
  h.norm[0] = h.norm[2] = true;
  h.inv_d[0] = h.inv_d[2] = 1.0f / float(cache->dk);
  h.eps = eps;
  const bool vec = head_norm_vec_ok(h, cache->dtype);
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  return launch_head_norm(h, cache->dtype, vec, stream);
}

size_t wq_attention_shared_prefix_workspace_size(int64_t T, int B, int max_q, int q_heads,
                                                 const wq_paged_cache *cache, int64_t prefix_len,
                                                 int64_t max_suffix) {
  AttnArgs a;
  if (T == 0 || fill_attention(a, T, B, max_q, q_heads, cache, prefix_len, max_suffix) != WQ_OK) return 0;
  return attention_ws_bytes(a);
}

int wq_attention_shared_prefix(const void *q, int64_t q_token, int64_t q_head, int64_t T, int B,
                               const int32_t *cu_q, int max_q, int q_heads,
                               const wq_paged_cache *cache, const int32_t *prefix_pages,
                               int64_t prefix_len, const int32_t *page_table, int64_t ld_table,
                               const int32_t *suffix_len, int64_t max_suffix, float scale,
                               void *out, int64_t o_token, int64_t o_head, float *lse, void *ws,
                               size_t ws_bytes, int32_t *status, wq_stream_t stream) {
  AttnArgs a;
  int rc = fill_attention(a, T, B, max_q, q_heads, cache, prefix_len, max_suffix);
  if (rc != WQ_OK) return rc;
  if (q_token < 0 || q_head < 0 || o_token < 0 || o_head < 0 || ld_table < 0 || !(scale > 0.0f) ||
      !(scale < INFINITY))
    return WQ_ERR_INVALID_ARG;
  if (T == 0) return WQ_OK;
  if (B < 1 || !q || !out || !cache->k || !cache->v || (prefix_len > 0 && !prefix_pages))
    return WQ_ERR_INVALID_ARG;
  if (max_suffix > 0 && (!page_table || !suffix_len || max_suffix > ld_table * cache->page_size))
    return WQ_ERR_INVALID_ARG;
  if (cu_q ? max_q < 1 : int64_t(max_q) * B != T) return WQ_ERR_INVALID_ARG;
  if ((T > 1 && (!q_token || !o_token)) || (q_heads > 1 && (!q_head || !o_head))) return WQ_ERR_UNSUPPORTED;
  if (q_token % 8 || q_head % 8 || o_token % 2 || o_head % 2 || !al(q, 16) || !al(cache->k, 16) ||
      !al(cache->v, 16) || !al(out, 4) || !al(lse, 4))
    return WQ_ERR_UNSUPPORTED;
  if (attention_ws_bytes(a) > 0 && (!ws || !al(ws, 16) || ws_bytes < attention_ws_bytes(a)))
    return WQ_ERR_WORKSPACE;
  rc = device_ok();
  if (rc != WQ_OK) return rc;
  a.q = static_cast<const uint16_t *>(q);
  a.q_token = q_token;
  a.q_head = q_head;
  a.cu_q = cu_q;
  a.prefix_pages = prefix_pages;
  a.page_table = page_table;
  a.ld_table = ld_table;
  a.suffix_len = suffix_len;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = static_cast<uint16_t *>(out);
  a.o_token = o_token;
  a.o_head = o_head;
  a.lse = lse;
  a.status = status;
  if (a.slots > 1) {
    const size_t rows = size_t(a.T) * a.Hq * a.slots;
    a.o_part = static_cast<float *>(ws);
    a.lse_part = reinterpret_cast<float *>(static_cast<char *>(ws) +
                                           ((rows * a.dv * 4 + 255) & ~size_t(255)));
  }
  return launch_attention(a, cache->dtype, stream);
}

size_t wq_attention_weights_paged_workspace_size(int64_t T, int B, int max_q, int q_heads,
                                                 const wq_paged_cache *cache, int64_t max_len) {
  WeightArgs a;
  if (fill_weights(a, T, B, max_q, q_heads, cache, max_len) != WQ_OK) return 0;
  return weights_ws_bytes(a);
}

int wq_attention_weights_paged(const void *q, int64_t q_token, int64_t q_head, int64_t T, int B,
                               const int32_t *cu_q, int max_q, int q_heads,
                               const wq_paged_cache *cache, const int32_t *page_table,
                               int64_t ld_table, const int32_t *key_len, int64_t max_len, float scale,
                               const float *lse, float decay, float *weights, int64_t w_seq,
                               int64_t w_head, void *ws, size_t ws_bytes, int32_t *status,
                               wq_stream_t stream) {
  WeightArgs a;
  int rc = fill_weights(a, T, B, max_q, q_heads, cache, max_len);
  if (rc != WQ_OK) return rc;
  if (q_token < 0 || q_head < 0 || ld_table < 0 || w_seq < 0 || w_head < 0 || !(scale > 0.0f) ||
      !(scale < INFINITY) || !(decay >= 0.0f) || !(decay < INFINITY))
    return WQ_ERR_INVALID_ARG;
  if (B == 0 || max_len == 0) return WQ_OK;
  if (!cache->k || !page_table || !key_len || !weights || max_len > ld_table * cache->page_size ||
      (T > 0 && (!q || !lse)))
    return WQ_ERR_INVALID_ARG;
  if (cu_q ? T > 0 && max_q < 1 : int64_t(max_q) * B != T) return WQ_ERR_INVALID_ARG;
  if (!rows_apart(B, w_seq, a.heads, w_head, max_len)) return WQ_ERR_INVALID_ARG;
  if ((T > 1 && !q_token) || (q_heads > 1 && !q_head)) return WQ_ERR_UNSUPPORTED;
  if (q_token % 8 || q_head % 8 || !al(q, 16) || !al(cache->k, 16) || !al(lse, 4) || !al(weights, 4))
    return WQ_ERR_UNSUPPORTED;
  if (weights_ws_bytes(a) > 0 && (!ws || !al(ws, 16) || ws_bytes < weights_ws_bytes(a)))
    return WQ_ERR_WORKSPACE;
  rc = device_ok();
  if (rc != WQ_OK) return rc;
  a.q = static_cast<const uint16_t *>(q);
  a.q_token = q_token;
  a.q_head = q_head;
  a.cu_q = cu_q;
  a.page_table = page_table;
  a.ld_table = ld_table;
  a.key_len = key_len;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.decay = decay;
  a.lse = lse;
  a.w = weights;
  a.w_seq = w_seq;
  a.w_head = w_head;
  a.status = status;
  a.part = a.split ? static_cast<float *>(ws) : nullptr;
  return launch_weights(a, cache->dtype, stream);
}

size_t wq_evict_paged_workspace_size(int B, int heads, int64_t budget) {
  if (B < 1 || heads < 1 || budget < 1) return 0;
  return size_t(B) * size_t(heads) * size_t(budget) * sizeof(int4) + (size_t(B) + 1) * sizeof(int32_t);
}

int wq_evict_paged(const float *weights, int64_t w_seq, int64_t w_head, const wq_paged_cache *cache,
                   int B, const int32_t *page_table, int64_t ld_table, const int32_t *key_len,
                   int64_t max_len, int64_t budget, int64_t recent, int64_t first,
                   const int32_t *out_table, int64_t ld_out, float *weights_out, int64_t o_seq,
                   int64_t o_head, int32_t *new_len, int32_t *kept, void *ws, size_t ws_bytes,
                   int32_t *status, wq_stream_t stream) {
  if (B < 0 || max_len < 0 || budget < 1 || recent < 0 || first < 0 || recent + first > budget || !cache_ok(cache) ||
      ld_table < 0 || ld_out < 0 || w_seq < 0 || w_head < 0 || o_seq < 0 || o_head < 0)
    return WQ_ERR_INVALID_ARG;
  if (B == 0) return WQ_OK;
  const int64_t rows = budget < max_len ? budget : max_len;  // that a sequence has at the end, at most
  if (!key_len || !new_len || !kept || (max_len > 0 && (!weights || !weights_out || !page_table || !cache->k || !cache->v)))
    return WQ_ERR_INVALID_ARG;
  if (max_len > ld_table * cache->page_size || (out_table && rows > ld_out * cache->page_size)) return WQ_ERR_INVALID_ARG;
  if (!rows_apart(B, w_seq, cache->heads, w_head, max_len) || !rows_apart(B, o_seq, cache->heads, o_head, rows))
    return WQ_ERR_INVALID_ARG;
  if (weights_out == weights && (w_seq != o_seq || w_head != o_head)) return WQ_ERR_INVALID_ARG;
  // the lengths are read while the new ones are written
  if (new_len < key_len + B && key_len < new_len + B) return WQ_ERR_INVALID_ARG;
  if (B >= (1 << 24) || max_len >= (int64_t(1) << 30) || budget >= (int64_t(1) << 30) || cache->heads > (1 << 16) ||
      cache->dk > (1 << 14) || cache->dv > (1 << 14) || !al(cache->k, 2) || !al(cache->v, 2) || !al(weights, 4) ||
      !al(weights_out, 4))
    return WQ_ERR_UNSUPPORTED;
  if (!ws || !al(ws, 16) || ws_bytes < wq_evict_paged_workspace_size(B, cache->heads, budget)) return WQ_ERR_WORKSPACE;
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  EvictArgs a{};
  a.w = weights;
  a.w_seq = w_seq;
  a.w_head = w_head;
  a.k = static_cast<uint16_t *>(cache->k);
  a.v = static_cast<uint16_t *>(cache->v);
  a.k_page = cache->k_page;
  a.k_head = cache->k_head;
  a.k_token = cache->k_token;
  a.v_page = cache->v_page;
  a.v_head = cache->v_head;
  a.v_token = cache->v_token;
  a.num_pages = cache->num_pages;
  a.page_size = cache->page_size;
  a.heads = cache->heads;
  a.dk = cache->dk;
  a.dv = cache->dv;
  auto alike = [](int64_t extent, int64_t k, int64_t v) { return extent <= 1 || k == v; };
  if (a.k && a.k < a.v + a.dv && a.v < a.k + a.dk && alike(a.num_pages, a.k_page, a.v_page) &&
      alike(a.heads, a.k_head, a.v_head) && alike(a.page_size, a.k_token, a.v_token)) {
    // elements that both have move once
    uint16_t *end = std::max(a.k + a.dk, a.v + a.dv);
    a.k = std::min(a.k, a.v);
    a.dk = int(end - a.k);
    a.dv = 0;
  }
  a.B = B;
  a.page_table = page_table;
  a.ld_table = ld_table;
  a.in_place = out_table == nullptr || out_table == page_table;
  a.out_table = a.in_place ? page_table : out_table;
  a.ld_out = a.in_place ? ld_table : ld_out;
  a.key_len = key_len;
  a.max_len = int(max_len);
  a.budget = int(budget);
  a.recent = int(recent);
  a.first = int(first);
  a.w_out = weights_out;
  a.o_seq = o_seq;
  a.o_head = o_head;
  a.new_len = new_len;
  a.kept = kept;
  a.status = status;
  a.ways = static_cast<int4 *>(ws);
  a.moving = reinterpret_cast<int32_t *>(a.ways + int64_t(B) * a.heads * a.budget);
  bool vec = al(cache->k, 16) && al(cache->v, 16) && cache->dk % 8 == 0 && cache->dv % 8 == 0;
  for (int64_t p : {a.k_page, a.k_head, a.k_token, a.v_page, a.v_head, a.v_token}) vec = vec && p % 8 == 0;
  return launch_evict(a, vec, stream);
}

size_t wq_lora_add_workspace_size(int64_t T, int n, int r) {
  return T < 1 || n < 1 || r < 1 || r > 128 || T >= (1 << 24) ? 0 : lora_ws_bytes(T, n, r);
}

int wq_lora_add(const void *x, int64_t ldx, int64_t T, int64_t H, const void *A, const void *B,
                const float *scales, int n, int r, const int32_t *adapters, int64_t N, int dtype,
                void *y, int64_t ldy, void *ws, size_t ws_bytes, int32_t *status,
                wq_stream_t stream) {
  if (T < 0 || H < 0 || N < 0 || n < 0 || r < 1 || (dtype != WQ_DT_BF16 && dtype != WQ_DT_F16))
    return WQ_ERR_INVALID_ARG;
  if (T == 0 || N == 0 || n == 0 || H == 0) return WQ_OK;
  if (!x || !A || !B || !adapters || !y || ldx < H || ldy < N) return WQ_ERR_INVALID_ARG;
  if (H % 8 || N % 8 || r % 8 || r > 128 || ldx % 8 || ldy % 8 || n > 8192 || T >= (1 << 24) ||
      H > (1 << 20) || N > (1 << 20) || !al(x, 16) || !al(A, 16) || !al(B, 16) || !al(y, 16) || !al(scales, 4))
    return WQ_ERR_UNSUPPORTED;
  const size_t need = lora_ws_bytes(T, n, r);
  if (need > 0 && (!ws || !al(ws, 16) || ws_bytes < need)) return WQ_ERR_WORKSPACE;
  const int rc = device_ok();
  if (rc != WQ_OK) return rc;
  LoraArgs a{};
  a.x = static_cast<const uint16_t *>(x);
  a.ldx = ldx;
  a.y = static_cast<uint16_t *>(y);
  a.ldy = ldy;
  a.A = static_cast<const uint16_t *>(A);
  a.B = static_cast<const uint16_t *>(B);
  a.scales = scales;
  a.ids = adapters;
  a.T = int(T);
  a.H = int(H);
  a.N = int(N);
  a.r = r;
  a.n = n;
  a.status = status;
  return launch_lora(a, dtype, ws, stream);
}

}  // extern "C"
