// C ABI of the serving operators around the MoE layer: host-side argument
// checks.  Contracts are in include/wq.h.
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

}  // extern "C"
