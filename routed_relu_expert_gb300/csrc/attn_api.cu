// C ABI of the paged-attention operators: argument checks, workspace layout
// and launches.  Every kernel goes to the caller's stream.
#include "attn.h"

#include <cmath>

using namespace moe;

namespace {

constexpr int kMaxPlanRequests = 16384;
constexpr int kMaxRequests = 4096;
constexpr int kMaxRows = 1 << 24;

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline int elem_bytes(const moe_attn_config_t* c) { return c->dtype == MOE_DT_F32 ? 4 : 2; }

moe_status_t check_config(const moe_attn_config_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DT_F32 && c->dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  if (c->n_heads < 1 || c->n_kv_heads < 1 || c->n_heads % c->n_kv_heads || c->n_heads > 65536)
    return MOE_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->page_size < 1 || c->n_pages < 0 || c->max_pages < 0) return MOE_ERR_INVALID_ARG;
  if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 2) return MOE_ERR_INVALID_ARG;
  if (c->rope_interleaved != 0 && c->rope_interleaved != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->softmax_scale) || c->softmax_scale <= 0.f) return MOE_ERR_INVALID_ARG;
  if (c->head_dim % 8 || c->head_dim > 128 || c->n_heads / c->n_kv_heads > kAttnRows) return MOE_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return MOE_ERR_UNSUPPORTED;
  // token numbers of a request and their rounding up to a tile stay in 31 bits
  if ((int64_t)c->max_pages * c->page_size > (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// the cache's strides: whole 16-byte pieces, tokens and heads apart
moe_status_t check_cache(const moe_attn_config_t* c) {
  const int64_t D = c->head_dim, q = 16 / elem_bytes(c);
  if (c->n_pages < 1) return MOE_ERR_INVALID_ARG;
  if (c->token_stride < D || c->page_stride < D || (c->n_kv_heads > 1 && c->head_stride < D))
    return MOE_ERR_INVALID_ARG;
  if (c->token_stride % q || c->page_stride % q || c->head_stride % q) return MOE_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 36;       // elements; a tensor map's strides end at 2^40 bytes
  if (c->token_stride >= most || c->page_stride >= most || c->head_stride >= most) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool bad_rows(const moe_attn_config_t* c, const void* p, int64_t ld, int heads, int T) {
  return !p || !aligned(p, 16) || ld % (16 / elem_bytes(c)) || (T > 1 && ld < (int64_t)heads * c->head_dim) ||
         ld >= ((int64_t)1 << 36);
}
template <typename T>
bool bad_array(const T* p) {
  return !p || !aligned(p, sizeof(T));
}

constexpr size_t kWorkspaceBytes = MOE_ATTN_HEADER_BYTES + kAttnPartBytes + kAttnJoinBytes;

moe_status_t check_ws(const void* ws, size_t ws_bytes) {
  if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < kWorkspaceBytes ? MOE_ERR_WORKSPACE : MOE_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

moe_status_t launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

#define CHECK(x) do { const moe_status_t st_ = (x); if (st_ != MOE_OK) return st_; } while (0)

}  // namespace

extern "C" {

moe_status_t moe_check_attn_config(const moe_attn_config_t* cfg) { return check_config(cfg); }

size_t moe_attn_workspace_bytes(const moe_attn_config_t* cfg) {
  return check_config(cfg) == MOE_OK ? kWorkspaceBytes : 0;
}

moe_status_t moe_paged_plan(const moe_attn_config_t* cfg, int32_t R, int32_t T, const int32_t* ctx_len,
                            const int32_t* new_len, const int32_t* parents, int32_t* block_table,
                            const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                            int32_t* free_head_out, int32_t* q_start, int32_t* kv_len, int32_t* positions,
                            int64_t* slot_map, int32_t* tree_mask, int32_t mask_words, void* ws, size_t ws_bytes,
                            void* stream) {
  CHECK(check_config(cfg));
  if (R < 0 || T < 0 || n_free < 0 || mask_words < 0) return MOE_ERR_INVALID_ARG;
  if (R > kMaxPlanRequests || T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (bad_array(q_start) || bad_array(free_head) || bad_array(free_head_out)) return MOE_ERR_INVALID_ARG;
  if (R > 0 && (bad_array(ctx_len) || bad_array(new_len) || bad_array(kv_len))) return MOE_ERR_INVALID_ARG;
  if (R > 0 && cfg->max_pages > 0 && bad_array(block_table)) return MOE_ERR_INVALID_ARG;
  if (n_free > 0 && bad_array(free_pages)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (bad_array(positions) || bad_array(slot_map))) return MOE_ERR_INVALID_ARG;
  if ((parents && !aligned(parents, 4)) || (tree_mask && !aligned(tree_mask, 4))) return MOE_ERR_INVALID_ARG;
  if (tree_mask && (!parents || mask_words < 1)) return MOE_ERR_INVALID_ARG;
  PlanArgs a{};
  a.ctx_len = ctx_len;
  a.new_len = new_len;
  a.parents = parents;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.free_head_out = free_head_out;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.positions = positions;
  a.slot_map = slot_map;
  a.tree_mask = tree_mask;
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.R = R;
  a.T = T;
  a.n_free = n_free;
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  a.page_shift = log2_of(cfg->page_size);
  a.mask_words = tree_mask ? mask_words : 0;
  return launched(launch_paged_plan(a, (cudaStream_t)stream));
}

moe_status_t moe_rope_table(int32_t rot_dim, double theta, int32_t scaling, double factor,
                            int64_t original_context, uint64_t* table_host, float* rot_scale) {
  if (rot_dim < 0 || rot_dim > 128 || rot_dim % 2 || !rot_scale || (rot_dim > 0 && bad_array(table_host)))
    return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROPE_PLAIN && scaling != MOE_ROPE_LINEAR && scaling != MOE_ROPE_YARN) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(theta) || theta <= 1.0) return MOE_ERR_INVALID_ARG;
  if (scaling != MOE_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return MOE_ERR_INVALID_ARG;
  if (scaling == MOE_ROPE_YARN && original_context < 1) return MOE_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  double low = 0.0, high = 0.0;
  if (scaling == MOE_ROPE_YARN) {
    // the pair index at which a pair turns `turns` times over original_context
    auto place = [&](double turns) {
      return rot_dim * std::log((double)original_context / (turns * two_pi)) / (2.0 * std::log(theta));
    };
    low = std::fmax(std::floor(place(32.0)), 0.0);
    high = std::fmin(std::ceil(place(1.0)), (double)rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot_dim);
    if (scaling == MOE_ROPE_LINEAR) f /= factor;
    if (scaling == MOE_ROPE_YARN) {
      const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    // f <= 1 radian: at most 0.16 turns, so the product stays below 2^62
    table_host[i] = (uint64_t)std::nearbyint(f / two_pi * 18446744073709551616.0);
  }
  *rot_scale = scaling == MOE_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return MOE_OK;
}

moe_status_t moe_rope(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                      const int32_t* positions, const uint64_t* table, float rot_scale, int32_t inverse, void* out,
                      int64_t out_ld, void* stream) {
  CHECK(check_config(cfg));
  if (T < 0 || heads < 1 || heads > 65536 || (inverse != 0 && inverse != 1) || !std::isfinite(rot_scale))
    return MOE_ERR_INVALID_ARG;
  if (T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (bad_rows(cfg, x, x_ld, heads, T) || bad_rows(cfg, out, out_ld, heads, T)) return MOE_ERR_INVALID_ARG;
  if (x == out && x_ld != out_ld) return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim > 0 && (bad_array(positions) || bad_array(table))) return MOE_ERR_INVALID_ARG;
  RopeArgs a{};
  a.part[0] = RopeRows{x, out, x_ld, out_ld, heads, 1, 0};
  a.n_parts = 1;
  a.positions = positions;
  a.table = table;
  a.scale = rot_scale;
  a.T = T;
  a.D = cfg->head_dim;
  a.rot = cfg->rot_dim;
  a.inverse = inverse;
  return launched(launch_rope(a, cfg->dtype, cfg->rope_interleaved, (cudaStream_t)stream));
}

moe_status_t moe_rope_append(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld, const void* k,
                             int64_t k_ld, const void* v, int64_t v_ld, const int32_t* positions,
                             const uint64_t* table, float rot_scale, const int64_t* slot_map, void* q_out,
                             int64_t q_out_ld, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                             void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (T < 0 || !std::isfinite(rot_scale)) return MOE_ERR_INVALID_ARG;
  if (T > kMaxRows) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (T == 0) return MOE_OK;
  const int H = cfg->n_heads, Hkv = cfg->n_kv_heads;
  if (bad_rows(cfg, q, q_ld, H, T) || bad_rows(cfg, k, k_ld, Hkv, T) || bad_rows(cfg, v, v_ld, Hkv, T) ||
      bad_rows(cfg, q_out, q_out_ld, H, T))
    return MOE_ERR_INVALID_ARG;
  if (q == q_out && q_ld != q_out_ld) return MOE_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16) || k_cache == v_cache)
    return MOE_ERR_INVALID_ARG;
  if (bad_array(slot_map)) return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim > 0 && (bad_array(positions) || bad_array(table))) return MOE_ERR_INVALID_ARG;
  RopeArgs a{};
  a.part[0] = RopeRows{q, q_out, q_ld, q_out_ld, H, 1, 0};
  a.part[1] = RopeRows{k, k_cache, k_ld, 0, Hkv, 1, 1};
  a.part[2] = RopeRows{v, v_cache, v_ld, 0, Hkv, 0, 1};
  a.n_parts = 3;
  a.positions = positions;
  a.table = table;
  a.slot_map = slot_map;
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.page_shift = log2_of(cfg->page_size);
  a.n_slots = (int64_t)cfg->n_pages << a.page_shift;
  a.page_stride = cfg->page_stride;
  a.token_stride = cfg->token_stride;
  a.head_stride = cfg->head_stride;
  a.scale = rot_scale;
  a.T = T;
  a.D = cfg->head_dim;
  a.rot = cfg->rot_dim;
  return launched(launch_rope(a, cfg->dtype, cfg->rope_interleaved, (cudaStream_t)stream));
}

moe_status_t moe_tree_attention(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                const void* k_cache, const void* v_cache, const int32_t* tree_mask,
                                int32_t mask_words, void* out, int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (R < 0 || T < 0 || (tree_mask && mask_words < 1)) return MOE_ERR_INVALID_ARG;
  const int64_t tiles = ((int64_t)cfg->max_pages * cfg->page_size + 127) / 128 + 1 + kAttnPieceCost;
  if (R > kMaxRequests || T > kMaxRows || (int64_t)T * cfg->n_heads * 32 >= ((int64_t)1 << 31) ||
      ((int64_t)T + R) * cfg->n_kv_heads * tiles >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (T == 0) return MOE_OK;
  if (bad_rows(cfg, q, q_ld, cfg->n_heads, T) || bad_rows(cfg, out, out_ld, cfg->n_heads, T) || q == out)
    return MOE_ERR_INVALID_ARG;
  if (R > 0 && (bad_array(q_start) || bad_array(kv_len) || (cfg->max_pages > 0 && bad_array(block_table))))
    return MOE_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return MOE_ERR_INVALID_ARG;
  if ((tree_mask && !aligned(tree_mask, 4)) || (lse && !aligned(lse, 4))) return MOE_ERR_INVALID_ARG;
  AttnArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.block_table = block_table;
  a.tree_mask = tree_mask;
  a.out = out;
  a.lse = lse;
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + MOE_ATTN_HEADER_BYTES);
  a.part_ml = reinterpret_cast<float2*>(a.part + kAttnPartSlots * kAttnRows * kAttnPartDim);
  a.joins = reinterpret_cast<int4*>(a.part_ml + kAttnPartSlots * kAttnRows);
  a.q_ld = q_ld;
  a.out_ld = out_ld;
  a.page_stride = cfg->page_stride;
  a.token_stride = cfg->token_stride;
  a.head_stride = cfg->head_stride;
  a.scale = cfg->softmax_scale;
  a.R = R;
  a.T = T;
  a.H = cfg->n_heads;
  a.Hkv = cfg->n_kv_heads;
  a.G = cfg->n_heads / cfg->n_kv_heads;
  a.D = cfg->head_dim;
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  a.page_shift = log2_of(cfg->page_size);
  a.mask_words = mask_words;
  return launched(cfg->dtype == MOE_DT_F32 ? launch_attention_f32(a, (cudaStream_t)stream)
                                           : launch_attention_bf16(a, (cudaStream_t)stream));
}

}  // extern "C"
