// C ABI of the paged-attention operators: argument checks, workspace layout
// and launches.  Every kernel goes to the caller's stream.
#include "attn.h"

#include <cmath>

using namespace moe;

namespace {

constexpr int kMaxPlanRequests = 16384;
constexpr int kMaxRequests = 4096;
constexpr int kMaxForks = 4096;
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

// rows of a cache: 16-byte pieces
inline bool bad_caches(const void* k, const void* v) {
  return !k || !v || !aligned(k, 16) || !aligned(v, 16) || k == v;
}

// whether two arrays have memory in common
inline bool meet(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  return a && b && (uintptr_t)a < (uintptr_t)b + 4 * m && (uintptr_t)b < (uintptr_t)a + 4 * n;
}

// Behind attention's partials (kPartsEnd) moe_paged_release has a word a block and, where pages are shared, a word a
// page, so that it may run beside attention: kReleasePages of them in the workspace that every call asks for, more
// where a configuration has more pages.
constexpr size_t kPartsEnd = MOE_ATTN_HEADER_BYTES + kAttnPartBytes + kAttnJoinBytes;
constexpr size_t kReleasePages = 1 << 18;
constexpr size_t release_end(size_t pages) { return (kPartsEnd + (kAttnMaxCtas + pages) * 4 + 15) / 16 * 16; }
constexpr size_t kWorkspaceBytes = release_end(kReleasePages);
static_assert(kPartsEnd % 16 == 0, "16-byte pieces");

// of a configuration
size_t workspace_bytes(const moe_attn_config_t* c) {
  return (size_t)c->n_pages > kReleasePages ? release_end(c->n_pages) : kWorkspaceBytes;
}

moe_status_t check_ws(const void* ws, size_t ws_bytes) {
  if (!ws || !aligned(ws, 16)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < kWorkspaceBytes ? MOE_ERR_WORKSPACE : MOE_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// the partials of a call with shared prefixes, behind the workspace of the other calls (bytes)
struct PrefixLayout {
  size_t part, ml, parts_of, few_part, few_ml, pair_part, pair_ml, end;
};
PrefixLayout prefix_layout(const moe_attn_config_t* c, int64_t T) {
  const size_t rows = (size_t)T * c->n_heads, dp = c->head_dim <= 64 ? 64 : 128;
  PrefixLayout l;
  l.part = (workspace_bytes(c) + 255) / 256 * 256;
  l.ml = l.part + 2 * rows * dp * 4;
  l.parts_of = l.ml + 2 * rows * 8;
  l.few_part = l.parts_of + 2 * (size_t)T * c->n_kv_heads * 16;
  l.few_ml = l.few_part + 2 * (size_t)kFewRuns * kFewRows * dp * 4;
  l.pair_part = l.few_ml + 2 * (size_t)kFewRuns * kFewRows * 8;
  l.pair_ml = l.pair_part + kAttnPartSlots * 2 * kAttnRows * dp * 4;
  l.end = l.pair_ml + kAttnPartSlots * 2 * kAttnRows * 8;
  return l;
}

moe_status_t launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

#define CHECK(x) do { const moe_status_t st_ = (x); if (st_ != MOE_OK) return st_; } while (0)

}  // namespace

extern "C" {

moe_status_t moe_check_attn_config(const moe_attn_config_t* cfg) { return check_config(cfg); }

size_t moe_attn_workspace_bytes(const moe_attn_config_t* cfg) {
  return check_config(cfg) == MOE_OK ? workspace_bytes(cfg) : 0;
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

}  // extern "C"

namespace {

// positions [n_axes][T] and the pairs' axes (axis NULL: one axis)
moe_status_t rope_rows(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                       const int32_t* positions, int32_t n_axes, const uint8_t* axis, const uint64_t* table,
                       float rot_scale, int32_t inverse, void* out, int64_t out_ld, void* stream) {
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
  a.n_axes = n_axes;
  a.axis = axis;
  a.table = table;
  a.scale = rot_scale;
  a.T = T;
  a.D = cfg->head_dim;
  a.rot = cfg->rot_dim;
  a.inverse = inverse;
  return launched(launch_rope(a, cfg->dtype, cfg->rope_interleaved, (cudaStream_t)stream));
}

moe_status_t rope_append(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld, const void* k,
                         int64_t k_ld, const void* v, int64_t v_ld, const int32_t* positions, int32_t n_axes,
                         const uint8_t* axis, const uint64_t* table, float rot_scale, const int64_t* slot_map,
                         void* q_out, int64_t q_out_ld, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
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
  if (bad_caches(k_cache, v_cache)) return MOE_ERR_INVALID_ARG;
  if (bad_array(slot_map)) return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim > 0 && (bad_array(positions) || bad_array(table))) return MOE_ERR_INVALID_ARG;
  RopeArgs a{};
  a.part[0] = RopeRows{q, q_out, q_ld, q_out_ld, H, 1, 0};
  a.part[1] = RopeRows{k, k_cache, k_ld, 0, Hkv, 1, 1};
  a.part[2] = RopeRows{v, v_cache, v_ld, 0, Hkv, 0, 1};
  a.n_parts = 3;
  a.positions = positions;
  a.n_axes = n_axes;
  a.axis = axis;
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

moe_status_t check_axes(const moe_attn_config_t* cfg, int32_t n_axes, const uint8_t* axis) {
  CHECK(check_config(cfg));
  return n_axes < 1 || n_axes > MOE_ROPE_MAX_AXES || (cfg->rot_dim > 0 && !axis) ? MOE_ERR_INVALID_ARG : MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_rope(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                      const int32_t* positions, const uint64_t* table, float rot_scale, int32_t inverse, void* out,
                      int64_t out_ld, void* stream) {
  return rope_rows(cfg, T, heads, x, x_ld, positions, 1, nullptr, table, rot_scale, inverse, out, out_ld, stream);
}

moe_status_t moe_rope_append(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld, const void* k,
                             int64_t k_ld, const void* v, int64_t v_ld, const int32_t* positions,
                             const uint64_t* table, float rot_scale, const int64_t* slot_map, void* q_out,
                             int64_t q_out_ld, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                             void* stream) {
  return rope_append(cfg, T, q, q_ld, k, k_ld, v, v_ld, positions, 1, nullptr, table, rot_scale, slot_map, q_out,
                     q_out_ld, k_cache, v_cache, ws, ws_bytes, stream);
}

moe_status_t moe_rope_axes_table(int32_t n_axes, const int32_t* sections, int32_t interleaved, int32_t own_ladders,
                                 double theta, int32_t scaling, double factor, int64_t original_context,
                                 uint64_t* table_host, uint8_t* axis_host, float* rot_scale) {
  if (n_axes < 1 || n_axes > MOE_ROPE_MAX_AXES || !sections || (interleaved != 0 && interleaved != 1) ||
      (own_ladders != 0 && own_ladders != 1) || !rot_scale)
    return MOE_ERR_INVALID_ARG;
  int half = 0, most = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0 || sections[a] > 64) return MOE_ERR_INVALID_ARG;
    half += sections[a];
    most = sections[a] > most ? sections[a] : most;
  }
  if (half > 64 || (half > 0 && (bad_array(table_host) || !axis_host))) return MOE_ERR_INVALID_ARG;
  // one ladder of frequencies over all pairs, or one over each axis's pairs
  uint64_t ladder[MOE_ROPE_MAX_AXES][64];
  for (int a = 0; a < (own_ladders ? n_axes : 1); ++a)
    CHECK(moe_rope_table(2 * (own_ladders ? sections[a] : half), theta, scaling, factor, original_context, ladder[a],
                         rot_scale));
  int i = 0;
  auto deal = [&](int a, int j) {
    axis_host[i] = (uint8_t)a;
    table_host[i] = own_ladders ? ladder[a][j] : ladder[0][i];
    ++i;
  };
  if (interleaved) {
    for (int j = 0; j < most; ++j)
      for (int a = 0; a < n_axes; ++a)
        if (j < sections[a]) deal(a, j);
  } else {
    for (int a = 0; a < n_axes; ++a)
      for (int j = 0; j < sections[a]; ++j) deal(a, j);
  }
  return MOE_OK;
}

moe_status_t moe_rope_axes(const moe_attn_config_t* cfg, int32_t T, int32_t heads, const void* x, int64_t x_ld,
                           int32_t n_axes, const int32_t* positions, const uint8_t* axis, const uint64_t* table,
                           float rot_scale, int32_t inverse, void* out, int64_t out_ld, void* stream) {
  CHECK(check_axes(cfg, n_axes, axis));
  return rope_rows(cfg, T, heads, x, x_ld, positions, n_axes, axis, table, rot_scale, inverse, out, out_ld, stream);
}

moe_status_t moe_rope_append_axes(const moe_attn_config_t* cfg, int32_t T, const void* q, int64_t q_ld,
                                  const void* k, int64_t k_ld, const void* v, int64_t v_ld, int32_t n_axes,
                                  const int32_t* positions, const uint8_t* axis, const uint64_t* table,
                                  float rot_scale, const int64_t* slot_map, void* q_out, int64_t q_out_ld,
                                  void* k_cache, void* v_cache, void* ws, size_t ws_bytes, void* stream) {
  CHECK(check_axes(cfg, n_axes, axis));
  return rope_append(cfg, T, q, q_ld, k, k_ld, v, v_ld, positions, n_axes, axis, table, rot_scale, slot_map, q_out,
                     q_out_ld, k_cache, v_cache, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// checks and arguments that both attention entry points share; T > 0 after it where it returns MOE_OK and *a is filled
moe_status_t attention_args(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                            const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                            const void* k_cache, const void* v_cache, const int32_t* tree_mask, int32_t mask_words,
                            void* out, int64_t out_ld, float* lse, void* ws, AttnArgs* to) {
  if (bad_rows(cfg, q, q_ld, cfg->n_heads, T) || bad_rows(cfg, out, out_ld, cfg->n_heads, T) || q == out)
    return MOE_ERR_INVALID_ARG;
  if (R > 0 && (bad_array(q_start) || bad_array(kv_len) || (cfg->max_pages > 0 && bad_array(block_table))))
    return MOE_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return MOE_ERR_INVALID_ARG;
  if ((tree_mask && !aligned(tree_mask, 4)) || (lse && !aligned(lse, 4))) return MOE_ERR_INVALID_ARG;
  AttnArgs& a = *to;
  a = AttnArgs{};
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
  return MOE_OK;
}

// units that a walk over the requests (or groups) can have, in tiles and fixed costs, stay in 31 bits
bool too_much_work(const moe_attn_config_t* cfg, int64_t blocks, int64_t T) {
  const int64_t tiles = ((int64_t)cfg->max_pages * cfg->page_size + 127) / 128 + 1 + kAttnPieceCost;
  return T * cfg->n_heads * 32 >= ((int64_t)1 << 31) || blocks * cfg->n_kv_heads * tiles >= ((int64_t)1 << 31);
}

}  // namespace

extern "C" {

moe_status_t moe_tree_attention(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                const void* k_cache, const void* v_cache, const int32_t* tree_mask,
                                int32_t mask_words, void* out, int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (R < 0 || T < 0 || (tree_mask && mask_words < 1)) return MOE_ERR_INVALID_ARG;
  if (R > kMaxRequests || T > kMaxRows || too_much_work(cfg, (int64_t)T + R, T)) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (T == 0) return MOE_OK;
  AttnArgs a;
  CHECK(attention_args(cfg, R, T, q, q_ld, q_start, kv_len, block_table, k_cache, v_cache, tree_mask, mask_words, out,
                       out_ld, lse, ws, &a));
  return launched(cfg->dtype == MOE_DT_F32 ? launch_attention_f32(a, (cudaStream_t)stream)
                                           : launch_attention_bf16(a, (cudaStream_t)stream));
}

size_t moe_prefix_workspace_bytes(const moe_attn_config_t* cfg, int32_t T) {
  if (check_config(cfg) != MOE_OK || T < 0 || T > kMaxRows) return 0;
  return cfg->dtype == MOE_DT_F32 ? workspace_bytes(cfg) : prefix_layout(cfg, T).end;
}

moe_status_t moe_prefix_attention(const moe_attn_config_t* cfg, int32_t R, int32_t T, const void* q, int64_t q_ld,
                                  const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                  int32_t n_groups, const int32_t* group_start, const int32_t* prefix_row,
                                  const int32_t* prefix_len, const void* k_cache, const void* v_cache,
                                  const int32_t* tree_mask, int32_t mask_words, void* out, int64_t out_ld, float* lse,
                                  void* ws, size_t ws_bytes, void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (R < 0 || T < 0 || n_groups < 0 || n_groups > R || (tree_mask && mask_words < 1)) return MOE_ERR_INVALID_ARG;
  if (R > kPrefixMaxRequests || T > kMaxRows || too_much_work(cfg, 2 * (int64_t)T + R + n_groups, T))
    return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (ws_bytes < moe_prefix_workspace_bytes(cfg, T)) return MOE_ERR_WORKSPACE;
  if (T == 0) return MOE_OK;
  if (n_groups > 0 && (bad_array(group_start) || bad_array(prefix_row) || bad_array(prefix_len)))
    return MOE_ERR_INVALID_ARG;
  AttnArgs a;
  CHECK(attention_args(cfg, R, T, q, q_ld, q_start, kv_len, block_table, k_cache, v_cache, tree_mask, mask_words, out,
                       out_ld, lse, ws, &a));
  a.n_groups = n_groups;
  a.group_start = group_start;
  a.prefix_row = prefix_row;
  a.prefix_len = prefix_len;
  if (cfg->dtype == MOE_DT_F32) return launched(launch_prefix_attention_f32(a, (cudaStream_t)stream));
  const PrefixLayout l = prefix_layout(cfg, T);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  a.rows_part = reinterpret_cast<float*>(base + l.part);
  a.rows_ml = reinterpret_cast<float2*>(base + l.ml);
  a.parts_of = reinterpret_cast<int4*>(base + l.parts_of);
  a.few_part = reinterpret_cast<float*>(base + l.few_part);
  a.few_ml = reinterpret_cast<float2*>(base + l.few_ml);
  a.pair_part = reinterpret_cast<float*>(base + l.pair_part);
  a.pair_ml = reinterpret_cast<float2*>(base + l.pair_ml);
  return launched(launch_prefix_attention_bf16(a, (cudaStream_t)stream));
}

moe_status_t moe_paged_fork(const moe_attn_config_t* cfg, int32_t n, const int32_t* src_rows, const int32_t* dst_rows,
                            const int32_t* lengths, int32_t R, const int32_t* src_table, int32_t* dst_table,
                            int32_t* page_shares, const int32_t* free_pages, int32_t n_free, const int32_t* free_head,
                            int32_t* free_head_out, void* k_cache, void* v_cache, void* ws, size_t ws_bytes,
                            void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (n < 0 || R < 0 || n_free < 0) return MOE_ERR_INVALID_ARG;
  if (n > kMaxForks || R > kMaxPlanRequests) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (bad_array(free_head) || bad_array(free_head_out) || bad_array(page_shares)) return MOE_ERR_INVALID_ARG;
  if (n_free > 0 && bad_array(free_pages)) return MOE_ERR_INVALID_ARG;
  if (R > 0 && cfg->max_pages > 0 && (bad_array(src_table) || bad_array(dst_table))) return MOE_ERR_INVALID_ARG;
  if (bad_caches(k_cache, v_cache)) return MOE_ERR_INVALID_ARG;
  if (n > 0 && (bad_array(src_rows) || bad_array(dst_rows) || bad_array(lengths))) return MOE_ERR_INVALID_ARG;
  // one table, or two that do not meet
  const int64_t table_bytes = (int64_t)R * cfg->max_pages * 4, apart = (const char*)dst_table - (const char*)src_table;
  if (apart != 0 && apart < table_bytes && -apart < table_bytes) return MOE_ERR_INVALID_ARG;
  const int es = elem_bytes(cfg);
  if (2ll * cfg->n_kv_heads * (cfg->head_dim * es / 16) * cfg->page_size >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  ForkArgs a{};
  a.src = src_rows;
  a.dst = dst_rows;
  a.lengths = lengths;
  a.src_table = src_table;
  a.dst_table = dst_table;
  a.shares = page_shares;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.free_head_out = free_head_out;
  a.k = reinterpret_cast<uint8_t*>(k_cache);
  a.v = reinterpret_cast<uint8_t*>(v_cache);
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.page_stride = cfg->page_stride * es;
  a.token_stride = cfg->token_stride * es;
  a.head_stride = cfg->head_stride * es;
  a.n = n;
  a.R = R;
  a.n_free = n_free;
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  a.page_shift = log2_of(cfg->page_size);
  a.Hkv = cfg->n_kv_heads;
  a.row_bytes = cfg->head_dim * es;
  a.same = src_table == dst_table;
  return launched(launch_fork(a, (cudaStream_t)stream));
}

moe_status_t moe_paged_compact(const moe_attn_config_t* cfg, int32_t R, int32_t N, const int32_t* first,
                               const int32_t* keep_start, const int32_t* keep, const int32_t* block_table,
                               const int32_t* page_shares, int32_t* len_out, void* k_cache, void* v_cache, void* ws,
                               size_t ws_bytes, void* stream) {
  CHECK(check_config(cfg));
  CHECK(check_cache(cfg));
  if (R < 0 || N < 0) return MOE_ERR_INVALID_ARG;
  if (R > kMaxPlanRequests) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (R == 0) return MOE_OK;
  if (bad_array(first) || bad_array(keep_start) || (N > 0 && bad_array(keep)) ||
      (cfg->max_pages > 0 && bad_array(block_table)))
    return MOE_ERR_INVALID_ARG;
  if (bad_caches(k_cache, v_cache)) return MOE_ERR_INVALID_ARG;
  if ((page_shares && !aligned(page_shares, 4)) || (len_out && !aligned(len_out, 4))) return MOE_ERR_INVALID_ARG;
  // (other blocks read the lists while a length is written)
  if (meet(len_out, R, first, R) || meet(len_out, R, keep_start, (int64_t)R + 1) || meet(len_out, R, keep, N))
    return MOE_ERR_INVALID_ARG;
  const int es = elem_bytes(cfg);
  CompactArgs a{};
  a.scratch = reinterpret_cast<uint8_t*>(ws) + MOE_ATTN_HEADER_BYTES;
  a.scratch_bytes = kPartsEnd - MOE_ATTN_HEADER_BYTES;
  a.first = first;
  a.keep_start = keep_start;
  a.keep = keep;
  a.block_table = block_table;
  a.shares = page_shares;
  a.len_out = len_out;
  a.k = reinterpret_cast<uint8_t*>(k_cache);
  a.v = reinterpret_cast<uint8_t*>(v_cache);
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.page_stride = cfg->page_stride * es;
  a.token_stride = cfg->token_stride * es;
  a.head_stride = cfg->head_stride * es;
  a.R = R;
  a.N = N;
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  a.page_shift = log2_of(cfg->page_size);
  a.Hkv = cfg->n_kv_heads;
  a.row_bytes = cfg->head_dim * es;
  return launched(launch_compact(a, (cudaStream_t)stream));
}

moe_status_t moe_paged_release(const moe_attn_config_t* cfg, int32_t R, const int32_t* held_len,
                               const int32_t* keep_len, int32_t* block_table, int32_t* page_shares,
                               int32_t* free_pages, int32_t n_free, int32_t* free_head, void* ws, size_t ws_bytes,
                               void* stream) {
  CHECK(check_config(cfg));
  if (R < 0 || n_free < 0) return MOE_ERR_INVALID_ARG;
  if (R > kMaxPlanRequests || (int64_t)R * cfg->max_pages >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  CHECK(check_ws(ws, ws_bytes));
  if (page_shares && ws_bytes < workspace_bytes(cfg)) return MOE_ERR_WORKSPACE;
  if (bad_array(free_head) || (n_free > 0 && bad_array(free_pages))) return MOE_ERR_INVALID_ARG;
  if (R == 0) return MOE_OK;
  if (bad_array(held_len) || bad_array(keep_len) || (cfg->max_pages > 0 && bad_array(block_table)))
    return MOE_ERR_INVALID_ARG;
  if (page_shares && !aligned(page_shares, 4)) return MOE_ERR_INVALID_ARG;
  ReleaseArgs a{};
  a.held_len = held_len;
  a.keep_len = keep_len;
  a.block_table = block_table;
  a.shares = page_shares;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.hdr = reinterpret_cast<AttnHeader*>(ws);
  a.counts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(ws) + kPartsEnd);
  a.last = a.counts + kAttnMaxCtas;
  a.R = R;
  a.n_free = n_free;
  a.n_pages = cfg->n_pages;
  a.max_pages = cfg->max_pages;
  a.page_shift = log2_of(cfg->page_size);
  return launched(launch_release(a, (cudaStream_t)stream));
}

}  // extern "C"
