// C ABI of the paged cache's operators (include/cache.h): argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "api.h"
#include "cache.h"
#include "common.cuh"
#include "kernels.h"

using moe::aligned;
using moe::cuda_status;
using moe::device_sms;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 39;  // bf16 elements: 2^40 bytes

bool stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0 && s < kMaxStride; }

// Checks a rotation for heads of d elements and enters it in p. `placed`: tokens have
// positions of their own, so that NULL is one axis of those.
int enter_rope(moe::RopeParams& p, const moe_rope_t* rope, int tokens, bool placed) {
  if (!rope || rope->pairs == 0) return MOE_OK;
  const moe_rope_t& r = *rope;
  if (r.pairs < 0 || r.pairs > p.d / 2 || r.pairs % (r.adjacent ? 4 : 8) != 0) return MOE_ERR_SHAPE;
  if (r.n_axes < 1 || r.n_axes > MOE_ROPE_MAX_AXES) return MOE_ERR_SHAPE;
  int64_t sum = 0;
  for (int a = 0; a < r.n_axes; ++a) {
    if (r.sections[a] < 0 || r.sections[a] > r.pairs) return MOE_ERR_SHAPE;
    if (r.cyclic && a > 0 && r.sections[a] > 0 && r.n_axes * (r.sections[a] - 1) + a >= r.pairs) return MOE_ERR_SHAPE;
    sum += r.sections[a];
    p.sections[a] = r.sections[a];
  }
  if (sum != r.pairs) return MOE_ERR_SHAPE;
  if (!r.positions && placed && r.n_axes != 1) return MOE_ERR_SHAPE;
  if (r.positions && r.n_axes > 1 && r.ld_positions < 0) return MOE_ERR_SHAPE;
  if (tokens > 0) {
    if (!r.freqs || (!r.positions && !placed)) return MOE_ERR_NULL;
    if (!aligned(r.freqs, 4) || !aligned(r.positions, 4)) return MOE_ERR_ALIGN;
  }
  p.freqs = r.freqs;
  p.positions = r.positions;
  p.ld_positions = r.n_axes > 1 ? r.ld_positions : 0;
  p.pairs = r.pairs;
  p.n_axes = r.n_axes;
  p.cyclic = r.cyclic != 0;
  p.adjacent = r.adjacent != 0;
  return MOE_OK;
}

// The checks that a cache needs whoever uses it; copies it with the strides of axes of one
// entry set to such as a longer one could have.
int check_cache(const moe_paged_t* cache, moe_paged_t& c, int64_t max_positions) {
  if (!cache) return MOE_ERR_NULL;
  c = *cache;
  if (c.n_pages < 1 || c.page < 8 || c.page > 4096 || (c.page & (c.page - 1)) != 0 || c.width < 1 ||
      c.n_sequences < 1 || c.n_sequences > 65535 || c.n_kv_heads < 1 || c.n_kv_heads > 1024 || c.d < 8 || c.d % 8 != 0 ||
      c.d > 256 || (int64_t)c.width * c.page > max_positions)
    return MOE_ERR_SHAPE;
  if (c.n_kv_heads == 1) c.head_stride = c.d;
  if (c.n_pages == 1) c.page_stride = std::max(c.page * c.position_stride, c.n_kv_heads * c.head_stride);
  if (c.n_sequences == 1) c.ld_table = c.width;
  if (!stride_ok(c.page_stride, c.d) || !stride_ok(c.position_stride, c.d) || !stride_ok(c.head_stride, c.d) ||
      c.ld_table < c.width)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}
int check_cache_pointers(const moe_paged_t& c) {
  if (!c.k_pages || !c.v_pages || !c.table) return MOE_ERR_NULL;
  return aligned(c.k_pages, 16) && aligned(c.v_pages, 16) && aligned(c.table, 4) ? MOE_OK : MOE_ERR_ALIGN;
}
int log2_of(int page) {
  int n = 0;
  while (1 << n < page) ++n;
  return n;
}
constexpr int64_t kMaxPositions = (int64_t)1 << 28;

// Lays the partial states out in the workspace; returns its bytes.
size_t tree_carve(moe::TreeParams& p, void* ws, int ctas) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.rows = std::min(moe::kTreeRows, std::min(p.N, MOE_TREE_MAX_NEW) * (p.Hq / p.Hkv));
  const size_t parts = (size_t)ctas * moe::kTreeParts, states = parts * p.rows;
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t notes = 256, ml = notes + up(parts * sizeof(moe::TreePart)), o = ml + up(states * sizeof(float2));
  p.status = reinterpret_cast<int32_t*>(at);
  p.parts = reinterpret_cast<moe::TreePart*>(at + notes);
  p.part_ml = reinterpret_cast<float2*>(at + ml);
  p.part_o = reinterpret_cast<float*>(at + o);
  return o + states * p.d * sizeof(float);
}

bool tree_shape_supported(int N, int Hq, const moe_paged_t& c) {
  return N >= 0 && N < 1 << 24 && (c.d == 64 || c.d == 128 || c.d == 256) && Hq >= c.n_kv_heads &&
         Hq % c.n_kv_heads == 0 && Hq / c.n_kv_heads <= 16 && (int64_t)N * Hq < (int64_t)1 << 31 &&
         (int64_t)c.width * c.page * c.n_kv_heads < (int64_t)1 << 34;  // (a sequence's tiles in 32 bits)
}

}  // namespace

extern "C" {

int moe_qk_norm_rope(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, int T,
                     int n_q_heads, int n_kv_heads, int d, const uint16_t* q_weight,
                     const uint16_t* k_weight, float eps, const moe_rope_t* rope, uint16_t* q_out,
                     int64_t ldqo, uint16_t* k_out, int64_t ldko, void* stream) {
  if (T < 0 || n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > 1 << 20 || n_kv_heads > 1 << 20 || d < 8 || d > 256 || d % 8 != 0)
    return MOE_ERR_SHAPE;
  if ((int64_t)T * (n_q_heads + n_kv_heads) >= (int64_t)1 << 31) return MOE_ERR_SHAPE;
  if (!(eps > 0.f) || !std::isfinite(eps)) return MOE_ERR_SHAPE;
  const int64_t wq = (int64_t)n_q_heads * d, wk = (int64_t)n_kv_heads * d;
  if (n_q_heads > 0 && (!stride_ok(ldq, wq) || !stride_ok(ldqo, wq))) return MOE_ERR_SHAPE;
  if (n_kv_heads > 0 && (!stride_ok(ldk, wk) || !stride_ok(ldko, wk))) return MOE_ERR_SHAPE;
  moe::RopeParams p;
  memset(&p, 0, sizeof p);
  p.T = T;
  p.d = d;
  p.eps = eps;
  if (const int rc = enter_rope(p, rope, T, false); rc != MOE_OK) return rc;
  if (T == 0 || n_q_heads + n_kv_heads == 0) return MOE_OK;
  if ((n_q_heads > 0 && (!q || !q_out)) || (n_kv_heads > 0 && (!k || !k_out))) return MOE_ERR_NULL;
  if ((n_q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) || (n_kv_heads > 0 && (!aligned(k, 16) || !aligned(k_out, 16))) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return MOE_ERR_ALIGN;
  const int sms = device_sms();
  if (sms < 0) return sms;
  p.part[0] = {q, ldq, n_q_heads, q_weight, q_out, ldqo, p.pairs > 0};
  p.part[1] = {k, ldk, n_kv_heads, k_weight, k_out, ldko, p.pairs > 0};
  return cuda_status(moe::rope_launch(p, sms, static_cast<cudaStream_t>(stream)));
}

int moe_append_paged(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                     const int32_t* rows, int n_rows, int N, const int32_t* starts,
                     const int32_t* lens, const moe_paged_t* cache, const uint16_t* k_weight,
                     float eps, const moe_rope_t* rope, void* stream) {
  moe_paged_t c;
  if (const int rc = check_cache(cache, c, kMaxPositions); rc != MOE_OK) return rc;
  const int64_t width = (int64_t)c.n_kv_heads * c.d;
  if (N < 0 || n_rows < 0 || (!rows && n_rows != N) || (int64_t)N * c.n_kv_heads * 2 >= (int64_t)1 << 31) return MOE_ERR_SHAPE;
  if (!stride_ok(ldk, width) || !stride_ok(ldv, width)) return MOE_ERR_SHAPE;
  if (!(eps > 0.f) || !std::isfinite(eps)) return MOE_ERR_SHAPE;
  moe::RopeParams p;
  memset(&p, 0, sizeof p);
  p.T = N;
  p.d = c.d;
  p.eps = eps;
  if (const int rc = enter_rope(p, rope, N, true); rc != MOE_OK) return rc;
  if (N == 0) return MOE_OK;
  if (const int rc = check_cache_pointers(c); rc != MOE_OK) return rc;
  if (!starts || !lens || (n_rows > 0 && (!k || !v))) return MOE_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(rows, 4) || !aligned(starts, 4) || !aligned(lens, 4) ||
      !aligned(k_weight, 16))
    return MOE_ERR_ALIGN;
  const int sms = device_sms();
  if (sms < 0) return sms;
  p.part[0] = {k, ldk, c.n_kv_heads, k_weight, c.k_pages, 0, p.pairs > 0};
  p.part[1] = {v, ldv, c.n_kv_heads, nullptr, c.v_pages, 0, 0};
  p.starts = starts;
  p.lens = lens;
  p.rows = rows;
  p.n_rows = n_rows;
  p.table = c.table;
  p.ld_table = c.ld_table;
  p.page_stride = c.page_stride;
  p.position_stride = c.position_stride;
  p.head_stride = c.head_stride;
  p.B = c.n_sequences;
  p.width = c.width;
  p.n_pages = c.n_pages;
  p.page_log2 = log2_of(c.page);
  return cuda_status(moe::rope_launch(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_tree_attention_workspace_bytes(int N, int n_q_heads, const moe_paged_t* cache) {
  moe_paged_t c;
  if (check_cache(cache, c, kMaxPositions) != MOE_OK || !tree_shape_supported(N, n_q_heads, c)) return 0;
  moe::TreeParams p;
  memset(&p, 0, sizeof p);
  p.N = N;
  p.B = c.n_sequences;
  p.Hq = n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.d = c.d;
  return tree_carve(p, nullptr, moe::kTreeMaxSms);
}

int moe_tree_attention(const uint16_t* q, int64_t ldq, int N, int n_q_heads,
                       const int32_t* starts, const int32_t* lens, const int64_t* tree,
                       const moe_paged_t* cache, float scale, uint16_t* out, void* ws,
                       size_t ws_bytes, void* stream) {
  moe_paged_t c;
  if (const int rc = check_cache(cache, c, kMaxPositions); rc != MOE_OK) return rc;
  if (!tree_shape_supported(N, n_q_heads, c) || !stride_ok(ldq, (int64_t)n_q_heads * c.d)) return MOE_ERR_SHAPE;
  const float scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf((float)c.d)) * 1.4426950408889634f;
  if (!std::isfinite(scale) || !std::isfinite(scale_log2)) return MOE_ERR_SHAPE;
  if (N == 0) return MOE_OK;
  if (const int rc = check_cache_pointers(c); rc != MOE_OK) return rc;
  if (!q || !out || !starts || !lens) return MOE_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(starts, 4) || !aligned(lens, 4) || !aligned(tree, 8)) return MOE_ERR_ALIGN;
  if (!ws || !aligned(ws, 256) || ws_bytes < moe_tree_attention_workspace_bytes(N, n_q_heads, cache)) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms < 0) return sms;
  moe::TreeParams p;
  memset(&p, 0, sizeof p);
  p.q = q;
  p.ldq = ldq;
  p.k_pages = c.k_pages;
  p.v_pages = c.v_pages;
  p.page_stride = c.page_stride;
  p.position_stride = c.position_stride;
  p.head_stride = c.head_stride;
  p.ld_table = c.ld_table;
  p.table = c.table;
  p.starts = starts;
  p.lens = lens;
  p.tree = tree;
  p.N = N;
  p.B = c.n_sequences;
  p.Hq = n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.d = c.d;
  p.width = c.width;
  p.n_pages = c.n_pages;
  p.page_log2 = log2_of(c.page);
  p.scale_log2 = scale_log2;
  p.out = out;
  p.ctas = std::min(sms, moe::kTreeMaxSms);
  tree_carve(p, ws, moe::kTreeMaxSms);
  return cuda_status(moe::tree_launch(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
