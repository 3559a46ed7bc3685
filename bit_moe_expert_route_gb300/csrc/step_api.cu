// C ABI of the operators around the layer (include/step.h, and attention over
// a shared prefix in include/attn.h): argument checks and launches.
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"
#include "attn.h"
#include "step.h"

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  (void)cudaGetLastError();  // clear a non-sticky launch error
  return MOE_ERR_CUDA;
}

// The current device's SM count, or a status < 0. The attributes are looked
// up once a device (they are most of a small call's time on the host).
int device_sms() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev];  // 0 = not looked up
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  if (dev >= 0 && dev < kMaxDev) {
    const int v = known[dev].load(std::memory_order_relaxed);
    if (v) return v;
  }
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  const int r = major == 10 && minor == 3 ? sms : MOE_ERR_ARCH;
  if (dev >= 0 && dev < kMaxDev) known[dev].store(r, std::memory_order_relaxed);
  return r;
}

// A number that no other call has: from the clock and a random place, then counted.
uint64_t next_ticket() {
  static std::atomic<uint64_t> next{
      ((uint64_t)std::chrono::steady_clock::now().time_since_epoch().count() * 0x9E3779B97F4A7C15ull) ^
      (reinterpret_cast<uintptr_t>(&next_ticket) << 20)};
  uint64_t t = 0;
  while (t == 0) t = next.fetch_add(1, std::memory_order_relaxed);
  return t;
}
uint64_t* ticket_word(void* ws) {
  return ws ? reinterpret_cast<uint64_t*>(static_cast<int32_t*>(ws) + moe::kTicketWord) : nullptr;
}

// Lays the partial states out in the workspace; returns its bytes.
size_t prefix_carve(moe::PrefixParams& p, void* ws) {
  const size_t states = (size_t)(p.prefix_splits + p.suffix_splits) * p.B * p.Hq;
  p.status = static_cast<int32_t*>(ws);
  p.ticket_word = ticket_word(ws);
  p.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + 256);
  const size_t off = 256 + (states * sizeof(float2) + 255) / 256 * 256;
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + off);
  return off + states * p.d * sizeof(float);
}

}  // namespace

extern "C" {

int moe_add_rmsnorm_q8(const uint16_t* x, int64_t ldx, const uint16_t* residual,
                       const uint16_t* weight, int T, int d, float eps, int format,
                       uint16_t* residual_out, void* q, float* scale, uint16_t* values,
                       void* stream) {
  if (T < 0 || d < 8 || d > 16384 || d % 8 != 0 || ldx < d || ldx % 8 != 0) return MOE_ERR_SHAPE;
  if (format != MOE_Q8_INT8 && format != MOE_Q8_E4M3) return MOE_ERR_SHAPE;
  if (!(eps > 0.f) || !std::isfinite(eps)) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !weight || !q || !scale) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
      !aligned(residual_out, 16) || !aligned(q, 8) || !aligned(scale, 4) || !aligned(values, 16))
    return MOE_ERR_ALIGN;
  const int sms = device_sms();
  if (sms < 0) return sms;
  moe::NormParams p;
  p.x = x;
  p.ldx = ldx;
  p.residual = residual;
  p.weight = weight;
  p.T = T;
  p.d = d;
  p.eps = eps;
  p.e4m3 = format == MOE_Q8_E4M3;
  p.residual_out = residual_out;
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  p.values = values;
  return cuda_status(moe::norm_launch(p, sms, static_cast<cudaStream_t>(stream)));
}

static_assert(moe::kW8FewTokens == MOE_W8A8_NO_WORKSPACE_T, "the header's promise");

size_t moe_gemm_w8a8_workspace_bytes(int T, int N, int K) {
  if (T < 0 || N < 1 || K < 16 || K > 65536 || K % 16 != 0 || (int64_t)T * K >= (int64_t)1 << 40) return 0;
  // the status word, then the tokens' codes as f16
  return 256 + (moe::gemm_w8_few(T, N, K) ? 0 : ((size_t)T * K * 2 + 255) / 256 * 256);
}

int moe_gemm_w8a8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w,
                  const float* w_scale, int T, int N, int K, int type, void* out, int64_t ldo,
                  void* ws, size_t ws_bytes, void* stream) {
  const size_t need = moe_gemm_w8a8_workspace_bytes(T, N, K);
  if (need == 0 || lda < K || lda % 16 != 0 || ldo < N) return MOE_ERR_SHAPE;
  if (type != MOE_BF16 && type != MOE_F32) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return MOE_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(out, type == MOE_F32 ? 4 : 2))
    return MOE_ERR_ALIGN;
  if (ws ? !aligned(ws, 256) || ws_bytes < need : need > 256) return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms < 0) return sms;
  moe::GemmW8Params p;
  p.a = a;
  p.lda = lda;
  p.a_scale = a_scale;
  p.w = w;
  p.w_scale = w_scale;
  p.T = T;
  p.N = N;
  p.K = K;
  p.f32 = type == MOE_F32;
  p.out = out;
  p.ldo = ldo;
  p.status = static_cast<int32_t*>(ws);
  p.ticket_word = ticket_word(ws);
  p.ticket = next_ticket();
  p.a16 = ws ? reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + 256) : nullptr;
  return cuda_status(moe::gemm_w8_launch(p, sms, static_cast<cudaStream_t>(stream)));
}

int moe_token_logprobs(const void* logits, int type, int64_t ld, const int32_t* ids, int N, int V,
                       int k, float* logprob, float* entropy, int32_t* top_ids,
                       float* top_logprobs, void* stream) {
  if (type != MOE_BF16 && type != MOE_F32) return MOE_ERR_SHAPE;
  if (N < 0 || V < 1 || V >= 1 << 30 || ld < V || k < 0 || k > moe::kLogprobMaxK || k > V)
    return MOE_ERR_SHAPE;
  if (N == 0) return MOE_OK;
  if (!logits || (ids == nullptr) != (logprob == nullptr)) return MOE_ERR_NULL;
  if (k > 0 && (!top_ids || !top_logprobs)) return MOE_ERR_NULL;
  if (!aligned(logits, type == MOE_F32 ? 4 : 2) || !aligned(ids, 4) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4))
    return MOE_ERR_ALIGN;
  const int sms = device_sms();
  if (sms < 0) return sms;
  moe::LogprobParams p;
  p.logits = logits;
  p.ld = ld;
  p.ids = ids;
  p.N = N;
  p.V = V;
  p.k = k;
  p.f32 = type == MOE_F32;
  p.logprob = logprob;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  return cuda_status(moe::logprob_launch(p, sms, static_cast<cudaStream_t>(stream)));
}

static_assert(moe::kPrefixJoinedPositions == MOE_PREFIX_NO_WORKSPACE_POSITIONS, "the header's promise");

size_t moe_prefix_attention_workspace_bytes(int B, int P, int S, int n_q_heads, int n_kv_heads, int d) {
  if (!moe::prefix_shape_supported(B, P, S, n_q_heads, n_kv_heads, d)) return 0;
  moe::PrefixParams p;
  memset(&p, 0, sizeof p);
  p.B = B;
  p.P = P;
  p.S = S;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.d = d;
  if (moe::prefix_joined_blocks(B, P, S, n_kv_heads, d)) return 256;  // the status word, if one is wanted
  // the device's SM count decides the slices; the largest count has the most
  moe::prefix_plan(p, moe::kPrefixMaxSms);
  return prefix_carve(p, nullptr);
}

int moe_prefix_attention(const uint16_t* q, const uint16_t* k_prefix, const uint16_t* v_prefix,
                         int64_t ld_prefix, const uint16_t* k_suffix, const uint16_t* v_suffix,
                         int64_t seq_suffix, int64_t ld_suffix, const int32_t* lens, int B, int P,
                         int S, int n_q_heads, int n_kv_heads, int d, float scale, uint16_t* out,
                         void* ws, size_t ws_bytes, void* stream) {
  if (!moe::prefix_shape_supported(B, P, S, n_q_heads, n_kv_heads, d)) return MOE_ERR_SHAPE;
  const int64_t width = (int64_t)n_kv_heads * d;
  if (P > 0 && (ld_prefix < width || ld_prefix % 8 != 0)) return MOE_ERR_SHAPE;
  if (S > 0 && (ld_suffix < width || ld_suffix % 8 != 0 || seq_suffix < 0 || seq_suffix % 8 != 0))
    return MOE_ERR_SHAPE;
  if (std::isnan(scale) || std::isinf(scale)) return MOE_ERR_SHAPE;
  if (B == 0) return MOE_OK;
  if (!q || !out || (P > 0 && (!k_prefix || !v_prefix)) || (S > 0 && (!k_suffix || !v_suffix || !lens)))
    return MOE_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_prefix, 16) || !aligned(v_prefix, 16) ||
      !aligned(k_suffix, 16) || !aligned(v_suffix, 16) || !aligned(lens, 4))
    return MOE_ERR_ALIGN;
  moe::PrefixParams p;
  memset(&p, 0, sizeof p);
  p.q = q;
  p.kp = k_prefix;
  p.vp = v_prefix;
  p.ks = k_suffix;
  p.vs = v_suffix;
  p.ld_prefix = ld_prefix;
  p.ld_suffix = ld_suffix;
  p.seq_suffix = seq_suffix;
  p.lens = lens;
  p.B = B;
  p.P = P;
  p.S = S;
  p.Hq = n_q_heads;
  p.Hkv = n_kv_heads;
  p.d = d;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf((float)d)) * 1.4426950408889634f;
  p.out = out;
  p.joined = moe::prefix_joined_blocks(B, P, S, n_kv_heads, d);
  if (ws ? !aligned(ws, 256) || ws_bytes < moe_prefix_attention_workspace_bytes(B, P, S, n_q_heads, n_kv_heads, d)
         : !p.joined)
    return MOE_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms < 0) return sms;
  if (p.joined) {
    p.status = static_cast<int32_t*>(ws);
  } else {
    moe::prefix_plan(p, sms);
    prefix_carve(p, ws);
    p.ticket = next_ticket();
  }
  return cuda_status(moe::prefix_launch(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
