/*
 * C ABI of the operators that surround the layer in a decode or scoring step
 * (same library as moe.h: libmoe_gb300.so): the residual norm with an 8-bit
 * output, the 8-bit matrix product that consumes it, and log probabilities
 * from the output head's logits. (Attention over a shared prefix is in
 * attn.h.)
 *
 * Status codes, stream and ownership rules are those of moe.h. Every call
 * only enqueues work, and every launch is a programmatic dependent of the
 * previous one on its stream: it reads and writes nothing before that
 * launch's memory is visible.
 */
#ifndef MOE_GB300_STEP_H
#define MOE_GB300_STEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of moe_gemm_w8a8's output and moe_token_logprobs' logits. */
enum moe_float_type { MOE_BF16 = 0, MOE_F32 = 1 };

/* 8-bit output formats of moe_add_rmsnorm_q8. */
enum moe_q8_format {
  MOE_Q8_INT8 = 0, /* whole numbers -127 .. 127                                */
  MOE_Q8_E4M3 = 1  /* 8-bit floats, 4 exponent and 3 fraction bits, up to 448  */
};

/*
 * moe_add_rmsnorm_q8: residual addition, root-mean-square norm and an 8-bit
 * output with one scale per token. Per row t of d elements:
 *   r = bf16(x + residual)            (r = x when residual is NULL)
 *   u = r * weight                    a = max |u|,  rms = sqrt(mean(r^2) + eps)
 *   q = round(u * top / a),  scale = a / (top * rms),  top = 127 (int8) or 448 (e4m3)
 * so q * scale stands for r / rms * weight. Rounding is to nearest, ties to
 * even, of the exact quotient, at any size of u (a product of two bf16 values is
 * exact in fp32, and rows of a < 2^-80 keep its exponent apart; quotients next to
 * a tie are compared with it exactly).
 *   x            bf16 [T][d], rows ldx elements apart (ldx >= d, multiple of 8)
 *   residual     bf16 [T][d] or NULL
 *   weight       bf16 [d]
 *   residual_out bf16 [T][d]: r; may be `residual` itself; NULL = not written
 *   q            8-bit codes [T][d];  scale fp32 [T]
 *   values       bf16 [T][d]: q * scale, for a consumer that reads bf16; or NULL
 * All but scale (4 bytes) and q (8 bytes) 16-byte aligned; d a multiple of 8,
 * 8 <= d <= 16384; T >= 0 (0 launches nothing); eps > 0 and finite (else
 * MOE_ERR_SHAPE). A row of zeros gives q 0 and scale 0; a row that holds an
 * infinity or a NaN, or whose squares or products pass the fp32 range, gives q
 * 0 and scale NaN (values NaN), so that what consumes it is NaN too. One
 * launch; fp32 arithmetic.
 */
int moe_add_rmsnorm_q8(const uint16_t* x, int64_t ldx, const uint16_t* residual,
                       const uint16_t* weight, int T, int d, float eps, int format,
                       uint16_t* residual_out, void* q, float* scale, uint16_t* values,
                       void* stream);

/*
 * moe_gemm_w8a8: product of 8-bit integers with scales,
 *   out[t][n] = a_scale[t] * w_scale[n] * sum_k a[t][k] * w[n][k]
 *   a        int8 [T][K], rows lda bytes apart (lda >= K, multiple of 16)
 *   a_scale  fp32 [T];  w int8 [N][K];  w_scale fp32 [N]
 *   out      bf16 or fp32 (`type`, moe_float_type) [T][N], rows ldo >= N
 *            elements apart
 *   ws       256-byte aligned, >= moe_gemm_w8a8_workspace_bytes(T, N, K) bytes
 *            (no initialisation needed), holds the status word; may be NULL
 *            where that is 256 (then nothing in the call can fail), always so
 *            for up to MOE_W8A8_NO_WORKSPACE_T tokens. Where the status says
 *            MOE_DEV_TIMEOUT, what was not computed is NaN
 * a and w 16-byte aligned; T >= 0 (0 launches nothing), N >= 1, K a multiple of
 * 16, 16 <= K <= 65536, T * K < 2^40. The integer sum is exact while its
 * partial sums stay below 2^24 in magnitude (always for K <= 1024); a larger one is
 * held in fp32, and each step of 16 codes may cost it 2^-23 of itself (the tensor
 * cores may truncate). The scales multiply it in fp32 and the result is rounded
 * once. One launch for few tokens or little work, else two.
 */
#define MOE_W8A8_NO_WORKSPACE_T 24
size_t moe_gemm_w8a8_workspace_bytes(int T, int N, int K);
int moe_gemm_w8a8(const int8_t* a, int64_t lda, const float* a_scale, const int8_t* w,
                  const float* w_scale, int T, int N, int K, int type, void* out, int64_t ldo,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * moe_token_logprobs: per row of logits z [V], with lse = log sum exp(z):
 *   logprob      fp32 [N]: z[id] - lse of the row's token id (int32 [N]; NaN for
 *                an id outside 0 .. V-1). ids and logprob may both be NULL.
 *   entropy      fp32 [N]: -sum p log p, p = exp(z - lse); or NULL
 *   top_ids      int32 [N][k]: the k largest logits, ties to the lower index
 *   top_logprobs fp32 [N][k]: their log probabilities
 *                (both NULL when k == 0)
 *   logits       bf16 or fp32 (`type`, moe_float_type) [N][V], rows ld >= V
 *                elements apart, aligned to their element size only
 * 1 <= V < 2^30, 0 <= k <= min(32, V), N >= 0 (0 launches nothing). A logit of
 * -infinity has probability 0; a row of nothing else gives entropy 0 and log
 * probabilities of -infinity. A row that holds +infinity or a NaN gives NaN in
 * logprob, entropy and top_logprobs; a NaN ranks below every number in top_ids.
 * One launch: a row is one block's, or, with few rows, a cluster's of up to 8
 * blocks. Each logit is read once. fp32 arithmetic.
 */
int moe_token_logprobs(const void* logits, int type, int64_t ld, const int32_t* ids, int N, int V,
                       int k, float* logprob, float* entropy, int32_t* top_ids,
                       float* top_logprobs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_STEP_H */
