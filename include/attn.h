/*
 * C ABI of batch-1 decode attention with grouped KV heads (same library as
 * moe.h: libmoe_gb300.so).
 *
 * "Perplexity's Lily Beats MLX-LM by 1.35x Running Qwen3.6 on Apple Silicon":
 * section "What Lily actually does" (10 of the model's 40 layers are full
 * attention) and section "Decode optimizations", the GQA paragraph (eight
 * query heads share one KV head; packing the query heads of a group into one
 * threadgroup lets them share the KV loads). The page gives no formula; this
 * is scaled dot-product attention of one new token over L cached positions:
 *
 *   o_h = sum_j softmax_j(scale * q_h . k_{g,j}) v_{g,j},  g = h / (n_q_heads / n_kv_heads)
 *
 * Status codes, stream and ownership rules are those of moe.h.
 */
#ifndef MOE_GB300_ATTN_H
#define MOE_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes moe_decode_attention needs for these sizes (an upper bound that
   does not depend on the GPU); 0 for unsupported sizes. */
size_t moe_decode_attention_workspace_bytes(int L, int n_q_heads, int n_kv_heads, int d);

/*
 * moe_decode_attention: out = attention of the new token's queries over the
 * cache.
 *   q      bf16 [n_q_heads][d] device, 16-byte aligned
 *   K, V   bf16 [L][n_kv_heads][d] device (position-major, as appended per
 *          token), 16-byte aligned
 *   scale  multiplies every score; <= 0 means 1 / sqrt(d)
 *   out    fp32 [n_q_heads][d] device
 *   ws     device, 4-byte aligned, >= moe_decode_attention_workspace_bytes
 * L >= 1; d in {64, 128, 256}; n_q_heads a multiple of n_kv_heads with at most
 * 8 query heads per KV head. Others: MOE_ERR_SHAPE. Two launches: a split
 * kernel (one block per KV head and slice of the cache, all of the head's
 * query heads together; online softmax per warp, at least 8 positions per
 * warp, the warps' states merged in a fixed order into one partial per block
 * and query head) and a combine kernel (one block per query head and 32
 * outputs, merging the partials with fixed-order block reductions). fp32
 * arithmetic.
 */
int moe_decode_attention(const uint16_t* q, const uint16_t* K, const uint16_t* V, int L,
                         int n_q_heads, int n_kv_heads, int d, float scale, float* out, void* ws,
                         size_t ws_bytes, void* stream);

/*
 * moe_prefix_attention: decode attention of one new token for each of B
 * sequences that share a prefix of P cached positions and have len[b] positions
 * of their own after it. The prefix is read once for all sequences.
 *   o_{b,h} = sum_j softmax_j(scale * q_{b,h} . k_{g,j}) v_{g,j}
 * over the prefix's positions and sequence b's own, g = h / (n_q_heads / n_kv_heads).
 *   q                   bf16 [B][n_q_heads][d]
 *   k_prefix, v_prefix  bf16 [P][n_kv_heads][d], positions ld_prefix elements
 *                       apart (at least n_kv_heads * d); may be NULL when P == 0
 *   k_suffix, v_suffix  bf16 [B][S][n_kv_heads][d], positions ld_suffix and
 *                       sequences seq_suffix elements apart; NULL when S == 0.
 *                       Positions from len[b] on are not read.
 *   lens                int32 [B] device, 0 .. S (others are clamped); NULL when S == 0
 *   scale               multiplies every score; <= 0 means 1 / sqrt(d)
 *   out                 bf16 [B][n_q_heads][d]; zeros for a sequence without any
 *                       position (P == 0 and len[b] == 0), and for a row whose
 *                       every score is -infinity; NaN for a row with a score that
 *                       is NaN or +infinity
 *   ws                  256-byte aligned, >= moe_prefix_attention_workspace_bytes
 *                       (no initialisation needed), holds the status word.
 *                       May be NULL where little work takes one launch (then
 *                       nothing in it can fail); MOE_ERR_WORKSPACE says that it
 *                       may not, before anything is enqueued. Where the status
 *                       says MOE_DEV_TIMEOUT, the rows not computed are NaN
 * All pointers but lens (4 bytes) 16-byte aligned, strides multiples of 8
 * elements. 0 <= B <= 65535 (0 launches nothing), P and S up to 2^28, d in {64,
 * 128, 256}, n_q_heads a multiple of n_kv_heads with at most 16 query heads a
 * KV head. Scores and softmax in fp32; the softmax weights multiply the values as
 * two bf16 parts (2^-16 of each weight), with fp32 sums. Up to three launches: with little
 * work one, of clusters that merge their slices; else partial
 * states over slices of the prefix and of the sequences' own positions (with
 * more than 32 query rows a KV head the prefix has a launch of its own), then
 * their merge in a fixed order. Each is a programmatic dependent of the launch
 * before it on the stream.
 */
#define MOE_PREFIX_NO_WORKSPACE_POSITIONS 2048 /* with P + S above it, a workspace is always needed */
size_t moe_prefix_attention_workspace_bytes(int B, int P, int S, int n_q_heads, int n_kv_heads, int d);
int moe_prefix_attention(const uint16_t* q, const uint16_t* k_prefix, const uint16_t* v_prefix,
                         int64_t ld_prefix, const uint16_t* k_suffix, const uint16_t* v_suffix,
                         int64_t seq_suffix, int64_t ld_suffix, const int32_t* lens, int B, int P,
                         int S, int n_q_heads, int n_kv_heads, int d, float scale, uint16_t* out,
                         void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif
