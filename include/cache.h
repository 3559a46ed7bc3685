/*
 * C ABI of the paged cache of keys and values (same library as moe.h:
 * libmoe_gb300.so): norms and position rotation of new queries and keys,
 * appending new tokens to the cache, and attention of a few new tokens a
 * sequence (one, or a tree of drafted ones) over it.
 *
 * Status codes, stream and ownership rules are those of moe.h. Every call
 * only enqueues work, and every launch is a programmatic dependent of the
 * previous one on its stream: it reads and writes nothing before that
 * launch's memory is visible.
 */
#ifndef MOE_GB300_CACHE_H
#define MOE_GB300_CACHE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ROPE_MAX_AXES 4

/*
 * A rotation of heads by their token's position (or by several: time, height and
 * width of a patch). Pair i < pairs of a head turns by
 *   angle_i = positions[axis(i)][token] * freqs[i]   (radians),
 *   a' = a cos(angle) - b sin(angle),  b' = a sin(angle) + b cos(angle),
 * (a, b) being elements (i, i + pairs), or, where `adjacent` is set, (2i, 2i + 1);
 * elements from 2 pairs on stay. Angles are reduced in whole numbers, so that
 * cos and sin are exact to fp32 (2^-22) at every int32 position.
 *   freqs         fp32 [pairs] device, below 2^16 in magnitude (any other makes its pair NaN)
 *   positions     int32 [n_axes][tokens] device, axes ld_positions elements apart (0: all
 *                 axes have the same)
 *   pairs         0 (no rotation) .. d / 2; a multiple of 8, of 4 if adjacent
 *   n_axes        1 .. 4
 *   sections      pairs of each axis, pairs in all: axis 0's come first, then axis
 *                 1's, ...; or, where `cyclic` is set, axis(i) = i % n_axes while
 *                 i < n_axes * sections[i % n_axes], and 0 for the rest (sections
 *                 of the axes from 1 on have to fit: n_axes * (sections[a] - 1) + a
 *                 < pairs)
 */
typedef struct moe_rope {
  const float* freqs;
  const int32_t* positions;
  int64_t ld_positions;
  int32_t pairs, n_axes;
  int32_t sections[MOE_ROPE_MAX_AXES];
  int32_t cyclic, adjacent;
} moe_rope_t;

/*
 * moe_qk_norm_rope: norms of each head's queries and keys and their rotation, in one
 * pass. Per token and head x of d elements:
 *   y = x / sqrt(mean(x^2) + eps) * weight   (y = x where the weight is NULL)
 * then y turned as above (not at all where rope is NULL), rounded to bf16 once.
 *   q, k       bf16 [T][n_heads][d], tokens ldq, ldk elements apart (views of a
 *              projection's output); k may be NULL (n_kv_heads 0), q too
 *   weights    bf16 [d] or NULL
 *   q_out      bf16 [T][n_q_heads][d], tokens ldqo apart; may be q itself (with ldqo
 *              = ldq); k_out likewise. Other overlaps are not allowed
 * All pointers but freqs and positions (4 bytes) 16-byte aligned, strides multiples
 * of 8 elements and at least n_heads * d; d a multiple of 8, 8 <= d <= 256; T >= 0 (0
 * launches nothing), T * heads < 2^31; eps > 0 and finite. fp32 arithmetic; a row
 * whose squares pass the fp32 range has its norm all the same. With a norm, a row with
 * an infinity has zeros for its finite elements and NaN for the infinite ones, before
 * it is turned; a row with a NaN is NaN. One launch.
 */
int moe_qk_norm_rope(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, int T,
                     int n_q_heads, int n_kv_heads, int d, const uint16_t* q_weight,
                     const uint16_t* k_weight, float eps, const moe_rope_t* rope, uint16_t* q_out,
                     int64_t ldqo, uint16_t* k_out, int64_t ldko, void* stream);

/*
 * A paged cache: position p of sequence b is place p % page of page
 * table[b][p / page].
 *   k_pages, v_pages  bf16, a page's place's head of d elements at
 *                     id * page_stride + place * position_stride + head * head_stride
 *                     (heads inside positions or positions inside heads; K and V alike)
 *   table             int32 [n_sequences][width] device, rows ld_table apart; entries
 *                     that no position needs are not read
 *   page              a power of two, 8 .. 4096
 * n_pages >= 1, 1 <= n_sequences <= 65535, 1 <= n_kv_heads <= 1024, width >= 1, width * page
 * <= 2^28
 */
typedef struct moe_paged {
  uint16_t *k_pages, *v_pages;
  int64_t page_stride, position_stride, head_stride;
  const int32_t* table;
  int64_t ld_table;
  int32_t n_pages, page, width, n_sequences, n_kv_heads, d;
} moe_paged_t;

/*
 * moe_append_paged: writes the new tokens' keys and values to the cache. Tokens
 * starts[b] .. starts[b + 1] - 1 are sequence b's, in order, and go to its positions
 * from lens[b] on. Keys are normed and turned on the way, as above (weight, rope or both
 * may be NULL); values are copied.
 *   k, v     bf16 [n_rows][n_kv_heads][d], rows ldk, ldv elements apart
 *   rows     int32 [N] device: token t's k and v are those of row rows[t] (a path of
 *            a tree of drafted tokens, say, appended again after it was accepted); or
 *            NULL: row t, and then n_rows has to be N
 *   starts   int32 [n_sequences + 1] device, rising, 0 .. N. Tokens outside starts[0] ..
 *            starts[n_sequences] - 1 belong to no sequence and are left out
 *   lens     int32 [n_sequences] device: positions in the cache before the call (below
 *            0 counts as 0). They are not changed
 *   rope     its positions may be NULL: a token turns by its position in the cache (with
 *            n_axes 1); else they are [n_axes][N], of token t
 * A token whose row is outside 0 .. n_rows - 1, whose position is past the table's width or
 * whose page is outside 0 .. n_pages - 1 is left out. k and v share no memory with the pages. Two tokens may not come to the same
 * place (sequences share no page that is written), and no two places, of K or V, share
 * elements. Sizes, alignment and arithmetic as above; strides of the cache multiples of 8 elements below 2^39, pages at a 16-byte
 * aligned address; table, starts, lens and rows 4-byte aligned. One launch.
 */
int moe_append_paged(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                     const int32_t* rows, int n_rows, int N, const int32_t* starts,
                     const int32_t* lens, const moe_paged_t* cache, const uint16_t* k_weight,
                     float eps, const moe_rope_t* rope, void* stream);

/*
 * moe_tree_attention: attention of sequences' new tokens over a paged cache that holds
 * them already (moe_append_paged, at positions lens[b] on). Token t of sequence b, the i-th
 * of its n = starts[b + 1] - starts[b] <= 64, attends to the positions before lens[b] and,
 * of the new ones, to position lens[b] + j (j < n) where bit j of tree[t] is set; where
 * tree is NULL, where j <= i.
 *   o_{t,h} = sum_j softmax_j(scale * q_{t,h} . k_{g,j}) v_{g,j},  g = h / (n_q_heads / n_kv_heads)
 *   q      bf16 [N][n_q_heads][d], tokens ldq elements apart (ldq a multiple of 8)
 *   tree   int64 [N] device, 8-byte aligned, or NULL
 *   scale  multiplies every score, finite and below 2^127; <= 0 means 1 / sqrt(d)
 *   out    bf16 [N][n_q_heads][d]. Tokens of no sequence are left as they were. Zeros for a
 *          row that attends to nothing or whose every score is -infinity. NaN for a row
 *          with a score that is NaN or +infinity, and for all rows of a sequence with more
 *          than 64 new tokens, with positions past the table's width, or with a page
 *          outside 0 .. n_pages - 1. What a position that a row does not attend to holds, infinities
 *          and NaN too, does not come into the row. An infinite value of one that it does attend to
 *          makes its element of the row that infinity, whatever the position's weight; infinities of both
 *          signs, or a NaN, make it NaN. (Weights are up to 2^10 until they are divided by their sum: sums
 *          of them times finite values that pass the fp32 range are infinite or NaN too)
 *   ws     256-byte aligned, >= moe_tree_attention_workspace_bytes (no initialisation
 *          needed), holds the status word; where the status says MOE_DEV_TIMEOUT, the rows
 *          not computed are NaN
 * out and ws overlap nothing else. Sequences may share pages. 0 <= N < 2^24 (0 launches nothing), width * page
 * below 2^34 / n_kv_heads, d in {64, 128, 256}, n_q_heads a multiple of n_kv_heads with at most 16 query heads a KV head.
 * Scores and softmax in fp32; the softmax weights multiply the values as two bf16 parts
 * (2^-16 of each weight), with fp32 sums. Two launches: partial states over slices of the
 * sequences, cut evenly over the SMs whatever their lengths, then their merge in a fixed
 * order.
 */
#define MOE_TREE_MAX_NEW 64
size_t moe_tree_attention_workspace_bytes(int N, int n_q_heads, const moe_paged_t* cache);
int moe_tree_attention(const uint16_t* q, int64_t ldq, int N, int n_q_heads,
                       const int32_t* starts, const int32_t* lens, const int64_t* tree,
                       const moe_paged_t* cache, float scale, uint16_t* out, void* ws,
                       size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_CACHE_H */
