// Attention of sequences' new tokens (one, or a tree of drafted ones) over a paged cache.
//
//   o_{t,h} = sum_j softmax_j(scale q_{t,h} . k_j) v_j  over the positions before the
//   sequence's new tokens, and those of its new tokens that bits of a mask name.
//
// The n G query rows of a sequence that read one KV head (G query heads of each of n
// tokens) form one matrix, in tiles of 128 rows: each K and V tile is read once for
// all of them. Bound by HBM up to 128 rows (the MMAs of a tile of 64 KB take 1824 cycles
// at head size 256, 1536 at 128, against about 3000 that an SM's share of HBM needs for it);
// with more rows the MMAs are two thirds of the time (4 sequences of 64 tokens, 4 row tiles: 94 of 150 us).
//
// Work is cut by key tiles, not by sequences: the tiles of all (sequence, KV head, row
// tile) items, one behind another, go in equal runs to one persistent CTA an SM. Lengths
// are known on the device only, so every CTA sums the sequences' tiles and finds its own
// run. What a CTA has of an item is a segment. A whole item's output is written at once;
// a part's state (m, l, o) goes to the workspace with a note of whose it is, and a second
// kernel merges the parts.
//
// Row tiles of one KV head read the same keys. Where there are several, long items are cut into
// chunks of about a run, and a chunk's row tiles stand next to one another: the CTAs that have
// them go over the same keys at the same time, and HBM is read once. (4 sequences of 64
// tokens over up to 50001 positions, 4 row tiles: 188 us with an item's tiles in one piece.)
//
// A segment: S = Q K^T into tensor memory, weights P = 2^(scale S - m) over the scores as
// two bf16 parts (of 32 keys each, one behind the other, where their scores were), O += P V
// with P as the MMA's A operand from tensor memory. One thread
// issues the scores' products, another the outputs', three tiles behind at most. K and V
// tiles come by TMA, a box a page (or a tile, where pages are longer), through one ring of
// slots in the order K0 K1 V0 K2 V1 ... that runs on through the segments, so that the next
// segment's tiles land while this one ends. Which segments there are one thread works out
// ahead of the others, who read it from shared memory.
//
// The code is kept short (waits that wait and what happens once a segment out of line, loops
// rolled): with 130 KB of it, a call of few tiles spent most of its time fetching instructions, and
// so did the softmax warps (64 sequences over 4096 positions 154 us).
//
// What rows do not attend to: scores are set to -infinity by the row's mask, whatever they
// were. In V, a weight of 0 would still make NaN of an infinity or a NaN. Rows past the
// sequence's end (a page's rest) are set to 0 in shared memory; so are infinite and NaN elements of the
// new tokens' V, and rows that do attend to such a token have the element added at the end. Cached positions, which
// all rows attend to, are looked through for such elements where an output is not finite.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTrThreads = 256;  // warp 0 TMA, warps 1 and 2 MMA, warps 4-7 softmax
constexpr float kMostSum = 1024.f;  // of 64 weights, from which on their reference moves
constexpr int kBadRing = 16;     // tiles whose pages are known to be bad or not: more than the ring holds

template <int D>
struct TrCfg {
  static constexpr int KT = D == 256 ? 64 : 128;    // keys a tile
  static constexpr int kSlot = KT * D * 2;          // K or V of a tile
  static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 6 : 8;
  static constexpr int kQ = kTreeRows * D * 2;
  static constexpr int kBufs = 3;                   // tiles between their scores and their outputs
  static constexpr int kSegs = 4;                   // segments that are worked out ahead
  static constexpr int kOffSlots = kQ;
  static constexpr int kOffBar = kOffSlots + kSlots * kSlot;
  static constexpr int kBars = 2 * kSlots + 2 + 3 * kBufs + 1 + 2 * kSegs;
  static constexpr int kSmem = kOffBar + (8 * kBars + 15) / 16 * 16 + 512 + 1024;
  static constexpr int kColS = D;                   // tensor memory: O, then the score buffers
  static_assert(kColS + kBufs * KT <= 512, "tensor memory exceeded");
  static_assert(kSmem <= 232448, "shared memory exceeded");
  // V of tile i takes the slot that load 2 i + 2 - kSlots had: that has to be one whose landing the outputs' issuer
  // knows of (K of tile i - 1 or an earlier load), or its wait for V would take the phase before for this one.
  static_assert(kSlots >= 4, "a wait may be two phases ahead of its barrier");
  static_assert(kSlots < kBadRing, "a tile's note is overwritten before it is read");
};

struct TrArgs {
  CUtensorMap tm_k, tm_v;
  TreeParams p;
  int box_log2;    // keys a box: min(page, KT)
  int heads_out;   // the map's axes: d, place, head, page (else d, head, place, page)
};

// A sequence's new tokens and cached positions, and how many tiles they make.
struct Sequence {
  int tok0, n, L;
  bool bad;  // too many new tokens, or positions past the table
};
MOE_DEVINL Sequence sequence_of(const TreeParams& p, int b) {
  Sequence s;
  s.tok0 = min(max(p.starts[b], 0), p.N);
  s.n = max(0, min(max(p.starts[b + 1], 0), p.N) - s.tok0);
  s.L = max(0, p.lens[b]);
  s.bad = s.n > MOE_TREE_MAX_NEW || (int64_t)s.L + s.n > ((int64_t)p.width << p.page_log2);
  return s;
}
template <int KT>
MOE_DEVINL int key_tiles(const Sequence& s) {
  return (int)(((int64_t)s.L + s.n + KT - 1) / KT);
}
MOE_DEVINL int row_tiles(const TreeParams& p, const Sequence& s) {
  return (s.n * (p.Hq / p.Hkv) + kTreeRows - 1) / kTreeRows;
}
template <int KT>
MOE_DEVINL int64_t tiles_of(const TreeParams& p, const Sequence& s) {
  return s.bad || s.n == 0 ? 0 : (int64_t)p.Hkv * row_tiles(p, s) * key_tiles<KT>(s);
}

// CTA `cta`'s run begins here. With fewer tiles than CTAs the first `tiles` have one each.
MOE_DEVINL int64_t run_begin(int64_t tiles, int cta, int ctas) {
  return tiles <= ctas ? min((int64_t)cta, tiles) : tiles * cta / ctas;
}

// What a CTA has of an item: keys k0 .. k1 - 1 (in tiles) of `rows` query rows from row0 on.
struct alignas(16) Segment {
  int64_t item;  // as no other's
  int b, tok0, n, L, h, row0, rows, k0, k1, whole;
};

// A CTA's run of tiles, segment by segment. A sequence's tiles in order: KV head, chunk of
// keys, row tile, key. (A sequence has fewer than 2^31.)
template <int KT>
struct Walk {
  int64_t cur, end, base;  // of all tiles: the next, the run's end, this sequence's first
  uint32_t count, run;     // this sequence's tiles; the longest run's
  int b;
  Sequence s;
  uint32_t kt, rt, chunks, size, longer;  // chunks of `size` tiles, the first `longer` of them of one more
  MOE_DEVINL void start(const TreeParams& p, const int64_t* found, const Sequence& first) {
    cur = found[0], end = found[1], b = (int)found[2], base = found[3], run = (uint32_t)found[4];
    s = first;
    load(p);
  }
  MOE_DEVINL void load(const TreeParams& p) {
    kt = key_tiles<KT>(s), rt = row_tiles(p, s), count = (uint32_t)tiles_of<KT>(p, s);
    // chunks of 3/4 to 3/2 of a run
    chunks = rt > 1 ? max(1u, (2 * kt + run) / (2 * run)) : 1u;
    size = kt / chunks;
    longer = kt - size * chunks;
  }
  MOE_DEVINL bool next(const TreeParams& p, Segment& g) {
    if (cur >= end) return false;
    while (cur >= base + count) {
      if (b + 1 >= p.B) return false;  // (only if the lengths changed under the kernel)
      base += count;
      s = sequence_of(p, ++b);
      load(p);
    }
    const uint32_t head = kt * rt, off = (uint32_t)(cur - base), h = off / head, in = off - h * head, x = in / rt;
    const uint32_t chunk = x < longer * (size + 1) ? x / (size + 1) : longer + (x - longer * (size + 1)) / size;
    const uint32_t from = chunk * size + min(chunk, longer), length = size + (chunk < longer);
    const uint32_t at = in - from * rt, row = at / length, k0 = from + at - row * length;
    const uint32_t n = (uint32_t)min((int64_t)(from + length - k0), end - cur);
    cur += n;
    g.item = base + (int64_t)(h * rt + row) * kt;
    g.b = b, g.tok0 = s.tok0, g.n = s.n, g.L = s.L;
    g.h = (int)h;
    g.row0 = (int)row * kTreeRows;
    g.rows = min(kTreeRows, s.n * (p.Hq / p.Hkv) - g.row0);
    g.k0 = (int)k0, g.k1 = (int)(k0 + n);
    g.whole = n == kt;
    return true;
  }
};

// The note of a part, other than its item.
MOE_DEVINL int what_of(const Segment& g) { return g.h << 16 | g.row0 / kTreeRows << 12 | (g.rows - 1) << 4 | (g.k0 == 0); }

// mbar_wait, out of line where it has to wait.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status, int where) {
  return mbar_wait(bar, parity, abort, status, where);
}
MOE_DEVINL bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status, int where) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort, status, where);
}
MOE_DEVINL bool warp_wait_for(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status, int where) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort, status, where));
}

// After a wait that ran out: NaN for what the run has from its seg-th segment on, by the 128
// softmax threads (`parts` of its parts have states already).
template <int KT>
__device__ __noinline__ void give_up(const TreeParams& p, const int64_t* found, const Sequence* first, int seg, int parts, int tid) {
  Walk<KT> walk;
  walk.start(p, found, *first);
  Segment g;
  const int G = p.Hq / p.Hkv;
  TreePart* notes = p.parts + (int64_t)blockIdx.x * kTreeParts;
  for (int i = 0; walk.next(p, g); ++i) {
    if (i < seg) continue;
    if (g.whole) {
      for (int r = tid; r < g.rows; r += 128) {
        const int x = g.row0 + r;
        uint4* out = reinterpret_cast<uint4*>(p.out + ((int64_t)(g.tok0 + x / G) * p.Hq + g.h * G + x % G) * p.d);
        for (int c = 0; c < p.d / 8; ++c) out[c] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
      }
    } else if (parts < kTreeParts) {
      if (tid < g.rows) p.part_ml[((int64_t)blockIdx.x * kTreeParts + parts) * p.rows + tid] = make_float2(0.f, __int_as_float(0x7fc00000));
      if (tid == 0) notes[parts] = TreePart{g.item, g.tok0, what_of(g)};
      ++parts;
    }
  }
  if (tid == 0)
    for (; parts < kTreeParts; ++parts) notes[parts].item = -1;
}

MOE_DEVINL bool not_finite2(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }

// Elements of new tokens' V that are not finite, for the rows that attend to them (a row a lane).
template <int D, int KT>
__device__ __noinline__ void add_not_finite(const TreeParams& p, const Segment& g, uint32_t tmem, uint64_t bits, bool mine) {
  const int64_t from = max((int64_t)g.k0 * KT, (int64_t)g.L), to = min((int64_t)g.k1 * KT, (int64_t)g.L + g.n);
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld_32x32b_x16(tmem + c, o);
    tc_wait_ld();
#pragma unroll 1
    for (int64_t at = from; at < to; ++at) {
      if (!mine || !(bits >> (at - g.L) & 1)) continue;
      const int64_t id = p.table[g.b * p.ld_table + (at >> p.page_log2)];
      const uint16_t* v = p.v_pages + id * p.page_stride + (at & ((1 << p.page_log2) - 1)) * p.position_stride + g.h * p.head_stride + c;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float x = bf16_bits_to_f32(v[j]);
        if (!(fabsf(x) <= 3.4e38f)) o[j] = __float_as_uint(__uint_as_float(o[j]) + x);
      }
    }
    __syncwarp();
    tmem_st_32x32b_x16(tmem + c, o);
  }
  tc_wait_st();
}

// Outputs where cached values are infinite or NaN. The weights' two parts make NaN of most of them (the second is as often
// negative or 0 as not), so the columns are looked for in the segment's cached V, all of which every row attends
// to, and set: an infinity where those of a column are of one sign, else NaN. Only where outputs are not finite: a warp reads
// the segment's V once more (8 x 16 tokens over 32768 positions 630 us instead of 79).
template <int D, int KT>
__device__ __noinline__ void show_not_finite(const TreeParams& p, const Segment& g, uint32_t tmem) {
  constexpr int kLanes = D / 8;  // of a position: 8 columns each
  const int lane = threadIdx.x & 31;
  const int64_t to = min((int64_t)g.k1 * KT, (int64_t)g.L);
  const uint16_t* v = p.v_pages + g.h * p.head_stride + lane % kLanes * 8;
  uint32_t signs = 0;  // of this lane's columns: + infinity, 8 bits on - infinity; NaN is both
#pragma unroll 1
  for (int64_t at0 = (int64_t)g.k0 * KT + lane / kLanes; at0 < to; at0 += 8 * (32 / kLanes)) {
    int64_t at[8];
    int id[8];
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      at[i] = min(at0 + i * (32 / kLanes), to - 1);  // (the last one again past the end)
      id[i] = p.table[g.b * p.ld_table + (at[i] >> p.page_log2)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const uint4*>(v + id[i] * p.page_stride + (at[i] & ((1 << p.page_log2) - 1)) * p.position_stride);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(not_finite2(x[i].x) || not_finite2(x[i].y) || not_finite2(x[i].z) || not_finite2(x[i].w))) continue;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t e = w[j / 2] >> (j & 1) * 16 & 0xFFFFu;
        if ((e & 0x7FFFu) > 0x7F80u) signs |= 0x101u << j;
        if (e == 0x7F80u) signs |= 1u << j;
        if (e == 0xFF80u) signs |= 0x100u << j;
      }
    }
  }
#pragma unroll
  for (int off = kLanes; off < 32; off *= 2) signs |= __shfl_xor_sync(0xffffffffu, signs, off);
  if (!__any_sync(0xffffffffu, signs != 0)) return;
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    const uint32_t of[2] = {__shfl_sync(0xffffffffu, signs, c / 8), __shfl_sync(0xffffffffu, signs, c / 8 + 1)};
    if ((of[0] | of[1]) == 0) continue;
    uint32_t o[16];
    tmem_ld_32x32b_x16(tmem + c, o);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t sign = of[j / 8] >> j % 8 & 0x101u;
      if (sign) o[j] = sign == 1u ? 0x7F800000u : sign == 0x100u ? 0xFF800000u : 0x7FC00000u;
    }
    tmem_st_32x32b_x16(tmem + c, o);
  }
  tc_wait_st();
}

// Which of the 32 positions from the rel-th new token on (rel < 0: cached ones before) a
// row with the mask `bits` attends to.
MOE_DEVINL uint32_t attended(int64_t rel, uint64_t bits) {
  if (rel <= -32) return 0xFFFFFFFFu;
  if (rel < 0) return (uint32_t)((bits << -rel) | ((1ull << -rel) - 1));
  return rel < 64 ? (uint32_t)(bits >> rel) : 0u;
}

// The scores of a tile that rows do not attend to: -infinity.
template <int KT>
__device__ __noinline__ void mask_scores(uint32_t cols, int64_t rel, uint64_t bits) {
#pragma unroll 1
  for (int c = 0; c < KT; c += 32) {
    uint32_t s[32];
    tmem_ld_32x32b_x32(cols + c, s);
    tc_wait_ld();
    const uint32_t in = attended(rel + c, bits);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!(in >> j & 1)) s[j] = 0xFF800000u;
    tmem_st_32x32b_x32(cols + c, s);
  }
  tc_wait_st();
}

// A row's softmax so far: its reference m and sum l, and how weights are taken: 2^(scale s - at), at = m (0
// without any score yet). Scores are scaled apart where m is large (scale 1): what the fused
// product leaves of its rounding would pass 2^-8.
struct Running {
  float m, l, at, scale;
};

// The reference m of each row moves up to the largest of the 64 scores from column c on (by whole steps of
// log2, so that what there is scales without rounding): the sum, the tile's weights so far and, where there
// are any, the outputs, whose products are complete.
template <int D>
__device__ __noinline__ Running move_reference(uint32_t cols, int c, uint32_t outputs, bool any_output, float scale_log2, float m, float l) {
  float top = -INFINITY;
  {
    tc_wait_st();
#pragma unroll 1
    for (int e = 0; e < 64; e += 32) {
      uint32_t s[32];
      tmem_ld_32x32b_x32(cols + c + e, s);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(s[j]));
    }
  }
  const float nm = fmaxf(m, ceilf(__fmul_rn(top, scale_log2)));
  // 2^(m - nm), exactly
  const float f = nm == -INFINITY ? 1.f : m - nm < -126.f ? 0.f : __int_as_float((127 + (int)(m - nm)) << 23);
  l *= f;
#pragma unroll 1
  for (int e = 0; e < c; e += 16) {
    uint32_t w[16];
    tmem_ld_32x32b_x16(cols + e, w);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_bf16(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f);
    tmem_st_32x32b_x16(cols + e, w);
  }
  if (any_output) {
    tc_fence_after();
#pragma unroll 1
    for (int e = 0; e < D; e += 16) {
      uint32_t o[16];
      tmem_ld_32x32b_x16(outputs + e, o);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
      tmem_st_32x32b_x16(outputs + e, o);
    }
  }
  tc_wait_st();
  const float at = nm == -INFINITY ? 0.f : nm;
  return {nm, l, at, __any_sync(0xffffffffu, fabsf(at) >= 65536.f) ? 1.f : scale_log2};
}

template <int D>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const __grid_constant__ TrArgs args) {
  using C = TrCfg<D>;
  constexpr int KT = C::KT, NS = C::kSlots, NB = C::kBufs, NG = C::kSegs;
  const TreeParams& p = args.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [NS] a slot's tile has landed
  uint64_t* empty = full + NS;                                      // [NS] its products are done
  uint64_t* q_full = empty + NS;                                    // [1] a segment's queries are there
  uint64_t* v_ready = q_full + 1;                                   // [1] a tile's V has no infinities or NaN of new tokens
  uint64_t* s_full = v_ready + 1;                                   // [NB] scores are complete
  uint64_t* p_full = s_full + NB;                                   // [NB] weights are written, over the scores
  uint64_t* pv_done = p_full + NB;                                  // [NB] their product is complete: the columns are free
  uint64_t* drain = pv_done + NB;                                   // [1]
  uint64_t* g_full = drain + 1;                                     // [NG] a segment is worked out
  uint64_t* g_empty = g_full + NG;                                  // [NG] all have read it
  Segment* segments = reinterpret_cast<Segment*>(smem + C::kOffBar + (8 * C::kBars + 15) / 16 * 16);  // [NG]
  int64_t* found = reinterpret_cast<int64_t*>(segments + NG);       // the run: first tile, end, sequence, its first tile, the longest's tiles
  int64_t* sums = found + 5;                                        // [8] a warp's tiles
  Sequence* first_seq = reinterpret_cast<Sequence*>(sums + 8);      // the run's first
  int* bad_tile = reinterpret_cast<int*>(first_seq + 1);            // [kBadRing] 1 + tile of the run with a bad page
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bad_tile + kBadRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* v_bad = abort_flag + 1;  // 1 + segment whose new V holds infinities or NaN
  static_assert(NG * sizeof(Segment) + 13 * 8 + sizeof(Sequence) + kBadRing * 4 + 12 <= 512, "shared memory exceeded");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * NS; ++i) mbar_init(&full[i], 1);
    mbar_init(q_full, 4);
    mbar_init(v_ready, 4);
    for (int i = 0; i < NB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 2);
    for (int i = 0; i < NG; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], 7);  // TMA, two issuers, four softmax warps
    }
    found[0] = found[1] = 0;
    *abort_flag = 0;
    *v_bad = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tm_k);
    tma_prefetch_desc(&args.tm_v);
  }
  if (threadIdx.x < kBadRing) bad_tile[threadIdx.x] = 0;
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The run: the sum of all sequences' tiles, then where its share of it begins.
  {
    int64_t total = 0, all = 0, from = 0, to = 0;
    int bad = 0;
    // (256 sequences at a time; more than those are gone through twice)
    const int rounds = p.B > kTrThreads ? 2 : 1;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      total = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < p.B; b0 += kTrThreads) {
        const int b = b0 + threadIdx.x;
        Sequence s;
        int64_t mine = 0;
        if (b < p.B) {
          s = sequence_of(p, b);
          mine = tiles_of<KT>(p, s);
          bad |= s.bad;
        }
        int64_t upto = mine;  // of the warp's lanes up to this one
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
          const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += v;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int64_t first = total + upto - mine;
#pragma unroll
        for (int w = 0; w < kTrThreads / 32; ++w) {
          if (w < warp) first += sums[w];
          total += sums[w];
        }
        if (rounds == 1 || (round == 0 && b0 + kTrThreads >= p.B)) {
          all = total;
          from = run_begin(all, blockIdx.x, p.ctas), to = run_begin(all, blockIdx.x + 1, p.ctas);
        }
        if (round + 1 == rounds && from < to && first <= from && from < first + mine) {
          found[0] = from, found[1] = to, found[2] = b, found[3] = first;
          found[4] = min((all + p.ctas - 1) / p.ctas, (int64_t)1 << 28);
          *first_seq = s;
        }
        if (rounds > 1) __syncthreads();
      }
    }
    if (__syncthreads_or(bad)) {  // sequences that cannot be right: NaN, by all CTAs
#pragma unroll 1
      for (int b = 0; b < p.B; ++b) {
        const Sequence s = sequence_of(p, b);
        if (!s.bad) continue;
        const int64_t words = (int64_t)s.n * p.Hq * (D / 8);
        uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)s.tok0 * p.Hq * D);
#pragma unroll 1
        for (int64_t i = (int64_t)blockIdx.x * kTrThreads + threadIdx.x; i < words; i += (int64_t)p.ctas * kTrThreads)
          out[i] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
      }
    }
  }
  const int total = (int)(found[1] - found[0]);  // tiles of the run
  TreePart* const parts = p.parts + (int64_t)blockIdx.x * kTreeParts;

  // Segment number i, once it is worked out; false after the last (rows 0) and after a wait that ran out.
  // (Each reader, once it has copied it, says so on g_empty.)
  auto segment = [&](int i, Segment& g) {
    if (!wait_for(&g_full[i % NG], (i / NG) & 1, abort_flag, p.status, 115)) return g.rows = 0, false;
    g = segments[i % NG];
    return g.rows > 0;
  };

  if (total == 0) {  // fewer tiles than CTAs
    if (threadIdx.x < kTreeParts) parts[threadIdx.x].item = -1;
  } else if (warp == 3) {
    if (lane == 0) {
      Walk<KT> walk;
      walk.start(p, found, *first_seq);
      Segment g;
#pragma unroll 1
      for (int i = 0;; ++i) {
        const bool more = walk.next(p, g);
        if (!more) g.rows = 0;
        if (i >= NG && !wait_for(&g_empty[i % NG], (i / NG - 1) & 1, abort_flag, p.status, 116)) break;
        segments[i % NG] = g;
        mbar_arrive(&g_full[i % NG]);
        if (!more) break;
      }
    }
  } else if (warp == 0) {
    fence_proxy_async_global();  // the pages are written by ordinary stores of earlier launches
    // Keys leave L2 first: they are read once, or by the next CTAs at about the same time (8 sequences of 16
    // tokens over 32768 positions 77 us, without a policy 84; 4 of 64 over 50001, four row tiles, 153 and 155).
    const uint64_t policy = l2_policy_evict_first();
    const int pieces_log2 = (KT == 64 ? 6 : 7) - args.box_log2, pieces = 1 << pieces_log2;
    // a lane's box of each tile: 64 columns, one page's (or the tile's) positions
    const int piece = lane & (pieces - 1), col = lane >> pieces_log2;
    const bool mine = col < D / 64;
    const uint32_t dst = col * (KT * 128) + ((piece << args.box_log2) * 128);
    int slot = 0, phase = 1, loads = 0, seg = -1, key = 0;
    Segment g;
    g.k1 = 0;
    struct Tile {
      int h, place, page;
      bool bad;
    };
    // A tile's page, looked up a tile ahead; past the sequence's end, or bad: past the pool, which reads as zeros.
    auto look_up = [&](Tile& t) {
      if (++key >= g.k1) {
        if (!__all_sync(0xffffffffu, segment(++seg, g))) return false;
        if (lane == 0) mbar_arrive(&g_empty[seg % NG]);
        key = g.k0;
      }
      const int64_t at = (int64_t)key * KT + (piece << args.box_log2);
      t.h = g.h;
      t.place = (int)(at & ((1 << p.page_log2) - 1));
      t.page = p.n_pages;
      t.bad = false;
      if (at < (int64_t)g.L + g.n) {
        const int id = p.table[g.b * p.ld_table + (at >> p.page_log2)];
        t.bad = id < 0 || id >= p.n_pages;
        if (!t.bad) t.page = id;
      }
      return true;
    };
    Tile before, now, next;
    bool alive = look_up(next);
    // K0, then K and V of the tile before in turn, then the last V
#pragma unroll 1
    for (int i = 0; i < 2 * total && alive; ++i) {
      const int it = (i + 1) / 2;
      const bool is_k = i == 0 || (i & 1 && it < total);
      Tile t = before;
      if (is_k) {
        t = next;
        if (__any_sync(0xffffffffu, t.bad) && lane == 0) bad_tile[it % kBadRing] = it + 1;
        before = it > 0 ? now : t;  // (its V is next; the first tile's comes after the second's K)
        now = t;
        if (it + 1 < total && !look_up(next)) break;
      } else if (i + 1 == 2 * total) {
        t = now;
      }
      if (!(alive = warp_wait_for(&empty[slot], phase, abort_flag, p.status, 101))) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kSlot);
      __syncwarp();
      if (mine)
        tma_load_4d(smem + C::kOffSlots + slot * C::kSlot + dst, is_k ? &args.tm_k : &args.tm_v, col * 64, args.heads_out ? t.place : t.h,
                    args.heads_out ? t.h : t.place, t.page, &full[slot], policy);
      __syncwarp();
      ++loads;
      if (++slot == NS) slot = 0, phase ^= 1;
    }
    // every load lands before the CTA ends, also when another role gave up
    volatile int drained = 0;
#pragma unroll 1
    for (int j = loads > NS ? loads - NS : 0; j < loads; ++j)
      warp_wait_for(&full[j % NS], (j / NS) & 1, &drained, p.status, 102);
  } else if (warp == 1 || warp == 2) {
    if (lane == 0) {
      const uint32_t slots = smem_u32(smem + C::kOffSlots);
      int slot = 0, phase = 0, buf = 0, turn = 0, it = 0;
      bool alive = true;
      auto advance = [&](int by) {
        if ((slot += by) >= NS) slot -= NS, phase ^= 1;
        if (++buf == NB) buf = 0, turn ^= 1;
      };
      Segment g;
      if (warp == 1) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kTreeRows, KT);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem));
#pragma unroll 1
        for (int seg = 0; alive && segment(seg, g); ++seg) {
          mbar_arrive(&g_empty[seg % NG]);
          alive = wait_for(q_full, seg & 1, abort_flag, p.status, 104);
#pragma unroll 1
          for (int key = g.k0; key < g.k1 && alive; ++key, ++it) {
            // the columns hold the weights of NB tiles before until their product is complete
            if ((it >= NB && !wait_for(&pv_done[buf], turn ^ 1, abort_flag, p.status, 111)) ||
                !wait_for(&full[slot], phase, abort_flag, p.status, 103)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t k_desc = smem_desc_sw128(slots + slot * C::kSlot);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_bf16(tmem + C::kColS + buf * KT, q_desc + ((c * (kTreeRows * 128) + kk * 32) >> 4),
                            k_desc + ((c * (KT * 128) + kk * 32) >> 4), idesc_s, (c | kk) != 0);
            tc_commit(&empty[slot]);
            tc_commit(&s_full[buf]);
            advance(it == 0 ? 1 : 2);  // K0 K1 V0 K2 V1 ...
          }
        }
      } else {
        constexpr uint32_t idesc_o = idesc_bf16_f32(kTreeRows, D) | (1u << 16);  // B (V) is MN-major
        slot = total > 1 ? 2 : 1;
#pragma unroll 1
        for (int seg = 0; alive && segment(seg, g); ++seg) {
          mbar_arrive(&g_empty[seg % NG]);
          // (the segment before: its outputs are read by the warps that write this one's weights)
#pragma unroll 1
          for (int key = g.k0; key < g.k1 && alive; ++key, ++it) {
            if (!wait_for(&full[slot], phase, abort_flag, p.status, 106) ||
                !wait_for(&p_full[buf], turn, abort_flag, p.status, 105)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t v_desc = smem_desc_mn(slots + slot * C::kSlot, KT * 128);
#pragma unroll 1
            for (int k2 = 0; k2 < KT / 32; ++k2)
#pragma unroll
              for (int in = 0; in < 4; ++in)  // 16 keys' first parts and second ones
                tc_mma_ts(tmem, tmem + C::kColS + buf * KT + k2 * 32 + (in & 1) * 16 + (in >> 1) * 8,
                          v_desc + (((2 * k2 + (in >> 1)) * 2048) >> 4), idesc_o, ((key - g.k0) | k2 | in) != 0);
            tc_commit(&empty[slot]);
            tc_commit(&pv_done[buf]);
            advance(it + 2 < total ? 2 : 1);  // the last V follows the one before it
          }
        }
      }
      volatile int drained = 0;
      tc_commit(drain);  // all MMAs complete before tensor memory is freed
      wait_for(drain, 0, &drained, p.status, 107);
    }
  } else {
    const int quarter = warp & 3, r = quarter * 32 + lane, tid = threadIdx.x - 128;  // r: this thread's row of the tile
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    bool alive = true;
    int buf = 0, turn = 0, last = 0, last_turn = 0, it = 0, seg = 0, tails = 0, n_parts = 0;  // of this tile and of the one before
    const uint32_t per_group = (65535 + G) / G;  // x / G = x per_group >> 16 for x < 4096
    // A segment's queries into the swizzled K-major operand, as zeros past the end up to whole warps
    // (which choose together when to rescale: what another call left there may not decide that;
    // warps without rows hold what was there). `ready`: they have landed.
    auto fetch_queries = [&](const Segment& g) {
      constexpr int kChunks = D / 8;
      const uint16_t* q = p.q + g.tok0 * p.ldq + (int64_t)g.h * G * D;
#pragma unroll 2
      for (int j = tid; j < (g.rows + 31) / 32 * 32 * kChunks; j += 128) {
        const int row = j / kChunks, c = j % kChunks;
        const bool in = row < g.rows;
        const int x = g.row0 + (in ? row : 0), i = (int)(x * per_group >> 16);
        cp_async_16(smem_u32(smem + (c / 8) * (kTreeRows * 128) + sw128_offset(row, c % 8)),
                    q + i * p.ldq + (x - i * G) * D + c * 8, in ? 16u : 0u);
      }
      cp_async_commit();
    };
    Segment next, g;
    // the segment after this one, if there is one (alive is false after a wait that ran out)
    auto look_ahead = [&](int i) {
      const bool more = __all_sync(0xffffffffu, segment(i, next));
      __syncwarp();
      if (more && lane == 0) mbar_arrive(&g_empty[i % NG]);
      if (!more && *abort_flag) alive = false;
      return more;
    };
    bool more = look_ahead(0), ready = false;
    if (more) fetch_queries(next);
#pragma unroll 1
    for (; more && alive; ++seg) {
      g = next;
      const bool mine = r < g.rows, warp_rows = quarter * 32 < g.rows;
      const int x = g.row0 + (mine ? r : 0), i_new = (int)(x * per_group >> 16);
      uint64_t bits = p.tree ? (uint64_t)p.tree[g.tok0 + i_new] : (2ull << i_new) - 1;
      if (g.n < 64) bits &= (1ull << g.n) - 1;
      if (!ready) {
        cp_async_wait<0>();
        fence_proxy_async_smem();
        warp_arrive(q_full);
      }
      Running now = {-INFINITY, 0.f, 0.f, p.scale_log2};
      bool poison = false;
#pragma unroll 1
      for (int key = g.k0; key < g.k1; ++key, ++it) {
        if (!(alive = warp_wait_for(&s_full[buf], turn, abort_flag, p.status, 108))) break;
        tc_fence_after();
        if (bad_tile[it % kBadRing] == it + 1) poison = true;
        const int64_t rel = (int64_t)key * KT - g.L;  // of the tile's first position to the first new token
        const bool tail = rel + KT > 0;
        if (warp_rows) {
          // Once over the scores in tensor memory, 64 keys at a time, with the reference at hand, their weights
          // over them. The sum of the weights shows where the reference has to move. (128 keys take 0.9 us; 32 at a
          // time 1.0, 16 1.4. Neither the exponentials nor the conversions set the pace: with products in their place
          // they take the same.)
          const uint32_t cols = tmem + lanes + C::kColS + buf * KT;
          if (tail) mask_scores<KT>(cols, rel, bits);
          bool moved = false;
#pragma unroll 1
          for (int c = 0; c < KT;) {
            uint32_t s[2][32], hi[2][16], lo[2][16];
            tmem_ld_32x32b_x32(cols + c, s[0]);
            tmem_ld_32x32b_x32(cols + c + 32, s[1]);
            const float2 sc = make_float2(now.scale, now.scale), nr = make_float2(-now.at, -now.at);
            tc_wait_ld();
            if (now.scale == 1.f) {  // (the same for the whole warp)
#pragma unroll
              for (int j = 0; j < 64; ++j) s[j >> 5][j & 31] = __float_as_uint(__fmul_rn(__uint_as_float(s[j >> 5][j & 31]), p.scale_log2));
            }
            float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[z][2 * j]), __uint_as_float(s[z][2 * j + 1])), sc, nr);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                sums[z] = __fadd2_rn(sums[z], e);
                split_bf16(e.x, e.y, hi[z][j], lo[z][j]);
              }
            const float sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
            if (__any_sync(0xffffffffu, !(sum <= kMostSum) || now.m == -INFINITY) && !moved) {
              if (key > g.k0 && !(alive = warp_wait_for(&pv_done[last], last_turn, abort_flag, p.status, 109))) break;
              now = move_reference<D>(cols, c, tmem + lanes, key > g.k0, p.scale_log2, now.m, now.l);
              moved = true;
              continue;
            }
            moved = false;
            now.l += sum;
            tmem_st_32x32b_x16(cols + c, hi[0]);
            tmem_st_32x32b_x16(cols + c + 16, lo[0]);
            tmem_st_32x32b_x16(cols + c + 32, hi[1]);
            tmem_st_32x32b_x16(cols + c + 48, lo[1]);
            c += 64;
          }
          if (!alive) break;
          tc_wait_st();
        }
        if (tail) {
          // V of this tile: what no row attends to as zeros, and elements of the new tokens that are not
          // finite (their rows' outputs have them added below)
          const int at = it + 1 < total ? 2 * it + 2 : 2 * it + 1;  // of the ring's loads
          if (!(alive = warp_wait_for(&full[at % NS], (at / NS) & 1, abort_flag, p.status, 113))) break;
          uint8_t* v = smem + C::kOffSlots + (at % NS) * C::kSlot;
          const int first = (int)max((int64_t)0, -rel), none = (int)min((int64_t)KT, g.n - rel);
          bool odd = false;
#pragma unroll 4
          for (int j = first * (D / 8) + tid; j < KT * (D / 8); j += 128) {
            const int row = j / (D / 8), c = j % (D / 8);
            uint4* w = reinterpret_cast<uint4*>(v + (c / 8) * (KT * 128) + sw128_offset(row, c % 8));
            uint4 e = make_uint4(0, 0, 0, 0);
            if (row < none) {
              e = *w;
              if (!(not_finite2(e.x) || not_finite2(e.y) || not_finite2(e.z) || not_finite2(e.w))) continue;
              odd = true;
              uint32_t* pair = &e.x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((pair[k] & 0x7F80u) == 0x7F80u) pair[k] &= 0xFFFF0000u;
                if ((pair[k] & 0x7F800000u) == 0x7F800000u) pair[k] &= 0xFFFFu;
              }
            }
            *w = e;
          }
          if (odd) *v_bad = seg + 1;
          fence_proxy_async_smem();
          warp_arrive(v_ready);
          if (!(alive = warp_wait_for(v_ready, tails++ & 1, abort_flag, p.status, 114))) break;  // (also: v_bad is known)
        }
        tc_fence_before();
        warp_arrive(&p_full[buf]);
        last = buf, last_turn = turn;
        if (++buf == NB) buf = 0, turn ^= 1;
      }
      if (!alive) break;
      // The next segment's queries: the products that read these are complete (their scores were), and
      // the next scores' run while this segment's outputs are read.
      more = look_ahead(seg + 1);
      if (more) fetch_queries(next);
      // the segment's outputs: every product is complete with the last one
      if (!(alive = alive && warp_wait_for(&pv_done[last], last_turn, abort_flag, p.status, 110))) break;
      tc_fence_after();
      // (read before the arrival: once all warps have arrived, the next segment's scores run, and a warp that is ahead may
      // set it for that one)
      const bool odd_values = *v_bad == seg + 1;
      if (more) {
        cp_async_wait<0>();
        fence_proxy_async_smem();
        warp_arrive(q_full);
        ready = true;
      }
      float m = now.m, l = now.l;
      if (l != l && m == -INFINITY) m = 0.f;  // nothing but NaN: not a state without positions
      if (poison) m = 0.f, l = __int_as_float(0x7fc00000);  // a bad page: NaN
      int part = 0;
      if (!g.whole) {
        part = min(n_parts++, kTreeParts - 1);  // (never more: a chunk has 3/4 of a run at least)
        if (tid == 0) parts[part] = TreePart{g.item, g.tok0, what_of(g)};
      }
      const int64_t state = ((int64_t)blockIdx.x * kTreeParts + part) * p.rows;  // of the tile's first row
      if (mine && !g.whole) p.part_ml[state + r] = make_float2(m, l);
      if (warp_rows && !poison && odd_values) add_not_finite<D, KT>(p, g, tmem + lanes, bits, mine);
      // A quad of lanes holds 8 columns of a row at a time: stores are whole sectors of 8 rows. (A row a
      // lane: 16 bytes of each of 32 rows, 5 us for 128 rows of 256.)
      // nothing attended to: zeros (a part's are, but for infinities, which the merge takes out)
      const float inv = l != l ? l : !g.whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      const int q = lane & 3;
      bool looked = poison || g.L <= g.k0 * (int64_t)KT;  // for infinite cached values (there may be none)
#pragma unroll 1
      for (int half = 0; half < 32 && quarter * 32 + half < g.rows;) {
        float f[2];
        float2 none[2];  // f, or NaN once outputs are not finite: 0 times those is NaN
        uint8_t* dst[2];  // of the two rows that this lane has parts of; null past the end
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int in = half + 8 * k + (lane >> 2), row = quarter * 32 + in;
          f[k] = __shfl_sync(0xffffffffu, inv, in);
          none[k] = make_float2(f[k], f[k]);
          const int y = g.row0 + row, i = (int)(y * per_group >> 16);
          dst[k] = row >= g.rows ? nullptr
                   : g.whole ? reinterpret_cast<uint8_t*>(p.out + ((int64_t)(g.tok0 + i) * p.Hq + g.h * G + y - i * G) * D) + (8 * (q & 1) + 2 * (q & 2)) * 2
                             : reinterpret_cast<uint8_t*>(p.part_o + (state + row) * D) + 2 * q * 4;
        }
        const uint32_t from = tmem + ((uint32_t)(quarter * 32 + half) << 16);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[16];
          tmem_ld_16x256b_x4(from + c, o);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            none[j & 1] = __ffma2_rn(make_float2(__uint_as_float(o[2 * j]), __uint_as_float(o[2 * j + 1])), make_float2(0.f, 0.f), none[j & 1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float2 v[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              v[b] = make_float2(__uint_as_float(o[4 * b + 2 * k]), __uint_as_float(o[4 * b + 2 * k + 1]));
              v[b] = f[k] == 0.f ? make_float2(0.f, 0.f) : __fmul2_rn(v[b], make_float2(f[k], f[k]));
            }
            if (g.whole) {  // lanes exchange with their neighbours: 8 bytes of one of two blocks
#pragma unroll
              for (int b = 0; b < 4; b += 2) {
                const uint32_t w0 = pack_bf16(v[b].x, v[b].y), w1 = pack_bf16(v[b + 1].x, v[b + 1].y);
                const uint32_t x = __shfl_xor_sync(0xffffffffu, q & 1 ? w0 : w1, 1);
                if (dst[k]) *reinterpret_cast<uint2*>(dst[k] + (c + 8 * b) * 2) = q & 1 ? make_uint2(x, w1) : make_uint2(w0, x);
              }
            } else if (dst[k]) {
#pragma unroll
              for (int b = 0; b < 4; ++b) *reinterpret_cast<float2*>(dst[k] + (c + 8 * b) * 4) = v[b];
            }
          }
        }
        bool odd = false;  // (rows of NaN need no looking for)
#pragma unroll
        for (int k = 0; k < 2; ++k) odd |= f[k] == f[k] && !(none[k].x == f[k] && none[k].y == f[k]);
        if (!looked && __any_sync(0xffffffffu, odd)) {
          looked = true;
          show_not_finite<D, KT>(p, g, tmem + lanes);
          if (odd_values) add_not_finite<D, KT>(p, g, tmem + lanes, bits, mine);
          continue;  // these rows once more
        }
        half += 16;
      }
      tc_fence_before();
    }
    cp_async_wait<0>();  // (after a wait that ran out: queries on their way)
    if (!alive)
      give_up<KT>(p, found, first_seq, seg, n_parts, tid);
    else if (tid < kTreeParts && tid >= n_parts)
      parts[tid].item = -1;
  }
  __syncwarp();  // the single-lane roles join their warps
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Merges items' parts. Every block reads all notes and counts the rows that need it; it takes a row
// at a time, a warp every eighth part, where they are few, else eight rows, a warp each.
// (Grids over all rows would mostly find nothing to do: 60 sequences of 59 tokens, 48000
// rows in 480 items that no run cuts, 206 us instead of 33.)
constexpr int kMergeWarps = 8;
MOE_DEVINL float not_finite(float x) { return fabsf(x) < INFINITY ? 0.f : x; }
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeParams p) {
  constexpr int kC = D < 128 ? 1 : D / 128;  // float4 a lane (D = 64: half the lanes)
  constexpr int kAll = kTreeMaxSms * kTreeParts, kThreads = 32 * kMergeWarps, kPer = (kAll + kThreads - 1) / kThreads;
  __shared__ int list[kAll];
  __shared__ float weight[kMergeWarps][kAll];
  __shared__ float4 sums[kMergeWarps][D / 4];
  __shared__ int counts[kMergeWarps];
  __shared__ TreePart chosen;
  __shared__ int chosen_row;  // of the item
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, all = p.ctas * kTreeParts;
  // this thread's notes, and the rows of all first parts
  TreePart mine[kPer];
  int rows_of[kPer], rows = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    mine[k].item = -1;
    if (tid * kPer + k < all) mine[k] = p.parts[tid * kPer + k];
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) rows += rows_of[k] = mine[k].item >= 0 && (mine[k].what & 1) ? (mine[k].what >> 4 & 255) + 1 : 0;
  auto ordered = [&](int x, int& before) {  // the sum over the block, and that of the threads before
    int upto = x;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    if (lane == 31) counts[warp] = upto;
    __syncthreads();
    int total = 0;
    before = upto - x;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) before += counts[w];
      total += counts[w];
    }
    return total;
  };
  int before;
  const int n_rows = ordered(rows, before);
  const bool alone = n_rows <= (int)gridDim.x;  // a row a block
  const int per = alone ? 1 : kMergeWarps;
  int units_before = before, units = rows, n_units = n_rows;
  if (!alone) {
    __syncthreads();
    units = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) units += (rows_of[k] + per - 1) / per;
    n_units = ordered(units, units_before);
  }
  const int G = p.Hq / p.Hkv;
  for (int unit = blockIdx.x; unit < n_units; unit += gridDim.x) {
    __syncthreads();  // (the unit before is done with what is shared)
    if (units_before <= unit && unit < units_before + units) {
      int u = units_before;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int n = (rows_of[k] + per - 1) / per;
        if (u <= unit && unit < u + n) chosen = mine[k], chosen_row = (unit - u) * per;
        u += n;
      }
    }
    __syncthreads();
    const TreePart first = chosen;
    const int r = chosen_row + (alone ? 0 : warp);
    // the item's parts, in the order of their places
    int is = 0, at;
#pragma unroll
    for (int k = 0; k < kPer; ++k) is += mine[k].item == first.item;
    const int n = ordered(is, at);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (mine[k].item == first.item) list[at++] = tid * kPer + k;
    __syncthreads();
    if (r > (first.what >> 4 & 255)) continue;
    // every warp: the weights of all parts (as many as 32 at once)
    float M = -INFINITY, mass = 0.f;
    float2 ml = make_float2(-INFINITY, 0.f);
    for (int i = lane; i < n; i += 32) {
      const float2 x = p.part_ml[(int64_t)list[i] * p.rows + r];
      M = fmaxf(M, x.x);
      if (i < 32) ml = x;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int i = lane; i < n; i += 32) {
      const float2 x = i < 32 ? ml : p.part_ml[(int64_t)list[i] * p.rows + r];
      const float f = x.x == -INFINITY ? 0.f : ex2(x.x - M);
      weight[warp][i] = f;
      mass = fmaf(f, x.y, mass);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, off);
    __syncwarp();
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool in = lane * 4 < D;
    const float* o = p.part_o + (int64_t)r * D + (in ? lane * 4 : 0);
    const int step = alone ? kMergeWarps : 1;
    for (int i0 = alone ? warp : 0; i0 < n; i0 += 4 * step) {
      float4 v[4][kC];
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (a part in which the row attends to nothing has zeros, or infinities)
        const int k = i0 + i * step;
        f[i] = 0.f;
        if (k >= n) continue;
        f[i] = weight[warp][k];
        const float* from = o + (int64_t)list[k] * p.rows * D;
#pragma unroll
        for (int c = 0; c < kC; ++c) v[i][c] = *reinterpret_cast<const float4*>(from + c * 128);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i0 + i * step >= n) continue;
        if (f[i] == 0.f) {  // what is infinite or NaN has no weight
#pragma unroll
          for (int c = 0; c < kC; ++c)
            v[i][c] = make_float4(not_finite(v[i][c].x), not_finite(v[i][c].y), not_finite(v[i][c].z), not_finite(v[i][c].w));
          f[i] = 1.f;
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          acc[c].x = fmaf(f[i], v[i][c].x, acc[c].x);
          acc[c].y = fmaf(f[i], v[i][c].y, acc[c].y);
          acc[c].z = fmaf(f[i], v[i][c].z, acc[c].z);
          acc[c].w = fmaf(f[i], v[i][c].w, acc[c].w);
        }
      }
    }
    if (alone) {
#pragma unroll
      for (int c = 0; c < kC; ++c)
        if (in) sums[warp][lane + 32 * c] = acc[c];
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const float4 v = sums[w][in ? lane + 32 * c : 0];
          acc[c].x += v.x;
          acc[c].y += v.y;
          acc[c].z += v.z;
          acc[c].w += v.w;
        }
    }
    if (!in) continue;
    const float inv = 1.f / mass;
    const int x = (first.what >> 12 & 15) * kTreeRows + r;
    uint16_t* out = p.out + ((int64_t)(first.tok0 + x / G) * p.Hq + (first.what >> 16) * G + x % G) * D + lane * 4;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      *reinterpret_cast<uint2*>(out + c * 128) =
          mass == 0.f ? make_uint2(0, 0) :  // nothing attended to
          make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv), pack_bf16(acc[c].z * inv, acc[c].w * inv));
  }
}

bool encode_pages(CUtensorMap* tm, const uint16_t* base, const TreeParams& p, int box, bool heads_out) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  // axes in the order of their strides; of the heads always one a box
  const cuuint64_t page = 1ull << p.page_log2, hs = (cuuint64_t)p.head_stride * 2, ps = (cuuint64_t)p.position_stride * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)p.d, heads_out ? page : (cuuint64_t)p.Hkv, heads_out ? (cuuint64_t)p.Hkv : page,
                              (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {heads_out ? ps : hs, heads_out ? hs : ps, (cuuint64_t)p.page_stride * 2};
  const cuuint32_t boxes[4] = {64, heads_out ? (cuuint32_t)box : 1u, heads_out ? 1u : (cuuint32_t)box, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t tree_launch_t(const TreeParams& p, cudaStream_t s) {
  using C = TrCfg<D>;
  TrArgs args;
  memset(&args, 0, sizeof args);
  args.p = p;
  args.box_log2 = std::min(p.page_log2, C::KT == 64 ? 6 : 7);
  args.heads_out = p.head_stride > p.position_stride;
  if (!encode_pages(&args.tm_k, p.k_pages, p, 1 << args.box_log2, args.heads_out) ||
      !encode_pages(&args.tm_v, p.v_pages, p, 1 << args.box_log2, args.heads_out))
    return cudaErrorInvalidValue;
  static SharedMemoryOptIn opt_in;
  if (const cudaError_t err = opt_in(tree_kernel<D>, C::kSmem); err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kTrThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (const cudaError_t err = cudaLaunchKernelEx(&cfg, tree_kernel<D>, args); err != cudaSuccess) return err;
  cfg.gridDim = dim3((unsigned)std::min(4 * p.ctas, p.ctas * ((p.rows + kMergeWarps - 1) / kMergeWarps)));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, p);
}

}  // namespace

cudaError_t tree_launch(const TreeParams& p, cudaStream_t s) {
  if (p.d == 256) return tree_launch_t<256>(p, s);
  if (p.d == 128) return tree_launch_t<128>(p, s);
  return tree_launch_t<64>(p, s);
}

}  // namespace moe
