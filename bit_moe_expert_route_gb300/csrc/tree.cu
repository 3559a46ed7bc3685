// Attention of sequences' new tokens (one, or a tree of drafted ones) over a paged cache.
//
//   o_{t,h} = sum_j softmax_j(scale q_{t,h} . k_j) v_j  over the positions before the
//   sequence's new tokens, and those of its new tokens that bits of a mask name.
//
// The n G query rows of a sequence that read one KV head (G query heads of each of n
// tokens) form one matrix, in tiles of 128 rows: each K and V tile is read once for
// all of them. Bound by HBM up to 128 rows (the MMAs of a tile of 64 KB take 1824 cycles
// at head size 256, 1536 at 128, against about 3000 that an SM's share of HBM needs for it),
// by the MMAs with more.
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
// segment's tiles land while this one ends.
//
// What rows do not attend to: scores are set to -infinity by the row's mask, whatever they
// were. In V, a weight of 0 would still make NaN of an infinity or a NaN. Rows past the
// sequence's end (a page's rest) are set to 0 in shared memory; so are infinite and NaN elements of the
// new tokens' V, and rows that do attend to such a token have the element added at the end.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTrThreads = 256;  // warp 0 TMA, warps 1 and 2 MMA, warps 4-7 softmax
constexpr float kLazyLog2 = 8.f;
constexpr int kBadRing = 16;     // tiles whose pages are known to be bad or not: more than the ring holds

template <int D>
struct TrCfg {
  static constexpr int KT = D == 256 ? 64 : 128;    // keys a tile
  static constexpr int kSlot = KT * D * 2;          // K or V of a tile
  static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 6 : 8;
  static constexpr int kQ = kTreeRows * D * 2;
  static constexpr int kBufs = 3;                   // tiles between their scores and their outputs
  static constexpr int kOffSlots = kQ;
  static constexpr int kOffBar = kOffSlots + kSlots * kSlot;
  static constexpr int kBars = 2 * kSlots + 2 + 3 * kBufs + 1;
  static constexpr int kSmem = kOffBar + 8 * kBars + 512 + 1024;
  static constexpr int kColS = D;                   // tensor memory: O, then the score buffers
  static_assert(kColS + kBufs * KT <= 512, "tensor memory exceeded");
  static_assert(kSmem <= 232448, "shared memory exceeded");
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

// A CTA's run of tiles, segment by segment. A sequence's tiles in order: KV head, chunk of
// keys, row tile, key.
template <int KT>
struct Walk {
  int64_t cur, end, base, count;  // of all tiles: the next, the run's end, this sequence's first; how many it has
  int b, run;                     // (run: tiles of the longest one)
  Sequence s;
  int kt, rt, chunks;
  // the segment: keys k0 .. k1 - 1 (in tiles) of row tile row0 / 128
  int h, row0, rows, k0, k1;
  MOE_DEVINL void start(const TreeParams& p, const int64_t* found) {
    cur = found[0], end = found[1], b = (int)found[2], base = found[3], run = (int)found[4];
    if (cur < end) load(p);
  }
  MOE_DEVINL void load(const TreeParams& p) {
    s = sequence_of(p, b);
    kt = key_tiles<KT>(s), rt = row_tiles(p, s), count = tiles_of<KT>(p, s);
    // chunks of 3/4 to 3/2 of a run
    chunks = rt > 1 ? max(1, (int)((2 * (int64_t)kt + run) / (2 * (int64_t)run))) : 1;
  }
  MOE_DEVINL int bound(int chunk) const { return chunks == 1 ? (chunk ? kt : 0) : (int)((int64_t)kt * chunk / chunks); }
  MOE_DEVINL bool next(const TreeParams& p) {
    if (cur >= end) return false;
    while (cur >= base + count) {
      if (b + 1 >= p.B) return cur = end, false;  // (only if the lengths changed under the kernel)
      base += count;
      ++b;
      load(p);
    }
    const int64_t head = (int64_t)kt * rt, off = cur - base;
    h = (int)(off / head);
    const int64_t in = off - h * head;
    int chunk = 0;
    if (chunks > 1) {
      chunk = (int)(in / rt * chunks / kt);
      while (chunk + 1 < chunks && (int64_t)bound(chunk + 1) * rt <= in) ++chunk;
      while (chunk > 0 && (int64_t)bound(chunk) * rt > in) --chunk;
    }
    const int from = bound(chunk), to = bound(chunk + 1);
    const int64_t at = in - (int64_t)from * rt;
    const int row = (int)(at / (to - from));
    k0 = from + (int)(at - (int64_t)row * (to - from));
    k1 = (int)min((int64_t)to, k0 + (end - cur));
    cur += k1 - k0;
    row0 = row * kTreeRows;
    rows = min(kTreeRows, s.n * (p.Hq / p.Hkv) - row0);
    return true;
  }
  MOE_DEVINL bool whole() const { return k0 == 0 && k1 == kt; }
  // The segment's item, as no other's.
  MOE_DEVINL int64_t item() const { return base + ((int64_t)h * rt + row0 / kTreeRows) * kt; }
};

// Which of the 32 positions from the rel-th new token on (rel < 0: cached ones before) a
// row with the mask `bits` attends to.
MOE_DEVINL uint32_t attended(int64_t rel, uint64_t bits) {
  if (rel <= -32) return 0xFFFFFFFFu;
  if (rel < 0) return (uint32_t)((bits << -rel) | ((1ull << -rel) - 1));
  return rel < 64 ? (uint32_t)(bits >> rel) : 0u;
}

MOE_DEVINL bool not_finite2(uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; }

template <int D>
__global__ void __launch_bounds__(kTrThreads, 1) tree_kernel(const __grid_constant__ TrArgs args) {
  using C = TrCfg<D>;
  constexpr int KT = C::KT, NS = C::kSlots, NB = C::kBufs;
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
  int64_t* found = reinterpret_cast<int64_t*>(drain + 1);           // the run: first tile, end, sequence, its first tile, the longest's tiles
  int64_t* sums = found + 5;                                        // [8] a warp's tiles
  int* bad_tile = reinterpret_cast<int*>(sums + 8);                 // [kBadRing] 1 + tile of the run with a bad page
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bad_tile + kBadRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* v_bad = abort_flag + 1;  // 1 + segment whose new V holds infinities or NaN
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(v_ready, 4);
    for (int i = 0; i < NB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 2);
    for (int i = 0; i < kBadRing; ++i) bad_tile[i] = 0;
    found[0] = found[1] = 0;
    *abort_flag = 0;
    *v_bad = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tm_k);
    tma_prefetch_desc(&args.tm_v);
  }
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
    int64_t total = 0, first = 0, mine = 0;  // of all; before this thread's last sequence; that one's
    int bad = 0;
    auto add = [&](int b0) {  // of the sequences b0 .. b0 + 255
      const int b = b0 + threadIdx.x;
      mine = 0;
      if (b < p.B) {
        const Sequence s = sequence_of(p, b);
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
      first = total + upto - mine;
#pragma unroll
      for (int w = 0; w < kTrThreads / 32; ++w) {
        if (w < warp) first += sums[w];
        total += sums[w];
      }
      if (p.B > kTrThreads) __syncthreads();
    };
    for (int b0 = 0; b0 < p.B; b0 += kTrThreads) add(b0);
    const int64_t all = total, from = run_begin(all, blockIdx.x, p.ctas), to = run_begin(all, blockIdx.x + 1, p.ctas);
    auto note = [&](int b) {
      if (first <= from && from < first + mine) {
        found[0] = from, found[1] = to, found[2] = b, found[3] = first;
        found[4] = (all + p.ctas - 1) / p.ctas;
      }
    };
    if (p.B <= kTrThreads) {
      if (from < to) note(threadIdx.x);
    } else if (from < to) {
      total = 0;
      for (int b0 = 0; b0 < p.B; b0 += kTrThreads) {
        add(b0);
        note(b0 + threadIdx.x);
      }
    }
    if (__syncthreads_or(bad)) {  // sequences that cannot be right: NaN, by all CTAs
      for (int b = 0; b < p.B; ++b) {
        const Sequence s = sequence_of(p, b);
        if (!s.bad) continue;
        const int64_t words = (int64_t)s.n * p.Hq * (D / 8);
        uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)s.tok0 * p.Hq * D);
        for (int64_t i = (int64_t)blockIdx.x * kTrThreads + threadIdx.x; i < words; i += (int64_t)p.ctas * kTrThreads)
          out[i] = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
      }
    }
  }
  Walk<KT> walk;
  walk.start(p, found);
  const int total = (int)(found[1] - found[0]);  // tiles of the run
  TreePart* const parts = p.parts + (int64_t)blockIdx.x * kTreeParts;

  if (total == 0) {  // fewer tiles than CTAs
    if (threadIdx.x < kTreeParts) parts[threadIdx.x].item = -1;
  } else if (warp == 0) {
    fence_proxy_async_global();  // the pages are written by ordinary stores of earlier launches
    // keys that one CTA alone reads leave L2 first
    const uint64_t policy = p.rows < kTreeRows ? l2_policy_evict_first() : l2_policy_evict_normal();
    const int pieces_log2 = (KT == 64 ? 6 : 7) - args.box_log2, pieces = 1 << pieces_log2;
    // a lane's box of each tile: 64 columns, one page's (or the tile's) positions
    const int piece = lane & (pieces - 1), col = lane >> pieces_log2;
    const bool mine = col < D / 64;
    const uint32_t dst = col * (KT * 128) + ((piece << args.box_log2) * 128);
    int slot = 0, phase = 1, loads = 0, h = 0, place = 0, page = 0;
    int kh = 0, kplace = 0, kpage = 0;
    auto load = [&](const CUtensorMap* tm, int head, int at, int id) {
      if (!warp_wait(&empty[slot], phase, abort_flag, p.status, 101)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kSlot);
      __syncwarp();
      if (mine)
        tma_load_4d(smem + C::kOffSlots + slot * C::kSlot + dst, tm, col * 64, args.heads_out ? at : head,
                    args.heads_out ? head : at, id, &full[slot], policy);
      __syncwarp();
      ++loads;
      if (++slot == NS) slot = 0, phase ^= 1;
      return true;
    };
    // a tile's page, looked up a tile ahead; past the sequence's end, or bad: past the pool, which reads as zeros
    int key = 0, end = 0;
    bool bad = false;
    auto look_up = [&]() {
      const int64_t at = (int64_t)key * KT + (piece << args.box_log2);
      h = walk.h;
      place = (int)(at & ((1 << p.page_log2) - 1));
      page = p.n_pages;
      bad = false;
      if (at < (int64_t)walk.s.L + walk.s.n) {
        const int id = p.table[walk.b * p.ld_table + (at >> p.page_log2)];
        bad = id < 0 || id >= p.n_pages;
        if (!bad) page = id;
      }
    };
    auto advance = [&]() {
      if (++key >= end) {
        if (!walk.next(p)) return false;
        key = walk.k0, end = walk.k1;
      }
      return true;
    };
    bool alive = advance();
    if (alive) look_up();
    for (int it = 0; it < total && alive; ++it) {
      const int ph = kh, pplace = kplace, ppage = kpage;
      kh = h, kplace = place, kpage = page;
      if (__any_sync(0xffffffffu, bad) && lane == 0) bad_tile[it % kBadRing] = it + 1;
      if (it + 1 < total) {
        if (advance()) look_up(); else alive = false;
      }
      alive = alive && load(&args.tm_k, kh, kplace, kpage);
      if (it > 0) alive = alive && load(&args.tm_v, ph, pplace, ppage);
    }
    if (alive) load(&args.tm_v, kh, kplace, kpage);
    // every load lands before the CTA ends, also when another role gave up
    volatile int drained = 0;
    for (int j = loads > NS ? loads - NS : 0; j < loads; ++j)
      warp_wait(&full[j % NS], (j / NS) & 1, &drained, p.status, 102);
  } else if (warp == 1 || warp == 2) {
    if (lane == 0) {
      const uint32_t slots = smem_u32(smem + C::kOffSlots);
      int slot = 0, phase = 0, buf = 0, turn = 0, it = 0, seg = 0;
      bool alive = true;
      auto advance = [&](int by) {
        if ((slot += by) >= NS) slot -= NS, phase ^= 1;
        if (++buf == NB) buf = 0, turn ^= 1;
      };
      if (warp == 1) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kTreeRows, KT);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem));
        for (; alive && walk.next(p); ++seg) {
          alive = mbar_wait(q_full, seg & 1, abort_flag, p.status, 104);
          for (int key = walk.k0; key < walk.k1 && alive; ++key, ++it) {
            // the columns hold the weights of NB tiles before until their product is complete
            if ((it >= NB && !mbar_wait(&pv_done[buf], turn ^ 1, abort_flag, p.status, 111)) ||
                !mbar_wait(&full[slot], phase, abort_flag, p.status, 103)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t k_desc = smem_desc_sw128(slots + slot * C::kSlot);
#pragma unroll
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
        for (; alive && walk.next(p); ++seg) {
          // (the segment before: its outputs are read by the warps that write this one's weights)
          for (int key = walk.k0; key < walk.k1 && alive; ++key, ++it) {
            if (!mbar_wait(&full[slot], phase, abort_flag, p.status, 106) ||
                !mbar_wait(&p_full[buf], turn, abort_flag, p.status, 105)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t v_desc = smem_desc_mn(slots + slot * C::kSlot, KT * 128);
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
              for (int part = 0; part < 2; ++part)
                tc_mma_ts(tmem, tmem + C::kColS + buf * KT + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8, v_desc + ((kk * 2048) >> 4), idesc_o,
                          ((key - walk.k0) | kk | part) != 0);
            tc_commit(&empty[slot]);
            tc_commit(&pv_done[buf]);
            advance(it + 2 < total ? 2 : 1);  // the last V follows the one before it
          }
        }
      }
      volatile int drained = 0;
      tc_commit(drain);  // all MMAs complete before tensor memory is freed
      mbar_wait(drain, 0, &drained, p.status, 107);
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, r = quarter * 32 + lane, tid = threadIdx.x - 128;  // r: this thread's row of the tile
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    bool alive = true;
    int buf = 0, turn = 0, last = 0, last_turn = 0, it = 0, seg = 0, tails = 0, n_parts = 0;  // of this tile and of the one before
    const uint32_t per_group = (65535 + G) / G;  // x / G = x per_group >> 16 for x < 4096
    // The queries of the segment at hand into the swizzled K-major operand, as zeros past the end up to
    // whole warps (which choose together when to rescale: what another call left there may not decide
    // that; warps without rows hold what was there).
    auto fetch_queries = [&]() {
      constexpr int kChunks = D / 8;
      const uint16_t* q = p.q + walk.s.tok0 * p.ldq + (int64_t)walk.h * G * D;
#pragma unroll 4
      for (int j = tid; j < (walk.rows + 31) / 32 * 32 * kChunks; j += 128) {
        const int row = j / kChunks, c = j % kChunks;
        const bool in = row < walk.rows;
        const int x = walk.row0 + (in ? row : 0), i = (int)(x * per_group >> 16);
        cp_async_16(smem_u32(smem + (c / 8) * (kTreeRows * 128) + sw128_offset(row, c % 8)),
                    q + i * p.ldq + (x - i * G) * D + c * 8, in ? 16u : 0u);
      }
      cp_async_commit();
    };
    auto queries_ready = [&]() {
      cp_async_wait<0>();
      fence_proxy_async_smem();
      warp_arrive(q_full);
    };
    bool more = walk.next(p);
    if (more) {
      fetch_queries();
      queries_ready();
    }
    for (; more; ++seg) {
      const Walk<KT> now = walk;
      const int rows = now.rows, L = now.s.L, n = now.s.n;
      const bool mine = r < rows, warp_rows = quarter * 32 < rows;
      const int x = now.row0 + (mine ? r : 0), i_new = (int)(x * per_group >> 16);
      const int token = now.s.tok0 + i_new, head = now.h * G + x - i_new * G;
      uint64_t bits = p.tree ? (uint64_t)p.tree[token] : (2ull << i_new) - 1;
      if (n < 64) bits &= (1ull << n) - 1;
      float m = -INFINITY, l = 0.f;
      bool poison = false;
      for (int key = now.k0; key < now.k1 && alive; ++key, ++it) {
        if (!(alive = warp_wait(&s_full[buf], turn, abort_flag, p.status, 108))) break;
        tc_fence_after();
        if (bad_tile[it % kBadRing] == it + 1) poison = true;
        const int64_t rel = (int64_t)key * KT - L;  // of the tile's first position to the first new token
        const bool tail = rel + KT > 0;
        if (warp_rows) {
          // Twice over the scores in tensor memory, in pieces: the largest, then the weights, over
          // the scores of their piece. (All of a tile's scores in registers are one long piece of code,
          // which a call of few tiles spends its time fetching.)
          const uint32_t cols = tmem + lanes + C::kColS + buf * KT;
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < KT; c += 32) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(cols + c, s);
            tc_wait_ld();
            if (tail) {
              const uint32_t in = attended(rel + c, bits);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(in >> j & 1)) s[j] = 0xFF800000u;
              tmem_st_32x32b_x32(cols + c, s);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]));
          }
          if (tail) tc_wait_st();
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
          if (__any_sync(0xffffffffu, top > m + kLazyLog2)) {
            const float nm = fmaxf(m, top), f = nm == -INFINITY ? 1.f : ex2(m - nm);  // (m -infinity: 0)
            l *= f;
            m = nm;
            if (key > now.k0) {
              // O is whole once the product before is complete
              if (!(alive = warp_wait(&pv_done[last], last_turn, abort_flag, p.status, 109))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld_32x32b_x16(tmem + lanes + c, o);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st_32x32b_x16(tmem + lanes + c, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          // What the fused product leaves of a large reference's rounding would pass 2^-8: then scale apart,
          // rounded as the reference was.
          const bool apart = __any_sync(0xffffffffu, fabsf(ref) >= 65536.f);
          const float sc1 = apart ? 1.f : p.scale_log2;
          const float2 sc = make_float2(sc1, sc1), nr = make_float2(-ref, -ref);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < KT; c += 32) {
            uint32_t s[32], hi[16], lo[16];
            tmem_ld_32x32b_x32(cols + c, s);
            tc_wait_ld();
            if (apart) {
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__fmul_rn(__uint_as_float(s[j]), p.scale_log2));
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), sc, nr);
              const float2 e = make_float2(ex2(y.x), ex2(y.y));
              sum = __fadd2_rn(sum, e);
              split_bf16(e.x, e.y, hi[j], lo[j]);
            }
            tmem_st_32x32b_x16(cols + c, hi);
            tmem_st_32x32b_x16(cols + c + 16, lo);
          }
          l += sum.x + sum.y;
          tc_wait_st();
        }
        if (tail) {
          // V of this tile: what no row attends to as zeros, and elements of the new tokens that are not
          // finite (their rows' outputs have them added below)
          const int at = it + 1 < total ? 2 * it + 2 : 2 * it + 1;  // of the ring's loads
          if (!(alive = warp_wait(&full[at % NS], (at / NS) & 1, abort_flag, p.status, 113))) break;
          uint8_t* v = smem + C::kOffSlots + (at % NS) * C::kSlot;
          const int first = (int)max((int64_t)0, -rel), none = (int)min((int64_t)KT, n - rel);
          bool odd = false;
          for (int j = first * (D / 8) + tid; j < KT * (D / 8); j += 128) {
            const int row = j / (D / 8), c = j % (D / 8);
            uint4* w = reinterpret_cast<uint4*>(v + (c / 8) * (KT * 128) + sw128_offset(row, c % 8));
            uint4 x = make_uint4(0, 0, 0, 0);
            if (row < none) {
              x = *w;
              if (!(not_finite2(x.x) || not_finite2(x.y) || not_finite2(x.z) || not_finite2(x.w))) continue;
              odd = true;
              uint32_t* e = &x.x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((e[k] & 0x7F80u) == 0x7F80u) e[k] &= 0xFFFF0000u;
                if ((e[k] & 0x7F800000u) == 0x7F800000u) e[k] &= 0xFFFFu;
              }
            }
            *w = x;
          }
          if (odd) *v_bad = seg + 1;
          fence_proxy_async_smem();
          warp_arrive(v_ready);
          if (!(alive = warp_wait(v_ready, tails++ & 1, abort_flag, p.status, 114))) break;  // (also: v_bad is known)
        }
        tc_fence_before();
        warp_arrive(&p_full[buf]);
        last = buf, last_turn = turn;
        if (++buf == NB) buf = 0, turn ^= 1;
      }
      // The next segment's queries: the products that read these are complete (their scores were), and
      // the next scores' run while this segment's outputs are read.
      more = walk.next(p);
      if (alive && more) fetch_queries();
      // the segment's outputs: every product is complete with the last one
      if (alive) alive = warp_wait(&pv_done[last], last_turn, abort_flag, p.status, 110);
      if (alive && more) queries_ready();
      const bool whole = now.whole();
      int part = 0;
      if (!whole) {
        part = min(n_parts++, kTreeParts - 1);  // (never more: a chunk has 3/4 of a run at least)
        if (tid == 0) parts[part] = TreePart{now.item(), now.s.tok0, now.h << 16 | now.row0 / kTreeRows << 12 | (rows - 1) << 4 | (now.k0 == 0)};
      }
      const int64_t state = ((int64_t)blockIdx.x * kTreeParts + part) * p.rows + r;
      if (l != l && m == -INFINITY) m = 0.f;  // nothing but NaN: not a state without positions
      if (!alive || poison) {  // after a wait that ran out, or a bad page: NaN
        m = 0.f;
        l = __int_as_float(0x7fc00000);
      }
      if (alive) tc_fence_after();
      if (mine && !whole) p.part_ml[state] = make_float2(m, l);
      if (warp_rows && (alive || whole)) {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // nothing attended to: zeros
        const bool odd = alive && *v_bad == seg + 1;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (alive) {
            tmem_ld_32x32b_x32(tmem + lanes + c, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0x7fc00000u;
          }
          if (l == 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          if (odd && mine && !poison) {
            const int64_t from = max((int64_t)now.k0 * KT, (int64_t)L), to = min((int64_t)now.k1 * KT, (int64_t)L + n);
#pragma unroll 1
            for (int64_t at = from; at < to; ++at) {
              if (!(bits >> (at - L) & 1)) continue;
              const int64_t id = p.table[now.b * p.ld_table + (at >> p.page_log2)];
              const uint16_t* v = p.v_pages + id * p.page_stride + (at & ((1 << p.page_log2) - 1)) * p.position_stride +
                                  now.h * p.head_stride + c;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float x = bf16_bits_to_f32(v[j]);
                if (!(fabsf(x) <= 3.4e38f)) o[j] = __float_as_uint(__uint_as_float(o[j]) + x);
              }
            }
          }
          if (!mine) {
          } else if (whole) {
            uint16_t* out = p.out + ((int64_t)token * p.Hq + head) * D + c;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16(__uint_as_float(o[8 * j + 2 * k]) * inv, __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
              *reinterpret_cast<uint4*>(out + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float* out = p.part_o + state * D + c;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(out + 4 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
          __syncwarp();  // (tcgen05.ld wants the warp undivided)
        }
      }
      tc_fence_before();
    }
    cp_async_wait<0>();  // (after a wait that ran out: queries on their way)
    if (tid == 0)
      for (int i = n_parts; i < kTreeParts; ++i) parts[i].item = -1;
  }
  __syncwarp();  // the single-lane roles join their warps
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Merges items' parts. Every block reads all notes; eight rows of an item at a time, a warp a
// row. (Grids over all rows would mostly find nothing to do: 60 sequences of 59 tokens, 48000
// rows in 480 items that no run cuts, 206 us instead of 33.)
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeParams p) {
  constexpr int kC = D < 128 ? 1 : D / 128;  // float4 a lane (D = 64: half the lanes)
  constexpr int kAll = kTreeMaxSms * kTreeParts, kThreads = 32 * kMergeWarps, kPer = (kAll + kThreads - 1) / kThreads;
  __shared__ int list[kAll];
  __shared__ float weight[kMergeWarps][kAll];
  __shared__ int counts[kMergeWarps];
  __shared__ TreePart chosen;
  __shared__ int chosen_unit;  // of the item
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, all = p.ctas * kTreeParts;
  // this thread's notes, and the units of all
  TreePart mine[kPer];
  int units = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    mine[k].item = -1;
    if (tid * kPer + k < all) mine[k] = p.parts[tid * kPer + k];
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (mine[k].item >= 0 && (mine[k].what & 1)) units += ((mine[k].what >> 4 & 255) + kMergeWarps) / kMergeWarps;
  int upto = units;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += v;
  }
  if (lane == 31) counts[warp] = upto;
  __syncthreads();
  int n_units = 0, before = upto - units;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (w < warp) before += counts[w];
    n_units += counts[w];
  }
  const int G = p.Hq / p.Hkv;
  for (int unit = blockIdx.x; unit < n_units; unit += gridDim.x) {
    __syncthreads();  // (the unit before is done with what is shared)
    if (before <= unit && unit < before + units) {
      int u = before;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (mine[k].item < 0 || !(mine[k].what & 1)) continue;
        const int n = ((mine[k].what >> 4 & 255) + kMergeWarps) / kMergeWarps;
        if (u <= unit && unit < u + n) {
          chosen = mine[k];
          chosen_unit = unit - u;
        }
        u += n;
      }
    }
    __syncthreads();
    const TreePart first = chosen;
    const int rows = (first.what >> 4 & 255) + 1, r = chosen_unit * kMergeWarps + warp;
    // the item's parts, in the order of their places
    int is = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) is += mine[k].item == first.item;
    int at = is;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, at, off);
      if (lane >= off) at += v;
    }
    if (lane == 31) counts[warp] = at;
    __syncthreads();
    int n = 0;
    at -= is;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      if (w < warp) at += counts[w];
      n += counts[w];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (mine[k].item == first.item) list[at++] = tid * kPer + k;
    __syncthreads();
    if (r >= rows) continue;
    float M = -INFINITY, sum = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float2 ml = p.part_ml[(int64_t)list[i] * p.rows + r];
      M = fmaxf(M, ml.x);
      weight[warp][i] = ml.x;
      sum = i == lane ? ml.y : sum;  // (the lane's first; others are read again)
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float mass = 0.f;
    for (int i = lane; i < n; i += 32) {
      const float x = weight[warp][i], f = x == -INFINITY ? 0.f : ex2(x - M);
      weight[warp][i] = f;
      mass = fmaf(f, i == lane ? sum : p.part_ml[(int64_t)list[i] * p.rows + r].y, mass);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, off);
    __syncwarp();
    float4 acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane * 4 < D) {
      const float* o = p.part_o + (int64_t)r * D + lane * 4;
      for (int i0 = 0; i0 < n; i0 += 8) {
        float4 v[8][kC];
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (a part in which the row attends to nothing has zeros)
#pragma unroll
          for (int c = 0; c < kC; ++c)
            v[i][c] = *reinterpret_cast<const float4*>(o + (int64_t)list[min(i0 + i, n - 1)] * p.rows * D + c * 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i0 + i >= n) break;
          const float f = weight[warp][i0 + i];
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            acc[c].x = fmaf(f, v[i][c].x, acc[c].x);
            acc[c].y = fmaf(f, v[i][c].y, acc[c].y);
            acc[c].z = fmaf(f, v[i][c].z, acc[c].z);
            acc[c].w = fmaf(f, v[i][c].w, acc[c].w);
          }
        }
      }
      const float inv = mass == 0.f ? 0.f : 1.f / mass;  // nothing attended to: zeros
      const int x = (first.what >> 12 & 15) * kTreeRows + r;
      uint16_t* out = p.out + ((int64_t)(first.tok0 + x / G) * p.Hq + (first.what >> 16) * G + x % G) * D + lane * 4;
#pragma unroll
      for (int c = 0; c < kC; ++c)
        *reinterpret_cast<uint2*>(out + c * 128) =
            make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv), pack_bf16(acc[c].z * inv, acc[c].w * inv));
    }
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
