// Decode attention for a batch whose sequences share a prefix.
//
//   o_{b,h} = sum_j softmax_j(scale q_{b,h} . k_j) v_j  over the shared prefix's
//   positions and then sequence b's own.
//
// The prefix's keys and values are the same for every sequence, so the queries
// of all sequences that read one KV head (B G rows, G query heads a KV head)
// form one matrix: each K and V tile is read once for all of them, and the
// products go to the tensor cores. Softmax over the two parts is joined from
// partial states (m, l, o): a block takes one KV head, a tile of rows and a
// slice of the prefix, or one sequence's own positions; a second kernel merges
// a row's partials.
//
// A block: 4 warps, WM of them over 16-row tiles and 4 / WM over the keys of
// each 64-key tile, so that a few rows still use every warp. K and V tiles
// come through a ring of cp.async slots; m16n8k16 products with fp32 sums. The
// weights enter the second product as two bf16 parts: one would carry its
// roundings (2^-8 of each weight) to the output, and these products wait for memory
// anyway. The running maximum moves only when a score passes it by 2^8, which
// fp32 and bf16 hold without loss, so the output is rarely rescaled. (With more
// than 32 rows a KV head the prefix goes to prefix_tc.cu; the sequences' own
// positions stay here. Little work takes one launch of clusters, below.)
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kPfThreads = 128;
constexpr int kTileKeys = 64;
constexpr float kLazyLog2 = 8.f;
// (Two blocks on each of the 152 SMs for which the rule was measured; whether a call
// needs a workspace has to follow from its sizes alone.)
constexpr int kJoinedBlocks = 304, kJoinedTiles = 4, kJoinedWork = 2048;
static_assert(kJoinedTiles * 8 * kTileKeys == kPrefixJoinedPositions, "eight blocks' tiles");
constexpr int kPrefixTcMin = 256;  // positions from which the tensor-memory kernel takes a prefix

MOE_DEVINL void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
MOE_DEVINL void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
MOE_DEVINL void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a tile of D bf16 a row: chunks
// XORed with the row, so that eight rows' chunks lie in different banks.
template <int D>
MOE_DEVINL uint32_t tile_off(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

template <int D>
struct PfCfg {
  // Three slots of one K or one V tile each, filled two ahead (K0 V0 K1 V1 ...):
  // at head size 256 two blocks fit an SM, and one's loads and merges pass
  // beside the other's products.
  static constexpr int kSlots = 3;
  static constexpr int kTile = kTileKeys * D * 2;
  static constexpr int kMaxRows = 32;
  static constexpr int kSmem = kSlots * kTile + kMaxRows * D * 2;
  static constexpr int kBlocks = D == 256 ? 2 : D == 128 ? 3 : 4;  // an SM's
  static_assert(kBlocks * (kSmem + 1024) <= 233472, "shared memory exceeded");
  static_assert(64 * D * 4 + (64 + 16) * 8 <= kSlots * kTile, "the warps' states do not fit the ring");
};

// One block's work: `rows` query rows (row r: sequence b0 + r / G, head
// h G + r % G) against the keys k0 .. k1 - 1 at K, V (rows ld elements apart).
struct PfItem {
  int h, row0, rows, b0;
  const uint16_t *K, *V;
  int64_t ld;
  int k0, k1, slot;
  // JOINED: keys from n0 on are K2's, V2's from their first
  int n0;
  const uint16_t *K2, *V2;
  int64_t ld2;
};

// Where a JOINED block leaves its state: the rows' outputs at the start of
// shared memory, their (reference, sum) here.
template <int D>
MOE_DEVINL float2* joined_ml(uint8_t* smem) {
  return reinterpret_cast<float2*>(smem + 64 * D * 4 + 64 * 8);
}

// JOINED: the keys are one sequence's, the prefix's and then its own, and the
// state stays in shared memory; else it goes to the partial states.
template <int D, int WM, bool JOINED>
MOE_DEVINL void attend(const PrefixParams& p, const PfItem& it, uint8_t* smem) {
  using C = PfCfg<D>;
  constexpr int WK = 4 / WM, KS = kTileKeys / WK, NT = KS / 8;
  constexpr int kChunks = D / 8;  // 16-byte chunks a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wm = warp % WM, wk = warp / WM;
  const int G = p.Hq / p.Hkv, g = lane >> 2, t = lane & 3;
  uint8_t* qs = smem + C::kSlots * C::kTile;
  auto query_row = [&](int r) { return (int64_t)(it.b0 + r / G) * p.Hq + it.h * G + r % G; };  // of B Hq
  // queries: rows past the end as zeros
  for (int i = tid; i < 16 * WM * kChunks; i += kPfThreads) {
    const int r = i / kChunks, c = i % kChunks;
    const bool in = r < it.rows;
    cp_async_16(smem_u32(qs + tile_off<D>(r, c)), p.q + (in ? query_row(it.row0 + r) * D + c * 8 : 0), in ? 16u : 0u);
  }
  // A thread copies one 16-byte chunk of every kStep-th row of a tile, so that
  // addresses are one add apart (with 4 rows a step, the swizzle alternates).
  constexpr int kStep = kPfThreads / kChunks;
  const int lr = tid / kChunks, lc = tid % kChunks;
  const uint32_t dst[2] = {smem_u32(smem) + tile_off<D>(lr, lc), smem_u32(smem) + tile_off<D>(lr + kStep, lc) - kStep * (D * 2)};
  int fill = 0;  // the next slot to fill
  auto load_tile = [&](const uint16_t* base, const uint16_t* base2, int key) {
    if (key < it.k1) {
      const uint32_t at = fill * C::kTile;
      int64_t src = (int64_t)(key + lr) * it.ld + lc * 8;
      const int left = it.k1 - key - lr;
#pragma unroll 8
      for (int j = 0; j < kTileKeys / kStep; ++j) {
        const bool in = j * kStep < left;  // keys past the end as zeros: their weight is 0 too
        const uint16_t* from = base + src;
        if constexpr (JOINED) {
          const int own = key + lr + j * kStep - it.n0;
          if (own >= 0) from = base2 + own * it.ld2 + lc * 8;
        }
        cp_async_16(dst[j & 1] + at + j * kStep * (D * 2), in ? from : p.q, in ? 16u : 0u);
        src += kStep * it.ld;
      }
    }
    cp_async_commit();
    fill = fill + 1 == C::kSlots ? 0 : fill + 1;
  };
  load_tile(it.K, it.K2, it.k0);
  load_tile(it.V, it.V2, it.k0);
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  const float scale = p.scale_log2;
  int slot = 0;
  auto next_slot = [&]() -> const uint8_t* {  // the oldest tile, once it has landed and the one before is used up
    cp_async_wait<1>();
    __syncthreads();
    const uint8_t* at = smem + slot * C::kTile;
    slot = slot + 1 == C::kSlots ? 0 : slot + 1;
    return at;
  };
#pragma unroll 1
  for (int key = it.k0; key < it.k1; key += kTileKeys) {
    const uint8_t* ks = next_slot();
    load_tile(it.K, it.K2, key + kTileKeys);
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
#pragma unroll 4
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t a[4];
      ldsm4(a, smem_u32(qs + tile_off<D>(wm * 16 + (lane & 15), 2 * kk + (lane >> 4))));
#pragma unroll
      for (int j = 0; j < NT; j += 2) {
        uint32_t b[4];
        ldsm4(b, smem_u32(ks + tile_off<D>(wk * KS + j * 8 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1))));
        mma_bf16(s[j], a, b[0], b[1]);
        mma_bf16(s[j + 1], a, b[2], b[3]);
      }
    }
    const int first = key + wk * KS + 2 * t;  // this lane's first key
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = first + j * 8 + (i & 1) < it.k1;
        s[j][i] = in ? s[j][i] * scale : -INFINITY;
        mx[i >> 1] = fmaxf(mx[i >> 1], s[j][i]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    }
    const bool move = mx[0] > m[0] + kLazyLog2 || mx[1] > m[1] + kLazyLog2;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float nm = fmaxf(m[r], mx[r]);
        const float f = nm == -INFINITY ? 1.f : ex2(m[r] - nm);  // (m -infinity: 0)
        l[r] *= f;
        m[r] = nm;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][2 * r] *= f;
          o[j][2 * r + 1] *= f;
        }
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[j][i] = ex2(s[j][i] - ref[i >> 1]);
        l[i >> 1] += s[j][i];
      }
    const uint8_t* vs = next_slot();
    load_tile(it.V, it.V2, key + kTileKeys);
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) split_bf16(s[j + (q >> 1)][2 * (q & 1)], s[j + (q >> 1)][2 * (q & 1) + 1], hi[q], lo[q]);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t b[4];
        ldsm4_t(b, smem_u32(vs + tile_off<D>(wk * KS + j * 8 + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * c + (lane >> 4))));
        mma_bf16(o[2 * c], hi, b[0], b[1]);
        mma_bf16(o[2 * c + 1], hi, b[2], b[3]);
        mma_bf16(o[2 * c], lo, b[0], b[1]);
        mma_bf16(o[2 * c + 1], lo, b[2], b[3]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (l[r] != l[r] && m[r] == -INFINITY) m[r] = 0.f;  // nothing but NaN: not a state without positions
  cp_async_wait<0>();
  const int64_t state = (int64_t)it.slot * p.B * p.Hq;
  // the key groups' states of a row tile meet in shared memory
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                // [4 warps][16][D]
  float2* sml = reinterpret_cast<float2*>(smem + 64 * D * 4);  // [4 warps][16]
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = g + 8 * r;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      *reinterpret_cast<float2*>(so + (warp * 16 + row) * D + j * 8 + 2 * t) = make_float2(o[j][2 * r], o[j][2 * r + 1]);
    if (t == 0) sml[warp * 16 + row] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  for (int i = tid; i < 16 * WM * (D / 4); i += kPfThreads) {
    const int row = i / (D / 4), c = i % (D / 4), tile = row / 16, r = row % 16;
    if (row >= it.rows) break;  // (rows rise with i)
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < WK; ++k) M = fmaxf(M, sml[(k * WM + tile) * 16 + r].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < WK; ++k) {
      const int w = (k * WM + tile) * 16 + r;
      const float2 ml = sml[w];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      const float4 v = *reinterpret_cast<const float4*>(so + w * D + c * 4);
      L += f * ml.y;
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if constexpr (JOINED) {  // over warp 0's, which no other thread reads there
      *reinterpret_cast<float4*>(so + row * D + c * 4) = acc;
      if (c == 0) joined_ml<D>(smem)[row] = make_float2(M, L);
    } else {
      const int64_t at = state + query_row(it.row0 + row);
      *reinterpret_cast<float4*>(p.part_o + at * D + c * 4) = acc;
      if (c == 0) p.part_ml[at] = make_float2(M, L);
    }
  }
}

// Blocks 0 .. prefix_blocks - 1: (slice, row tile, KV head) of the prefix, KV
// head fastest; then (slice, sequence, KV head) of the sequences' own positions.
template <int D, int WM>
__global__ void __launch_bounds__(kPfThreads, PfCfg<D>::kBlocks) prefix_kernel(const PrefixParams p) {
  extern __shared__ __align__(128) uint8_t pf_smem[];
  // After the tensor-memory kernel (p.tc) these blocks run beside it: they
  // start once all of its blocks have waited for what came before and need
  // nothing that it writes; what came before is visible with its ticket. The last
  // one waits for its end, so that this launch ends after it and the merge finds
  // both. (Each block waiting would hold the SMs from the rest: 64 sequences of up
  // to 512 own positions, 32768 shared, 2 KV heads of 256: 66 us against 56.5.)
  const bool beside = p.tc != 0;
  if (!beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (beside) {
    if (threadIdx.x == 0) acquire_ticket(p.ticket_word, p.ticket);
    __syncthreads();
  }
  const int G = p.Hq / p.Hkv, R = p.B * G;
  const int prefix_blocks = beside ? 0 : p.prefix_blocks;
  if (!beside && blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  PfItem it;
  int i = blockIdx.x;
  if (i < prefix_blocks) {
    it.h = i % p.Hkv;
    i /= p.Hkv;
    const int tiles = (R + 16 * WM - 1) / (16 * WM), tile = i % tiles, split = i / tiles;
    it.row0 = tile * 16 * WM;
    it.rows = min(16 * WM, R - it.row0);
    it.b0 = 0;
    it.K = p.kp + (int64_t)it.h * D;
    it.V = p.vp + (int64_t)it.h * D;
    it.ld = p.ld_prefix;
    it.k0 = min(p.P, split * p.prefix_slice);
    it.k1 = min(p.P, it.k0 + p.prefix_slice);
    it.slot = split;
    attend<D, WM, false>(p, it, pf_smem);
  } else {
    i -= prefix_blocks;
    it.h = i % p.Hkv;
    i /= p.Hkv;
    const int b = i % p.B, split = i / p.B;
    const int len = max(0, min(p.lens[b], p.S));
    it.row0 = 0;
    it.rows = G;
    it.b0 = b;
    it.K = p.ks + (int64_t)b * p.seq_suffix + (int64_t)it.h * D;
    it.V = p.vs + (int64_t)b * p.seq_suffix + (int64_t)it.h * D;
    it.ld = p.ld_suffix;
    it.k0 = min(len, split * p.suffix_slice);
    it.k1 = min(len, it.k0 + p.suffix_slice);
    it.slot = p.prefix_splits + split;
    if (it.k0 == it.k1) {  // nothing here: only the state has to say so
      for (int r = threadIdx.x; r < G; r += kPfThreads)
        p.part_ml[(int64_t)it.slot * p.B * p.Hq + (int64_t)b * p.Hq + it.h * G + r] = make_float2(-INFINITY, 0.f);
    } else {
      attend<D, 1, false>(p, it, pf_smem);
    }
  }
  if (beside && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Little work: a cluster takes one sequence and KV head, its blocks slices of the
// prefix and the sequence's own positions joined, and merges their states from
// distributed shared memory: one launch and no workspace, where launches and
// allocations are most of the time. The prefix is then read once a sequence
// (from L2 but for the first).
template <int D>
__global__ void __launch_bounds__(kPfThreads, PfCfg<D>::kBlocks) prefix_joined_kernel(const PrefixParams p) {
  extern __shared__ __align__(128) uint8_t pf_smem[];
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = 0;
  const int c0 = blockIdx.x / ranks, h = c0 % p.Hkv, b = c0 / p.Hkv, G = p.Hq / p.Hkv;
  const int len = p.S > 0 ? max(0, min(p.lens[b], p.S)) : 0, n = p.P + len;
  const int slice = ((n + kTileKeys - 1) / kTileKeys + (int)ranks - 1) / (int)ranks * kTileKeys;
  PfItem it;
  it.h = h;
  it.row0 = 0;
  it.rows = G;
  it.b0 = b;
  it.K = p.kp + (int64_t)h * D;
  it.V = p.vp + (int64_t)h * D;
  it.ld = p.ld_prefix;
  it.n0 = p.P;
  it.K2 = p.ks + (int64_t)b * p.seq_suffix + (int64_t)h * D;
  it.V2 = p.vs + (int64_t)b * p.seq_suffix + (int64_t)h * D;
  it.ld2 = p.ld_suffix;
  it.k0 = min(n, (int)rank * slice);
  it.k1 = min(n, it.k0 + slice);
  it.slot = 0;
  float2* ml = joined_ml<D>(pf_smem);
  if (it.k0 < it.k1)
    attend<D, 1, true>(p, it, pf_smem);
  else if (threadIdx.x < 16)
    ml[threadIdx.x] = make_float2(-INFINITY, 0.f);
  cluster_sync();
  for (int i = rank * kPfThreads + threadIdx.x; i < G * (D / 4); i += ranks * kPfThreads) {
    const int row = i / (D / 4), c = i % (D / 4);
    float2 s[8];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      s[r] = make_float2(-INFINITY, 0.f);
      if (r < (int)ranks)
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(s[r].x), "=f"(s[r].y) : "r"(remote_addr(ml + row, r)) : "memory");
      M = fmaxf(M, s[r].x);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (s[r].x == -INFINITY) continue;  // (no state: its outputs were not written)
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(remote_addr(pf_smem + row * (D * 4) + c * 16, r))
                   : "memory");
      const float f = ex2(s[r].x - M);
      L = fmaf(f, s[r].y, L);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // no position at all: zeros
    const int64_t at = ((int64_t)b * p.Hq + h * G + row) * D + c * 4;
    *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
  cluster_sync();  // a block's shared memory stays until the others have read it
}

template <int D>
cudaError_t prefix_joined_launch(const PrefixParams& p, cudaStream_t s) {
  using C = PfCfg<D>;
  static SharedMemoryOptIn opt_in;
  if (const cudaError_t err = opt_in(prefix_joined_kernel<D>, C::kSmem); err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.joined;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * p.joined));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefix_joined_kernel<D>, p);
}

// One query row a block: merges its partial states. First the weights of the
// states (each thread some of them), then the weighted outputs, by groups of
// D / 4 threads over every kGroups-th state.
constexpr int kMaxStates = 2 * kPrefixMaxStates;
template <int D>
__global__ void __launch_bounds__(256) prefix_combine_kernel(const PrefixParams p) {
  constexpr int kCols = D / 4, kGroups = 256 / kCols;
  __shared__ float4 acc_s[kGroups][kCols];
  __shared__ float w_s[kMaxStates], red[2][8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int64_t row = blockIdx.x, rows = (int64_t)p.B * p.Hq;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.ticket_word = 0;
    if (p.prefix_splits + p.suffix_splits == 0) *p.status = 0;  // no launch before this one
  }
  const int tid = threadIdx.x, c = tid % kCols, grp = tid / kCols, n = p.prefix_splits + p.suffix_splits;
  constexpr int kPer = (kMaxStates + 255) / 256;
  float2 ml[kPer];
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid + i * 256;
    ml[i] = s < n ? p.part_ml[s * rows + row] : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, ml[i].x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if ((tid & 31) == 0) red[0][tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, red[0][w]);
  float L = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = tid + i * 256;
    const float f = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - M);
    if (s < n) w_s[s] = f;
    L = fmaf(f, ml[i].y, L);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  if ((tid & 31) == 0) red[1][tid >> 5] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) L += red[1][w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = grp; s < n; s += kGroups) {
    const float f = w_s[s];
    if (f == 0.f) continue;  // (a state without positions has no output)
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (s * rows + row) * D + c * 4);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  acc_s[grp][c] = acc;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int k = 1; k < kGroups; ++k) {
      const float4 v = acc_s[k][c];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // no position at all: zeros
    *reinterpret_cast<uint2*>(p.out + row * D + c * 4) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
}

template <int D, int WM>
cudaError_t prefix_launch_t(const PrefixParams& p, cudaStream_t s) {
  using C = PfCfg<D>;
  static SharedMemoryOptIn opt_in;
  if (const cudaError_t err = opt_in(prefix_kernel<D, WM>, C::kSmem); err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.tc) {
    const cudaError_t err = prefix_tc_launch(p, s);
    if (err != cudaSuccess) return err;
  }
  const int64_t blocks = (p.tc ? 0 : p.prefix_blocks) + (int64_t)p.suffix_splits * p.B * p.Hkv;
  if (blocks > 0) {
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kPfThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, prefix_kernel<D, WM>, p);
    if (err != cudaSuccess) return err;
  }
  cfg.gridDim = dim3((unsigned)(p.B * p.Hq));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefix_combine_kernel<D>, p);
}

template <int D>
cudaError_t prefix_launch_d(const PrefixParams& p, cudaStream_t s) {
  switch (p.row_warps) {
    case 1: return prefix_launch_t<D, 1>(p, s);
    default: return prefix_launch_t<D, 2>(p, s);
  }
}

}  // namespace

bool prefix_shape_supported(int B, int P, int S, int Hq, int Hkv, int d) {
  return B >= 0 && B <= 65535 && P >= 0 && S >= 0 && P <= 1 << 28 && S <= 1 << 28 && (d == 64 || d == 128 || d == 256) &&
         Hkv >= 1 && Hkv <= 1024 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 16;
}

int prefix_joined_blocks(int B, int P, int S, int Hkv, int d) {
  const int64_t kt = ((int64_t)P + S + kTileKeys - 1) / kTileKeys;
  int cluster = 1;
  while (cluster < 8 && cluster < kt) cluster *= 2;
  // One wave of blocks, two an SM, few tiles a block, and few enough in all that
  // reading the prefix once a sequence costs less than the launch and the
  // allocation saved (about 8 us of a call; 4 sequences over 2000 positions, 2 KV
  // heads of 256, 11 us, 19 over 1983 25).
  return (int64_t)B * Hkv * cluster <= kJoinedBlocks && kt <= kJoinedTiles * cluster &&
                 (int64_t)B * Hkv * kt * (d / 64) <= kJoinedWork
             ? cluster
             : 0;
}

void prefix_plan(PrefixParams& p, int sms) {
  const int R = p.B * (p.Hq / p.Hkv);
  const int per_sm = p.d == 64 ? 4 : 2;  // blocks an SM over which a prefix is cut
  const int64_t room = (int64_t)std::min(sms, kPrefixMaxSms) * per_sm;
  // More than 32 rows a KV head go to tensor memory, 128 rows a block, one block
  // an SM, against the warps' products (16 or 32 rows a block): 32768 positions, 2 KV
  // heads of 256, 40 rows 23.8 us against 34.1, heads of 128 13.9 against 23.1, of 64
  // 12.3 against 13.5; 33 rows, 4 KV heads of 128, 4000 positions 10.8 against 12.1
  // (300 positions 8.3 against 6.5: the longer chain of a short slice).
  p.tc = R > 32 && p.P >= kPrefixTcMin;
  p.row_warps = R <= 16 ? 1 : 2;
  const int tile_rows = p.tc ? 128 : 16 * p.row_warps, tiles = (R + tile_rows - 1) / tile_rows;
  // slices of whole key tiles, `least` of them or more, at most `blocks` blocks
  auto slices = [&](int len, int64_t blocks, int64_t others, int keys, int least, int& slice, int& splits) {
    const int64_t kt = ((int64_t)len + keys - 1) / keys;
    int64_t want = std::min<int64_t>((kt + least - 1) / least, std::max<int64_t>(1, blocks / std::max<int64_t>(1, others)));
    want = std::max<int64_t>(1, std::min<int64_t>(want, kPrefixMaxStates));
    slice = (int)((kt + want - 1) / want) * keys;
    splits = len ? (int)(((int64_t)len + slice - 1) / slice) : 0;
  };
  // The tensor-memory kernel leaves SMs to the blocks that run beside it: by the
  // work of both (a 64-key tile of one sequence takes about as long as one of 128
  // rows; lengths are taken to be half of S).
  int64_t tc_sms = std::min(sms, kPrefixMaxSms);
  if (p.tc) {
    const double own = 0.5 * p.S * p.B, shared = (double)p.P * tiles;
    tc_sms = std::max<int64_t>(tc_sms / 2, (int64_t)(tc_sms * (shared / (own + shared))));
  }
  // the prefix in one wave of blocks; the sequences' own positions, ragged, in up to four of shorter ones
  slices(p.P, p.tc ? tc_sms : room, (int64_t)p.Hkv * tiles, p.tc && p.d != 256 ? 128 : kTileKeys, 1,
         p.prefix_slice, p.prefix_splits);
  slices(p.S, 4 * room, (int64_t)p.Hkv * p.B, kTileKeys, 2, p.suffix_slice, p.suffix_splits);
  p.prefix_blocks = p.prefix_splits * p.Hkv * tiles;
}

cudaError_t prefix_launch(const PrefixParams& p, cudaStream_t s) {
  if (p.joined) {
    if (p.d == 256) return prefix_joined_launch<256>(p, s);
    return p.d == 128 ? prefix_joined_launch<128>(p, s) : prefix_joined_launch<64>(p, s);
  }
  if (p.d == 256) return prefix_launch_d<256>(p, s);
  if (p.d == 128) return prefix_launch_d<128>(p, s);
  return prefix_launch_d<64>(p, s);
}

}  // namespace moe
