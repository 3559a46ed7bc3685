// Matrix product of 8-bit integers with a scale per token and per output
// channel:  out[t][n] = a_scale[t] w_scale[n] sum_k a[t][k] w[n][k].
//
// The part's 8-bit integer tensor rate is far below its f16 rate, and every
// int8 is exact in f16 (as is every product, in fp32): so the codes are turned
// into f16 on chip, in three integer operations and two subtractions for four
// codes (the byte with its sign bit flipped under 0x64 is the f16 of 1152 + b),
// and multiplied by the f16 tensor cores with fp32 sums, which are exact while
// they stay below 2^24 in magnitude (always for K <= 1024). Weights stay 8-bit
// in memory.
//
// Two kernels, by the number of tokens:
//
// Few tokens: bound by the weights' bytes. A block owns 16 M weight rows
// and splits K over its 8 warps; a lane loads 16 consecutive codes of two
// rows per m16n8k16 product quadruple (the order of k is free as long as both
// operands agree, so the fragments need no shuffling), and the warps' sums
// meet in shared memory. One token by 4608 x 2048 weights: 3.4 us; 8 tokens by
// 100003 x 2048: 35 us (5.9 TB/s, 87% of the measured copy); 24: 52 us.
//
// More tokens: tcgen05. The MMA's M side is 128 weight rows, its N side up to
// 256 tokens. TMA brings the packed weight codes, converter warps write them as
// f16 straight into tensor memory (the A operand), so shared memory carries
// only the tokens' operand to the MMA. The tokens' codes (far fewer) are
// widened to f16 in the workspace by a first kernel; its launch lets the
// product's start early, and the product's weight stream does not wait for it.
// 8192 x 8192 x 2048: 183 us, 1.50 PFLOP/s (77% of the measured burst rate); the
// MMAs alone take 151 us at the clock that power leaves.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Four int8 codes as two f16 pairs, in order.
MOE_DEVINL uint2 widen4(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;  // 128 + code
  uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 bias = __floats2half2_rn(1152.f, 1152.f);  // 1024 + 128
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// a / b rounded up; a may be any int.
__host__ __device__ constexpr int ceil_div(int a, int b) { return (int)(((int64_t)a + b - 1) / b); }

MOE_DEVINL void store_out(void* out, int f32, int64_t at, float v) {
  if (f32)
    static_cast<float*>(out)[at] = v;
  else
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- few tokens
constexpr int kFewWarps = 8;

MOE_DEVINL void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 M weight rows x 8 NT tokens a block.
template <int M, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, M > 1 || NT <= 2 ? 3 : 2) gemm_w8_few_kernel(const GemmW8Params p) {
  // 64-code steps in flight. Blocks of many rows hide their loads behind each
  // other: three an SM with one step each beat two with two (52 us against 56 for
  // 24 tokens by 100003 x 2048 weights, 42 against 47 for 16).
  constexpr int U = M == 1 ? 4 : 1;
  constexpr int kPitch = 16 * M + 4;
  __shared__ float red[kFewWarps][8 * NT][kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * M);
  const int t0 = blockIdx.y * (8 * NT);  // the block's first token
  const int steps = (p.K + 63) / 64, per = (steps + kFewWarps - 1) / kFewWarps;
  const int s0 = warp * per, s1 = min(steps, s0 + per);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.status) *p.status = 0;
  float acc[M][NT][4];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.f;
  const int8_t* wrow[M][2];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows past the end repeat the last one and are not stored
      wrow[m][h] = p.w + min(n0 + 16 * m + 8 * h + g, (int64_t)p.N - 1) * p.K;
  const int8_t* arow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) arow[j] = p.a + (int64_t)min(t0 + 8 * j + g, p.T - 1) * p.lda;
#pragma unroll 1
  for (int s = s0; s < s1; s += U) {
    uint4 wv[U][M][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 64 + 16 * t;
      const bool in = s + u < s1 && k < p.K;  // K is a multiple of 16
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          wv[u][m][h] = in ? __ldcs(reinterpret_cast<const uint4*>(wrow[m][h] + k)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 64 + 16 * t;
      const bool in = s + u < s1 && k < p.K;
      uint4 av[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        av[j] = in ? __ldg(reinterpret_cast<const uint4*>(arow[j] + k)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        auto word = [&](const uint4& v) { return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w; };
        uint2 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = widen4(word(av[j]));
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const uint2 lo = widen4(word(wv[u][m][0])), hi = widen4(word(wv[u][m][1]));
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_16816(acc[m][j], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][8 * j + 2 * t + (i & 1)][16 * m + g + 8 * (i >> 1)] = acc[m][j][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * M * 8 * NT; i += 32 * kFewWarps) {
    const int r = i % (16 * M), c = i / (16 * M), tok = t0 + c;
    const int64_t n = n0 + r;
    if (tok < p.T && n < p.N) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += red[w][c][r];
      store_out(p.out, p.f32, (int64_t)tok * p.ldo + n, v * __ldg(p.a_scale + tok) * __ldg(p.w_scale + n));
    }
  }
}

template <int M, int NT>
cudaError_t few_launch(const GemmW8Params& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div(p.N, 16 * M), (unsigned)ceil_div(p.T, 8 * NT));
  cfg.blockDim = dim3(32 * kFewWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_w8_few_kernel<M, NT>, p);
}
// ---------------------------------------------------------------- many tokens
// The tokens' codes as f16 rows of K, contiguous; clears the status word. The first
// block releases the ticket with which the product's weight stream starts.
__global__ void __launch_bounds__(256) widen_kernel(const GemmW8Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (blockIdx.x == 0) {  // a block of its own: the others need not wait for the release
    if (threadIdx.x == 0) release_ticket(p.ticket_word, p.ticket);
    return;
  }
  const int64_t i = ((int64_t)blockIdx.x - 1) * 256 + threadIdx.x;
  const int vecs = p.K / 16;
  if (i == 0) *p.status = 0;
  if (i >= (int64_t)p.T * vecs) return;
  const int64_t row = i / vecs;
  const int k = (int)(i - row * vecs) * 16;
  const uint4 v = *reinterpret_cast<const uint4*>(p.a + row * p.lda + k);
  const uint2 a = widen4(v.x), b = widen4(v.y), c = widen4(v.z), d = widen4(v.w);
  uint4* dst = reinterpret_cast<uint4*>(p.a16 + row * p.K + k);
  dst[0] = make_uint4(a.x, a.y, b.x, b.y);
  dst[1] = make_uint4(c.x, c.y, d.x, d.y);
}

constexpr int kTileN = 128;               // weight rows a tile (the MMA's M)
constexpr int kKB = 128;                  // codes a k-block
constexpr int kQStage = kTileN * kKB;     // packed codes of a stage: 16 KB
constexpr int kEpiWarps = 8;

template <int BN>
struct CfgW8 {
  // Converter groups of four warps; group i converts k-blocks i, i + kGroups, ...
  // At 256 tokens two keep up with the MMAs, and the threads saved leave the
  // epilogue registers for 64 columns at a time.
  static constexpr int kGroups = BN == 256 ? 2 : 4;
  static constexpr int kEpiWarp0 = 4 + 4 * kGroups;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);  // by role, below
  static constexpr int kSQ = 4;                  // packed-code stages
  static constexpr int kSA = 4;                  // f16 weight stages in tensor memory, 64 columns each
  // Token stages of kBK codes. 256 tokens leave room for 160 KB of them beside
  // the packed codes: five stages of half a k-block.
  static constexpr int kBK = BN == 256 ? 64 : 128;
  static constexpr int kBSteps = kKB / kBK;      // token stages a k-block
  static constexpr int kSB = BN == 256 ? 5 : BN == 128 ? 4 : 6;
  static constexpr int kSD = kSA > kSB ? kSA : kSB;
  static constexpr int kBBytes = BN * kBK * 2;
  static constexpr int kAcc = BN == 256 ? 1 : 2;  // tiles in tensor memory: 256 columns in all
  static constexpr int kOffB = 0;
  static constexpr int kOffQ = kSB * kBBytes;
  static constexpr int kOffScale = kOffQ + kSQ * kQStage;  // 32 token scales an epilogue warp
  static constexpr int kOffBar = kOffScale + kEpiWarps * 128;
  // Threads that issue MMAs. What one does between two k-blocks (waits, a
  // commit) is not hidden behind the MMAs of 64 tokens (400 cycles of about
  // 1000): there two take k-blocks in turn, each with an accumulator of its
  // own that the epilogue adds.
  static constexpr int kIssuers = BN == 64 ? 2 : 1;
  static constexpr int kAccCols = kIssuers * BN;  // of one tile
  static constexpr int kACol = kAcc * kAccCols;
  static_assert(kSA % kIssuers == 0 && kSB % (kIssuers * kBSteps) == 0 && kSD % kIssuers == 0 || kIssuers == 1, "an issuer's stages come round to it");
  static constexpr int kBars = 2 * kSQ + kSA + kSB + kSD + 2 + 2 + 1;
  static constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
  static_assert(kACol + kSA * (kKB / 2) <= 512, "tensor memory exceeded");
  static_assert(kSmem <= 232448, "shared memory exceeded");
  // A group waits for its k-block's stage while earlier k-blocks may still be
  // loading: with fewer stages than groups it would wait on a barrier that is
  // two phases behind, whose parity looks like the phase it wants.
  static_assert(kSQ % kGroups == 0 && kSA % kGroups == 0, "every converter group needs stages of its own");
};

struct W8Args {
  CUtensorMap tm_w;  // packed weights [N][K] bytes, box 128 x 128
  CUtensorMap tm_a;  // f16 tokens [T][K], box 64 x BN
  GemmW8Params g;
};

// Roles: warp 0 streams the packed weights, warp 1 issues the MMAs, warp 2
// streams the tokens' operand (with two issuers warp 3 is the other), then the
// converters' warps and the epilogue's.
// Tiles of 128 weight rows by BN tokens, weights fastest, one CTA an SM.
template <int BN, bool F32>
__global__ void __launch_bounds__(CfgW8<BN>::kThreads, 1) gemm_w8_kernel(const __grid_constant__ W8Args args) {
  using C = CfgW8<BN>;
  const GemmW8Params& g = args.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_empty = q_full + C::kSQ;
  uint64_t* a_full = q_empty + C::kSQ;
  uint64_t* b_full = a_full + C::kSA;
  // done[i % kSD]: the MMAs of k-block i have read their operands. One commit
  // frees both: the converters of k-block i wait for k-block i - kSA, the
  // token stream's stage j for the k-block of stage j - kSB; the MMA cannot get
  // kSD k-blocks past either.
  uint64_t* done = b_full + C::kSB;
  uint64_t* acc_full = done + C::kSD;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int MT = ceil_div(g.N, kTileN), TT = ceil_div(g.T, BN), KB = (g.K + kKB - 1) / kKB;
  const int64_t units = (int64_t)MT * TT;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 4);
    }
    for (int i = 0; i < C::kSA; ++i) mbar_init(&a_full[i], 4);
    for (int i = 0; i < C::kSB; ++i) mbar_init(&b_full[i], 1);
    for (int i = 0; i < C::kSD; ++i) mbar_init(&done[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], C::kIssuers);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    mbar_init(drain, C::kIssuers);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tm_w);
    tma_prefetch_desc(&args.tm_a);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // The weights were there before the widening kernel ran (it waited for what
    // came before it) and are visible with its ticket: its end is waited for in warp
    // 2, for the f16 tokens, and by the epilogue. (Waiting here too: 32 tokens by
    // 19000 x 2048 13.9 us against 12.9, 300 by 8192 x 2048 19.1 against 18.3.)
    if (lane == 0) {
      acquire_ticket(g.ticket_word, g.ticket);
      fence_proxy_async_global();
      // With one tile of tokens the weights are read once and need not stay in L2:
      // 64 tokens by 100003 x 2048 weights 47.6 us against 48.9, 64 by 16384 x 2048
      // 12.1 against 13.0. With several, each of them reads the weights again.
      const uint64_t policy = TT == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
      uint32_t it = 0;
      bool alive = true;
      for (int64_t u = blockIdx.x; u < units && alive; u += gridDim.x) {
        const int row = (int)(u % MT) * kTileN;
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const int s = it % C::kSQ;
          if (!mbar_wait(&q_empty[s], ((it / C::kSQ) & 1) ^ 1, abort_flag, g.status, 61)) {
            alive = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[s], kQStage);
          tma_load_2d(smem + C::kOffQ + s * kQStage, &args.tm_w, kb * kKB, row, &q_full[s], policy);
        }
      }
      // every load lands before the CTA ends, also when another role gave up
      volatile int drained = 0;
      for (uint32_t j = it > (uint32_t)C::kSQ ? it - C::kSQ : 0; j < it; ++j)
        mbar_wait(&q_full[j % C::kSQ], (j / C::kSQ) & 1, &drained, g.status, 62);
    }
  } else if (warp == 2) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_last();
      uint32_t it = 0;
      bool alive = true;
      for (int64_t u = blockIdx.x; u < units && alive; u += gridDim.x) {
        const int row = (int)(u / MT) * BN;
        for (int ks = 0; ks < KB * C::kBSteps; ++ks, ++it) {
          const int s = it % C::kSB;
          const uint32_t before = (it - C::kSB) / C::kBSteps;  // the k-block that used this stage
          if (it >= (uint32_t)C::kSB &&
              !mbar_wait(&done[before % C::kSD], (before / C::kSD) & 1, abort_flag, g.status, 63)) {
            alive = false;
            break;
          }
          mbar_arrive_expect_tx(&b_full[s], C::kBBytes);
#pragma unroll
          for (int h = 0; h < C::kBK / 64; ++h)  // (columns and rows past the ends read as zero)
            tma_load_2d(smem + C::kOffB + s * C::kBBytes + h * (BN * 128), &args.tm_a, ks * C::kBK + h * 64, row,
                        &b_full[s], policy);
        }
      }
      volatile int drained = 0;
      for (uint32_t j = it > (uint32_t)C::kSB ? it - C::kSB : 0; j < it; ++j)
        mbar_wait(&b_full[j % C::kSB], (j / C::kSB) & 1, &drained, g.status, 62);
    }
  } else if (warp == 1 || (C::kIssuers == 2 && warp == 3)) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(kTileN, BN);
      // Stage indices and phases are carried, not divided out of a counter, and
      // descriptors are one add from a base: this thread's own work paces small N.
      constexpr uint32_t kI = C::kIssuers;
      const uint32_t me = kI == 2 ? warp >> 1 : 0;  // takes k-blocks me, me + kI, ... of all the CTA's
      const uint64_t b_desc0 = smem_desc_sw128(smem_u32(smem + C::kOffB));
      uint32_t sa = me, pa = 0, sb = me * C::kBSteps, pb = 0, sd = me, buf = 0, pacc = 1;
      int skip = (int)me;  // k-blocks of the next tile before this thread's first
      bool alive = true;
      for (int64_t u = blockIdx.x; u < units && alive; u += gridDim.x) {
        if (!mbar_wait(&acc_empty[buf], pacc, abort_flag, g.status, 64)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + buf * C::kAccCols + me * BN;
        uint32_t accumulate = 0;
        int kb = skip;
#pragma unroll 1
        for (; kb < KB; kb += kI) {
          if (!mbar_wait(&a_full[sa], pa, abort_flag, g.status, 66)) {
            alive = false;
            break;
          }
          const uint32_t a_tmem = tmem + C::kACol + sa * (kKB / 2);
#pragma unroll
          for (int h = 0; h < C::kBSteps; ++h) {
            if (!mbar_wait(&b_full[sb], pb, abort_flag, g.status, 65)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t b_desc = b_desc0 + sb * (C::kBBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < C::kBK / 16; ++kk) {
              tc_mma_ts(d_tmem, a_tmem + (h * (C::kBK / 16) + kk) * 8,
                        b_desc + (((kk / 4) * (BN * 128) + (kk % 4) * 32) >> 4), idesc, accumulate);
              accumulate = 1;
            }
            sb += h + 1 < C::kBSteps ? 1 : 1 + (kI - 1) * C::kBSteps;
            if (sb >= C::kSB) sb -= C::kSB, pb ^= 1;
          }
          if (!alive) break;
          tc_commit(&done[sd]);
          if ((sa += kI) >= C::kSA) sa -= C::kSA, pa ^= 1;
          if ((sd += kI) >= C::kSD) sd -= C::kSD;
        }
        if (!alive) break;
        skip = kb - KB;
        tc_commit(&acc_full[buf]);
        if (++buf == C::kAcc) buf = 0, pacc ^= 1;
      }
      volatile int drained = 0;
      tc_commit(drain);  // all MMAs complete before tensor memory is freed
      mbar_wait(drain, 0, &drained, g.status, 67);
    }
  } else if (warp >= 4 && warp < C::kEpiWarp0) {
    // thread = one weight row of every kGroups-th k-block: a k-block takes
    // its group about 1000 cycles from wait to signal, most of it latency, so
    // several are under way at once
    const int m = (warp & 3) * 32 + lane, group = (warp - 4) >> 2;
    const uint32_t a_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kACol;
    const int64_t mine = blockIdx.x < units ? ((units - 1 - blockIdx.x) / gridDim.x + 1) * KB : 0;  // this CTA's k-blocks
    for (int64_t it = group; it < mine; it += C::kGroups) {
      const int sq = (int)(it % C::kSQ), sa = (int)(it % C::kSA);
      if (!warp_wait(&q_full[sq], (uint32_t)(it / C::kSQ) & 1, abort_flag, g.status, 68)) break;
      uint4 q[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)  // 16-byte chunk index XOR (row % 8), as TMA wrote it
        q[c] = *reinterpret_cast<const uint4*>(smem + C::kOffQ + sq * kQStage + m * 128 + ((c ^ (m & 7)) << 4));
      if (it >= C::kSA &&
          !warp_wait(&done[(it - C::kSA) % C::kSD], (uint32_t)((it - C::kSA) / C::kSD) & 1, abort_flag, g.status, 69))
        break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t r[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t w[4] = {q[2 * h + c].x, q[2 * h + c].y, q[2 * h + c].z, q[2 * h + c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v = widen4(w[i]);
            r[8 * c + 2 * i] = v.x;
            r[8 * c + 2 * i + 1] = v.y;
          }
        }
        tmem_st_32x32b_x16(a_tmem + sa * (kKB / 2) + h * 16, r);
      }
      warp_arrive(&q_empty[sq]);  // (its codes were consumed)
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&a_full[sa]);
    }
  } else if (warp >= C::kEpiWarp0) {
    // lanes of quarter warp % 4 = 32 weight rows; the two groups of four warps take half the tokens each
    const int quarter = warp & 3, group = (warp - C::kEpiWarp0) >> 2;
    constexpr int kCols = BN / 2, kChunk = C::kIssuers == 2 ? 16 : BN == 256 ? 64 : 32;
    using Out = typename std::conditional<F32, float, __nv_bfloat16>::type;
    float4* scales = reinterpret_cast<float4*>(smem + C::kOffScale + (warp - C::kEpiWarp0) * 128);
    uint32_t tile = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (the scales)
    int64_t u = blockIdx.x;
    for (; u < units; u += gridDim.x, ++tile) {
      const uint32_t buf = tile % C::kAcc;
      const int64_t n = (u % MT) * kTileN + quarter * 32 + lane;
      const int64_t t0 = u / MT * BN + group * kCols;  // (may pass 32 bits where the tile ends past the tokens)
      const float ws = n < g.N ? __ldg(g.w_scale + n) : 0.f;
      if (!warp_wait(&acc_full[buf], (tile / C::kAcc) & 1, abort_flag, g.status, 70)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + buf * C::kAccCols + group * kCols;
      // a tile of one k-block has one issuer's sums only: those of the tile's turn
      const uint32_t single = KB == 1 ? (tile & 1) * BN : 0;
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += kChunk) {
        __syncwarp();  // (the stores of the chunk before part the lanes)
        uint32_t v[kChunk];
        if constexpr (C::kIssuers == 2) {
          uint32_t v2[kChunk];
          tmem_ld_32x32b_x16(taddr + single + c0, v);
          tmem_ld_32x32b_x16(taddr + BN + c0, v2);
          tc_wait_ld();
          if (KB > 1) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(v2[i]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < kChunk; i += 32) tmem_ld_32x32b_x32(taddr + c0 + i, reinterpret_cast<uint32_t(&)[32]>(v[i]));
          tc_wait_ld();
        }
        if (c0 + kChunk == kCols) {  // the accumulator is in registers: the next tile may start
          tc_fence_before();
          warp_arrive(&acc_empty[buf]);
        }
        constexpr int kPut = kChunk < 32 ? kChunk : 32;  // tokens whose scales are at hand
#pragma unroll
        for (int i0 = 0; i0 < kChunk; i0 += kPut) {
          const int64_t t = t0 + c0 + i0;
          const int live = (int)(g.T - t);
          __syncwarp();
          reinterpret_cast<float*>(scales)[lane] = lane < live ? __ldg(g.a_scale + t + lane) : 0.f;
          __syncwarp();
          Out* dst = static_cast<Out*>(g.out) + t * g.ldo + n;
          auto put = [&](uint32_t acc, float as) {
            const float y = __uint_as_float(acc) * as * ws;
            if constexpr (F32)
              *dst = y;
            else
              *dst = __float2bfloat16_rn(y);
            dst += g.ldo;
          };
          if (n < g.N) {  // one row of 32 outputs a store
            if (live >= kPut) {
#pragma unroll
              for (int i = 0; i < kPut / 4; ++i) {
                const float4 as = scales[i];
                put(v[i0 + 4 * i], as.x);
                put(v[i0 + 4 * i + 1], as.y);
                put(v[i0 + 4 * i + 2], as.z);
                put(v[i0 + 4 * i + 3], as.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < kPut; ++i)
                if (i < live) put(v[i0 + i], reinterpret_cast<const float*>(scales)[i]);
            }
          }
        }
      }
    }
    // after a wait that ran out: what was not computed is NaN, beside the status
#pragma unroll 1
    for (; u < units; u += gridDim.x) {
      const int64_t n = (u % MT) * kTileN + quarter * 32 + lane, t0 = u / MT * BN + group * kCols;
#pragma unroll 1
      for (int64_t t = t0; t < t0 + kCols && t < g.T; ++t)
        if (n < g.N) store_out(g.out, F32, t * g.ldo + n, __int_as_float(0x7fc00000));
    }
  }
  __syncwarp();  // the single-lane roles join their warps
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  // (a block that starts after this waits for the widening kernel instead)
  if (blockIdx.x == 0 && threadIdx.x == 0) *g.ticket_word = 0;
}

bool encode_2d(CUtensorMap* tm, CUtensorMapDataType type, int esize, const void* p, int64_t rows, int64_t cols, int box_cols,
               int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * esize};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(tm, type, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool F32>
cudaError_t many_launch_t(const GemmW8Params& p, int sms, cudaStream_t s) {
  using C = CfgW8<BN>;
  W8Args args;
  memset(&args, 0, sizeof args);
  args.g = p;
  if (!encode_2d(&args.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.w, p.N, p.K, kKB, kTileN) ||
      !encode_2d(&args.tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, p.a16, p.T, p.K, 64, BN))
    return cudaErrorInvalidValue;
  static SharedMemoryOptIn opt_in;
  if (const cudaError_t err = opt_in(gemm_w8_kernel<BN, F32>, C::kSmem); err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(((int64_t)p.T * (p.K / 16) + 255) / 256 + 1));
  cfg.blockDim = dim3(256);
  cudaError_t err = cudaLaunchKernelEx(&cfg, widen_kernel, p);
  if (err != cudaSuccess) return err;
  const int64_t units = (int64_t)ceil_div(p.N, kTileN) * ceil_div(p.T, BN);
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, units));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  return cudaLaunchKernelEx(&cfg, gemm_w8_kernel<BN, F32>, args);
}
template <int BN>
cudaError_t many_launch(const GemmW8Params& p, int sms, cudaStream_t s) {
  return p.f32 ? many_launch_t<BN, true>(p, sms, s) : many_launch_t<BN, false>(p, sms, s);
}

}  // namespace

// More than 24 tokens stay with the first kernel, 32 at a time, while its
// blocks of 16 weight rows fill the machine at most twice (once where K is
// short and a block has little to do): 64 tokens by 4608 x 2048 weights 7.9 us
// against 12.2, 64 by 2048 x 2048 4.6 against 12.2.
bool gemm_w8_few(int T, int N, int K) {
  const int64_t blocks = (int64_t)ceil_div(N, 16) * ceil_div(T, 32);
  return T <= kW8FewTokens || blocks <= (int64_t)kW8RuleSms * (K < 1024 ? 2 : 4);
}

cudaError_t gemm_w8_launch(const GemmW8Params& p, int sms, cudaStream_t s) {
  if (gemm_w8_few(p.T, p.N, p.K)) {
    const int nt = ceil_div(p.T, 8);
    // Rows a block: more reuse the tokens' fragments, fewer fill the machine. With 32
    // rows 100003 x 2048 weights take 34, 35, 42 and 52 us at 1, 8, 16 and 24 tokens
    // (with 64 rows 35 and 37 at 1 and 8; 32768 x 8192 at 1 token 44 to 47 against 55). In
    // tensor memory they take 60 us at 17 tokens, 55 at 24 and 49 at 25, from where
    // it serves. It is ahead sooner by long rows (17 and 24 tokens by 32768 x 8192: 59
    // us against 67 and 69; by 20480 x 4096 31 against 25), but wants a workspace,
    // which the interface promises not to want up to 24 tokens.
    if (p.N >= 32 * 4 * kW8RuleSms) {  // several blocks an SM even so
      if (nt == 1) return few_launch<2, 1>(p, s);
      return nt == 2 ? few_launch<2, 2>(p, s) : few_launch<2, 3>(p, s);
    }
    if (nt == 1) return few_launch<1, 1>(p, s);
    if (nt == 2) return few_launch<1, 2>(p, s);
    return nt == 3 ? few_launch<1, 3>(p, s) : few_launch<1, 4>(p, s);
  }
  // The token width whose waves cost least, by the measured time of a k-block
  // (about 0.48, 0.56 and 0.72 us at 64, 128 and 256 tokens) and a tile's ends.
  const int64_t MT = ceil_div(p.N, kTileN), kb = (p.K + kKB - 1) / kKB;
  auto cost = [&](int bn, int64_t step, int64_t ends) {
    return (MT * ceil_div(p.T, bn) + sms - 1) / sms * (kb * step + ends);
  };
  const int64_t c64 = cost(64, 48, 50), c128 = cost(128, 56, 80), c256 = cost(256, 72, 150);
  if (c256 <= c128 && c256 <= c64) return many_launch<256>(p, sms, s);
  return c128 <= c64 ? many_launch<128>(p, sms, s) : many_launch<64>(p, sms, s);
}

}  // namespace moe
