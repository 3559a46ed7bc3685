// Norms of each head's queries and keys, their rotation by position, and the writing of
// new keys and values to a paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pairs (a, b) of y turned by position * freq
//
// A block takes a few tokens. Their places in the cache (a lane a token) and their sines and
// cosines (a thread a pair) are made once and kept in shared memory; then one warp or several take a
// token's heads, four loads of heads at a time. A lane holds 8 elements of a head, four pairs
// (a, b) where it turns: (a0 a1 a2 a3 | b0 b1 b2 b3) from two places, or (a0 b0 a1 b1 | ...), so
// that no pair is spread over lanes; a head takes d / 8 lanes (rounded up to 8, 16 or 32), a warp's
// load 1, 2 or 4 whole heads. The weights go into the sines and cosines once a token. Loads of heads do not
// wait for angles or places. Bound by HBM for many tokens, by one chain of load - sum - store for few.
//
// Angles: a frequency is held as the part of a whole turn that one position makes, in
// 64 bits with the point in front (freq / 2 pi mod 1); times the position, mod 2^64,
// it is the part of a turn that is left, whole turns gone, to 2^-31 of a turn at any
// 32-bit position (for frequencies up to 1). The top 32 bits go to sincospi. (In fp32 position * freq alone is
// 0.06 radians off at a million; in FP64, a 64th of the fp32 rate here, the angles of a
// token would take longer than its heads.)
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;

// freq / (2 pi) mod 1 in units of 2^-64. freq = M 2^(e - 150) with a 24-bit M;
// M 2^40 * (2^64 / 2 pi) / 2^64 is freq / 2 pi in units of 2^(e - 126 - 64).
MOE_DEVINL uint64_t turns_per_position(float freq) {
  const uint32_t u = __float_as_uint(freq);
  int e = (int)((u >> 23) & 255u);
  uint32_t m = u & 0x7FFFFFu;
  if (e == 0)
    e = 1;  // subnormal
  else
    m |= 0x800000u;
  const uint64_t kInv2Pi = 2935890503282001226ull;  // round(2^64 / (2 pi))
  const uint64_t f = __umul64hi((uint64_t)m << 40, kInv2Pi);
  const int shift = e - 126;
  const uint64_t r = shift >= 0 ? (shift < 64 ? f << shift : 0) : (shift > -64 ? f >> -shift : 0);
  return (u >> 31) ? 0 - r : r;
}

// Eight elements as four pairs' first and second ones: (a0 a1 a2 a3 | b0 b1 b2 b3), or
// (a0 b0 a1 b1 a2 b2 a3 b3) where ADJ.
template <bool ADJ>
MOE_DEVINL void unpack(const uint2& x, const uint2& y, float2 (&a)[2], float2 (&b)[2]) {
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
  if constexpr (ADJ) {
    a[0] = make_float2(lo(x.x), lo(x.y));
    b[0] = make_float2(hi(x.x), hi(x.y));
    a[1] = make_float2(lo(y.x), lo(y.y));
    b[1] = make_float2(hi(y.x), hi(y.y));
  } else {
    a[0] = make_float2(lo(x.x), hi(x.x));
    a[1] = make_float2(lo(x.y), hi(x.y));
    b[0] = make_float2(lo(y.x), hi(y.x));
    b[1] = make_float2(lo(y.y), hi(y.y));
  }
}
template <bool ADJ>
MOE_DEVINL void pack(const float2 (&a)[2], const float2 (&b)[2], uint2& x, uint2& y) {
  if constexpr (ADJ) {
    x = make_uint2(pack_bf16(a[0].x, b[0].x), pack_bf16(a[0].y, b[0].y));
    y = make_uint2(pack_bf16(a[1].x, b[1].x), pack_bf16(a[1].y, b[1].y));
  } else {
    x = make_uint2(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y));
    y = make_uint2(pack_bf16(b[0].x, b[0].y), pack_bf16(b[1].x, b[1].y));
  }
}

// The place of token t: its sequence is the last b with starts[b] <= t.
MOE_DEVINL bool find_place(const RopeParams& p, int t, int64_t& place, int& position) {
  int lo = 0, hi = p.B + 1;  // starts[lo - 1] <= t (or lo 0), starts[hi] > t (or hi B + 1)
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.starts[mid] <= t) lo = mid + 1; else hi = mid;
  }
  const int b = lo - 1;
  if (b < 0 || b >= p.B) return false;  // no sequence's
  const int from = p.starts[b];
  if (t < from || t >= p.starts[b + 1]) return false;  // (only where starts do not rise)
  const int64_t at = (int64_t)max(p.lens[b], 0) + ((int64_t)t - from);
  const int64_t index = at >> p.page_log2;
  if (index >= p.width) return false;
  const int page = p.table[b * p.ld_table + index];
  if (page < 0 || page >= p.n_pages) return false;
  place = page * p.page_stride + (at & ((1 << p.page_log2) - 1)) * p.position_stride;
  position = (int)at;
  return true;
}

// cos and sin of the angle by which a pair of token t turns.
MOE_DEVINL float2 turn_of(const RopeParams& p, int t, int pair, int position) {
  int axis = 0;
  if (p.n_axes > 1) {
    if (p.cyclic) {
      axis = pair % p.n_axes;
      if (axis > 0 && pair >= p.n_axes * (axis == 1 ? p.sections[1] : axis == 2 ? p.sections[2] : p.sections[3])) axis = 0;
    } else {
      axis = (pair >= p.sections[0]) + (pair >= p.sections[0] + p.sections[1]) +
             (pair >= p.sections[0] + p.sections[1] + p.sections[2]);
      axis = min(axis, p.n_axes - 1);
    }
  }
  const int pos = p.positions ? p.positions[axis * p.ld_positions + t] : position;
  const float freq = p.freqs[pair];
  const uint64_t turn = turns_per_position(freq) * (uint64_t)(int64_t)pos;
  const int32_t left = (int32_t)(uint32_t)((turn + 0x80000000ull) >> 32);  // of a turn, in 2^-32
  float2 cs;
  sincospif((float)left * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
  const float bad = freq - freq;  // NaN for a frequency that is not finite
  return make_float2(cs.x + bad, cs.y + bad);
}

constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxTokens = 32;  // a block's

template <int LPR, bool PAGED, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeParams p) {
  constexpr int RPW = 32 / LPR;  // heads a warp's load holds: a group
  constexpr int U = 4;           // groups at a time
  extern __shared__ float2 rope_smem[];  // [tokens][pairs]
  __shared__ int64_t places[kRopeMaxTokens];
  __shared__ int ats[kRopeMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  // Up to 8 warps a token: a block has 8 / split tokens at a time, `tokens` in all. More: a block
  // has one token, of which it is the (blockIdx % token_blocks)-th.
  const int64_t t0 = (int64_t)(blockIdx.x / p.token_blocks) * p.tokens;
  const int n_tokens = (int)min((int64_t)p.tokens, p.T - t0);
  const int j_step = max(1, kRopeWarps / p.split);
  const int share = p.token_blocks > 1 ? (int)(blockIdx.x % p.token_blocks) * kRopeWarps + warp : warp & (p.split - 1);
  int j = p.token_blocks > 1 ? 0 : warp / p.split;  // token of the block
  const int groups0 = (p.part[0].heads + RPW - 1) / RPW, groups = groups0 + (p.part[1].heads + RPW - 1) / RPW;
  int g = share;                                    // first group of a batch
  bool more = j < n_tokens && share < groups;

  // this lane's elements of a head: four from the one place, four from the other
  const int turning = p.pairs / 4;  // lanes that turn
  const bool turns = c < turning, active = c * 8 < p.d;
  const int at_a = ADJ || !turns ? c * 8 : c * 4;
  const int at_b = ADJ || !turns ? at_a + 4 : at_a + p.pairs;

  uint2 va[U], vb[U];
  auto fetch = [&]() {
    int64_t row = t0 + j;
    if (PAGED && p.rows) {
      row = p.rows[row];
      if (row < 0 || row >= p.n_rows) return;  // (left out below)
    }
    const uint16_t* s0 = p.part[0].src + row * p.part[0].ld;
    const uint16_t* s1 = p.part[1].src + row * p.part[1].ld;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gu = g + u * p.split;
      const bool k = gu >= groups0;
      const int head = (k ? gu - groups0 : gu) * RPW + sub;
      if (active && head < (k ? p.part[1].heads : p.part[0].heads)) {
        const uint16_t* s = (k ? s1 : s0) + head * p.d;
        va[u] = *reinterpret_cast<const uint2*>(s + at_a);
        vb[u] = *reinterpret_cast<const uint2*>(s + at_b);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) va[u] = vb[u] = make_uint2(0, 0);
  if (more) fetch();

  if constexpr (PAGED) {
    if (threadIdx.x < n_tokens) {
      const int t = (int)t0 + threadIdx.x;
      int64_t place = 0;
      int position = 0;
      bool in = find_place(p, t, place, position);
      if (in && p.rows) {
        const int row = p.rows[t];
        in = row >= 0 && row < p.n_rows;
      }
      places[threadIdx.x] = in ? place : -1;
      ats[threadIdx.x] = position;
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n_tokens * p.pairs; i += kRopeThreads) {
    const int jt = i / p.pairs, pair = i - jt * p.pairs;
    rope_smem[i] = turn_of(p, (int)t0 + jt, pair, PAGED ? ats[jt] : 0);
  }
  __syncthreads();

  // cos and sin of this lane's pairs, times the weights: a' = a ca - b sb, b' = b cb + a sa
  float2 ca[2], cb[2], sa[2], sb[2];
  auto coefficients = [&](int k) {
    float2 wa[2], wb[2];
    if (const uint16_t* w = k ? p.part[1].weight : p.part[0].weight; w && active) {
      unpack<ADJ>(*reinterpret_cast<const uint2*>(w + at_a), *reinterpret_cast<const uint2*>(w + at_b), wa, wb);
    } else {
      wa[0] = wa[1] = wb[0] = wb[1] = make_float2(1.f, 1.f);
    }
    if (turns && (k ? p.part[1].turn : p.part[0].turn)) {
      const float2* from = rope_smem + j * p.pairs + c * 4;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = from[2 * i], y = from[2 * i + 1];
        const float2 cos = make_float2(x.x, y.x), sin = make_float2(x.y, y.y);
        ca[i] = __fmul2_rn(wa[i], cos);
        cb[i] = __fmul2_rn(wb[i], cos);
        sa[i] = __fmul2_rn(wa[i], sin);
        sb[i] = __fmul2_rn(wb[i], make_float2(-sin.x, -sin.y));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) ca[i] = wa[i], cb[i] = wb[i];
    }
  };
  // one group: the sum of a head's squares, then the head
  auto squares = [&](const float2 (&a)[2], const float2 (&b)[2]) {
    float2 s = __fmul2_rn(a[0], a[0]);
    s = __ffma2_rn(a[1], a[1], s);
    s = __ffma2_rn(b[0], b[0], s);
    s = __ffma2_rn(b[1], b[1], s);
    float ss = s.x + s.y;
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    return ss;
  };
  int made = -1;  // token and part of the coefficients
  while (more) {
    const int64_t place = PAGED ? places[j] : 0;
    if (!PAGED || place >= 0) {
      uint16_t* d0 = p.part[0].dst + (PAGED ? place : (t0 + j) * p.part[0].ld_dst);
      uint16_t* d1 = p.part[1].dst + (PAGED ? place : (t0 + j) * p.part[1].ld_dst);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int gu = g + u * p.split;
        const bool k = gu >= groups0;
        if (gu >= groups) break;  // (the warp's)
        const int head = (k ? gu - groups0 : gu) * RPW + sub;
        const bool norm = (k ? p.part[1].weight : p.part[0].weight) != nullptr, turn = k ? p.part[1].turn : p.part[0].turn;
        uint2 oa = va[u], ob = vb[u];
        if (norm || turn) {
          if (made != 2 * j + k) {
            made = 2 * j + k;
            coefficients(k);
          }
          float2 a[2], b[2];
          unpack<ADJ>(oa, ob, a, b);
          if (norm) {
            float ss = squares(a, b), eps = p.eps;
            const bool over = !(ss <= 3.4e38f);
            if (__any_sync(0xffffffffu, over)) {  // squares past fp32: of a row 2^-70 of this one
              const float f = over ? 8.470329472543003e-22f : 1.f;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                a[i] = make_float2(a[i].x * f, a[i].y * f);
                b[i] = make_float2(b[i].x * f, b[i].y * f);
              }
              const float s2 = squares(a, b);
              if (over) ss = s2, eps = 0.f;
            }
            const float inv = rsqrtf(fmaf(ss, p.inv_d, eps));
            const float2 inv2 = make_float2(inv, inv);
#pragma unroll
            for (int i = 0; i < 2; ++i) a[i] = __fmul2_rn(a[i], inv2), b[i] = __fmul2_rn(b[i], inv2);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 x = __fmul2_rn(a[i], ca[i]), y = __fmul2_rn(b[i], cb[i]);
            if (turns && turn) x = __ffma2_rn(b[i], sb[i], x), y = __ffma2_rn(a[i], sa[i], y);
            a[i] = x, b[i] = y;
          }
          pack<ADJ>(a, b, oa, ob);
        }
        if (active && head < (k ? p.part[1].heads : p.part[0].heads)) {
          uint16_t* to = (k ? d1 : d0) + head * (PAGED ? p.head_stride : (int64_t)p.d);
          *reinterpret_cast<uint2*>(to + at_a) = oa;
          *reinterpret_cast<uint2*>(to + at_b) = ob;
        }
      }
    }
    g += U * p.split;
    if (g >= groups) g = share, j += j_step;
    more = j < n_tokens;
    if (more) fetch();
  }
}

template <int LPR, bool PAGED, bool ADJ>
cudaError_t rope_launch_t(RopeParams p, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / LPR;
  const int groups = (p.part[0].heads + RPW - 1) / RPW + (p.part[1].heads + RPW - 1) / RPW;
  p.inv_d = 1.f / (float)p.d;
  // Few tokens: a token's heads go to several warps, while those are at most the 24 an SM that
  // run at once: 2, 4 or 8 of a block, or more blocks a token. Many: a warp takes several tokens
  // where they have few heads, for at least two batches of loads.
  const int64_t room = std::min<int64_t>(groups, (int64_t)sms * 24 / p.T);
  p.split = 1;
  while (p.split < kRopeWarps && 2 * p.split <= room) p.split *= 2;
  p.token_blocks = 1;
  if (room > kRopeWarps) {
    p.token_blocks = (int)((room + kRopeWarps - 1) / kRopeWarps);
    p.split = p.token_blocks * kRopeWarps;
  }
  p.tokens = std::max(1, kRopeWarps / p.split) * (p.split == 1 ? std::max(1, std::min(kRopeMaxTokens / kRopeWarps, 8 / groups)) : 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.T + p.tokens - 1) / p.tokens * p.token_blocks));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = (size_t)p.tokens * p.pairs * sizeof(float2);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<LPR, PAGED, ADJ>, p);
}

template <bool PAGED, bool ADJ>
cudaError_t rope_launch_p(const RopeParams& p, int sms, cudaStream_t s) {
  if (p.d <= 64) return rope_launch_t<8, PAGED, ADJ>(p, sms, s);
  if (p.d <= 128) return rope_launch_t<16, PAGED, ADJ>(p, sms, s);
  return rope_launch_t<32, PAGED, ADJ>(p, sms, s);
}

}  // namespace

cudaError_t rope_launch(const RopeParams& p, int sms, cudaStream_t s) {
  if (p.adjacent) return p.starts ? rope_launch_p<true, true>(p, sms, s) : rope_launch_p<false, true>(p, sms, s);
  return p.starts ? rope_launch_p<true, false>(p, sms, s) : rope_launch_p<false, false>(p, sms, s);
}

}  // namespace moe
