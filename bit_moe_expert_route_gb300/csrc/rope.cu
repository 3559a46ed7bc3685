// Norms of each head's queries and keys, their rotation by position, and the writing of
// new keys and values to a paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pairs (a, b) of y turned by position * freq
//
// A block takes a few tokens. Their places in the cache (a lane a token) and their sines and
// cosines (a thread a pair) are made once and kept in shared memory; then one warp or several take a
// token's heads, two loads of heads at a time. A lane holds 8 elements of a head, four pairs
// (a, b) where it turns: (a0 a1 a2 a3 | b0 b1 b2 b3) from two places, or (a0 b0 a1 b1 | ...), so
// that no pair is spread over lanes; a head takes d / 8 lanes (rounded up to 8, 16 or 32), a warp's
// load 1, 2 or 4 whole heads. The weights go into the sines and cosines once a token. Loads of heads do not
// wait for angles or places.
//
// Few tokens: one chain of load - sum - store, 2.2 us. 32768 tokens of 16 + 2 heads of 256: 109 us,
// 82% of the measured copy; the same without arithmetic 96 us. About 160 instructions a head fill two
// thirds of the issue slots. (Blocks of 128 threads; of 256, whose warps wait for each other's places and sines, 112
// us. Warps that go from token to token by themselves 119 to 128.) Appending 32768 tokens of 2 heads of 256: 32 us,
// 62% of the copy, blocks of 256 threads 36.
//
// Angles: a frequency is held as the part of a whole turn that one position makes, in
// 64 bits with the point in front (freq / 2 pi mod 1); times the position, mod 2^64,
// it is the part of a turn that is left, whole turns gone, to 2^-33 of a turn at any
// 32-bit position. The top 32 bits go to sincospi. (In fp32 position * freq alone is
// 0.06 radians off at a million; in FP64, a 64th of the fp32 rate here, the angles of a
// token would take longer than its heads.)
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRopeThreads = 128;

// freq / (2 pi) mod 1 in units of 2^-64, cut off below them, for |freq| < 2^16. freq = M 2^(e - 150) with a 24-bit M, and
// the product of M and 2^128 / (2 pi), times 2^(e - 214), is that. (128 bits: of 64, the places that a frequency of
// 2^15 shifts in would be missing, 2^-14 radians at position 2^31.)
MOE_DEVINL uint64_t turns_per_position(float freq) {
  const uint32_t u = __float_as_uint(freq);
  int e = (int)((u >> 23) & 255u);
  uint32_t m = u & 0x7FFFFFu;
  if (e == 0)
    e = 1;  // subnormal
  else
    m |= 0x800000u;
  const uint64_t kHigh = 2935890503282001226ull, kLow = 9154082963658192752ull;  // round(2^128 / (2 pi))
  const uint64_t carried = __umul64hi((uint64_t)m, kLow), low = m * kHigh + carried;
  const uint64_t high = __umul64hi((uint64_t)m, kHigh) + (low < carried);
  const int shift = max(1, 150 - e);  // of (high, low), the product's bits from the 64th on
  const uint64_t r = shift < 64 ? low >> shift | high << (64 - shift) : shift < 128 ? high >> (shift - 64) : 0;
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

// The last b with starts[b] <= t (-1: none; B: t is past the last), by a warp: 32 places a step.
MOE_DEVINL int find_sequence(const int32_t* starts, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;  // starts[lo - 1] <= t, starts[lo + n] > t
#pragma unroll 1
  while (n > 0) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = at < lo + n && starts[at] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // (rising: the first c lanes)
    if (c == 0) break;
    const int end = lo + n;
    lo += (c - 1) * step + 1;
    n = min(step - 1, end - lo);
  }
  return lo - 1;
}

// The place of token t, whose sequence is b or one after it.
MOE_DEVINL bool find_place(const RopeParams& p, int b, int t, int64_t& place, int& position) {
  b = max(b, 0);
  int from = b < p.B ? p.starts[b] : 0, to = b < p.B ? p.starts[b + 1] : 0;
#pragma unroll 1
  for (int i = 0; i < 3 && b < p.B && t >= to; ++i) {
    ++b;
    from = to;
    if (b < p.B) to = p.starts[b + 1];
  }
  if (b < p.B && t >= to) {  // many short sequences
    int hi = p.B + 1;
#pragma unroll 1
    while (b < hi) {
      const int mid = (b + hi) / 2;
      if (p.starts[mid] <= t) b = mid + 1; else hi = mid;
    }
    --b;
    if (b >= 0 && b < p.B) from = p.starts[b], to = p.starts[b + 1];
  }
  if (b < 0 || b >= p.B || t < from || t >= to) return false;  // no sequence's
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
MOE_DEVINL float2 turn_of(const RopeParams& p, int t, int pair, float freq, uint64_t turns, int position) {
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
  const uint64_t turn = turns * (uint64_t)(int64_t)pos;
  const int32_t left = (int32_t)(uint32_t)((turn + 0x80000000ull) >> 32);  // of a turn, in 2^-32
  float2 cs;
  sincospif((float)left * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
  const float bad = fabsf(freq) < 65536.f ? 0.f : __int_as_float(0x7fc00000);  // a frequency too large or not finite
  return make_float2(cs.x + bad, cs.y + bad);
}

constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxTokens = 32;  // a block's

// The sum of squares of 2^-70 of a head's elements.
template <int LPR>
__device__ __noinline__ float small_squares(float2 a0, float2 a1, float2 b0, float2 b1) {
  const float f = 8.470329472543003e-22f;
  const float x[8] = {a0.x * f, a0.y * f, a1.x * f, a1.y * f, b0.x * f, b0.y * f, b1.x * f, b1.y * f};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// Registers: 28 warps an SM without spills; of 32 and 24 the same 32768 tokens take 109.4 and 114 us, 4099 of 16 heads
// of 128 8.8 and 7.7 instead of 8.5. With places 36, which spill a few registers once a token and hide more of the
// chain (32768 appended tokens 32 us; 28 or 32 warps 34.8, 44 37. 301 accepted tokens 4.6 us, in blocks of 256 threads 4.0: the call takes 13.)
template <int LPR, bool PAGED, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, PAGED ? 9 : 7) rope_kernel(const RopeParams p) {
  constexpr int RPW = 32 / LPR;  // heads a warp's load holds: a group
  constexpr int U = 2;           // groups at a time
  extern __shared__ float2 rope_smem[];  // [tokens][pairs]
  __shared__ int64_t places[kRopeMaxTokens];
  __shared__ int ats[kRopeMaxTokens];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  // Up to 4 warps (a block's) a token: a block has 4 / split tokens at a time, `tokens` in all. More: a block
  // has one token, of which it is the (blockIdx % token_blocks)-th.
  const int64_t t0 = (int64_t)(blockIdx.x / p.token_blocks) * p.tokens;
  const int n_tokens = (int)min((int64_t)p.tokens, p.T - t0);
  const int j_step = max(1, kRopeWarps / p.split);
  const int share = p.token_blocks > 1 ? (int)(blockIdx.x % p.token_blocks) * kRopeWarps + warp : warp & (p.split - 1);
  int j = p.token_blocks > 1 ? 0 : warp / p.split;  // token of the block

  // this lane's elements of a head: four from the one place, four from the other (all lanes' first
  // four lie together, and their second four)
  const int turning = p.pairs / 4;  // lanes that turn
  const bool turns = c < turning, active = c * 8 < p.d;
  const int at_a = ADJ ? c * 8 : turns ? c * 4 : 2 * p.pairs + (c - turning) * 4;
  const int at_b = ADJ ? at_a + 4 : turns ? at_a + p.pairs : at_a + p.d / 2 - p.pairs;

  // A batch: U groups of one part's heads of one token, from group g on. The groups of both
  // parts are counted on, part 1's from `groups0`.
  const int groups0 = (p.part[0].heads + RPW - 1) / RPW, groups = groups0 + (p.part[1].heads + RPW - 1) / RPW;
  const int g1 = groups0 + (share + p.split - groups0 % p.split) % p.split;  // this warp's first group of part 1
  int g = share;
  bool more = j < n_tokens && g < groups;
  uint2 va[U], vb[U];
  auto heads_left = [&](int k) {  // of the part, from this lane's head on (0: none)
    return active ? p.part[k].heads - ((g - (k ? groups0 : 0)) * RPW + sub) : 0;
  };
  auto fetch = [&]() {
    const int k = g >= groups0;
    int64_t row = t0 + j;
    if (PAGED && p.rows) {
      row = p.rows[row];
      if (row < 0 || row >= p.n_rows) return;  // (left out below)
    }
    const uint16_t* s = p.part[k].src + row * p.part[k].ld + ((g - (k ? groups0 : 0)) * RPW + sub) * p.d;
    const int left = heads_left(k), step = p.split * RPW;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * step < left) {
        if constexpr (ADJ) {
          const uint4 x = *reinterpret_cast<const uint4*>(s + u * step * p.d + at_a);
          va[u] = make_uint2(x.x, x.y), vb[u] = make_uint2(x.z, x.w);
        } else {
          va[u] = *reinterpret_cast<const uint2*>(s + u * step * p.d + at_a);
          vb[u] = *reinterpret_cast<const uint2*>(s + u * step * p.d + at_b);
        }
      }
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) va[u] = vb[u] = make_uint2(0, 0);
  if (more) fetch();

  // this thread's first pair (beside the search for places; without one it only takes registers: 32768 tokens 119
  // us instead of 115)
  const bool early = PAGED && p.pairs > 0;
  int pair = early ? threadIdx.x % p.pairs : -1;
  float freq = early ? p.freqs[pair] : 0.f;
  uint64_t turns_by = early ? turns_per_position(freq) : 0;
  if constexpr (PAGED) {
    if (warp == 0) {
      const int t = (int)t0 + lane, first = find_sequence(p.starts, p.B, (int)t0);
      int64_t place = 0;
      int position = 0;
      bool in = lane < n_tokens && find_place(p, first, t, place, position);
      if (in && p.rows) {
        const int row = p.rows[t];
        in = row >= 0 && row < p.n_rows;
      }
      places[lane] = in ? place : -1;
      ats[lane] = position;
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < n_tokens * p.pairs; i += kRopeThreads) {
    const int jt = i / p.pairs, this_pair = i - jt * p.pairs;
    if (this_pair != pair) {  // (where the pairs do not divide the threads)
      pair = this_pair;
      freq = p.freqs[pair];
      turns_by = turns_per_position(freq);
    }
    rope_smem[i] = turn_of(p, (int)t0 + jt, pair, freq, turns_by, PAGED ? ats[jt] : 0);
  }
  __syncthreads();

  // cos and sin of this lane's pairs, times the weights: a' = a ca - b sb, b' = b cb + a sa
  float2 ca[2], cb[2], sa[2], sb[2];
  int made = -1;  // token and part that they are for
#pragma unroll 1
  while (more) {
    const int k = g >= groups0;
    const bool norm = p.part[k].weight != nullptr, turn = p.part[k].turn;
    if ((norm || turn) && made != 2 * j + k) {
      made = 2 * j + k;
      float2 wa[2], wb[2];
      wa[0] = wa[1] = wb[0] = wb[1] = make_float2(1.f, 1.f);
      if (norm && active) {
        const uint16_t* w = p.part[k].weight;
        unpack<ADJ>(*reinterpret_cast<const uint2*>(w + at_a), *reinterpret_cast<const uint2*>(w + at_b), wa, wb);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ca[i] = wa[i], cb[i] = wb[i];
        if (turns && turn) {
          const float2 x = rope_smem[j * p.pairs + c * 4 + 2 * i], y = rope_smem[j * p.pairs + c * 4 + 2 * i + 1];
          const float2 cos = make_float2(x.x, y.x), sin = make_float2(x.y, y.y);
          ca[i] = __fmul2_rn(wa[i], cos);
          cb[i] = __fmul2_rn(wb[i], cos);
          sa[i] = __fmul2_rn(wa[i], sin);
          sb[i] = __fmul2_rn(wb[i], make_float2(-sin.x, -sin.y));
        }
      }
    }
    if (norm || turn) {
      float2 a[U][2], b[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) unpack<ADJ>(va[u], vb[u], a[u], b[u]);
      if (norm) {
        float ss[U];
        bool over = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float2 s = __fmul2_rn(a[u][0], a[u][0]);
          s = __ffma2_rn(a[u][1], a[u][1], s);
          s = __ffma2_rn(b[u][0], b[u][0], s);
          s = __ffma2_rn(b[u][1], b[u][1], s);
          ss[u] = s.x + s.y;
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1)
#pragma unroll
          for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], off);
#pragma unroll
        for (int u = 0; u < U; ++u) over |= !(ss[u] <= 3.4e38f);
        float eps[U], f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) eps[u] = p.eps, f[u] = 1.f;
        if (__any_sync(0xffffffffu, over)) {  // squares past fp32: those of 2^-70 of the head
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float s = small_squares<LPR>(a[u][0], a[u][1], b[u][0], b[u][1]);
            if (!(ss[u] <= 3.4e38f)) ss[u] = s, eps[u] = 0.f, f[u] = 8.470329472543003e-22f;
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float inv = rsqrtf(fmaf(ss[u], p.inv_d, eps[u]));
          if (over) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              a[u][i] = make_float2(a[u][i].x * f[u], a[u][i].y * f[u]);
              b[u][i] = make_float2(b[u][i].x * f[u], b[u][i].y * f[u]);
            }
          }
          const float2 inv2 = make_float2(inv, inv);
#pragma unroll
          for (int i = 0; i < 2; ++i) a[u][i] = __fmul2_rn(a[u][i], inv2), b[u][i] = __fmul2_rn(b[u][i], inv2);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 x = __fmul2_rn(a[u][i], ca[i]), y = __fmul2_rn(b[u][i], cb[i]);
          if (turns && turn) x = __ffma2_rn(b[u][i], sb[i], x), y = __ffma2_rn(a[u][i], sa[i], y);
          a[u][i] = x, b[u][i] = y;
        }
        pack<ADJ>(a[u], b[u], va[u], vb[u]);
      }
    }
    const int64_t place = PAGED ? places[j] : (t0 + j) * p.part[k].ld_dst;
    if (!PAGED || place >= 0) {
      const int left = heads_left(k), step = p.split * RPW;
      const int64_t hs = PAGED ? p.head_stride : (int64_t)p.d;
      uint16_t* to = p.part[k].dst + place + ((g - (k ? groups0 : 0)) * RPW + sub) * hs;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * step < left) {
          if constexpr (ADJ) {
            *reinterpret_cast<uint4*>(to + u * step * hs + at_a) = make_uint4(va[u].x, va[u].y, vb[u].x, vb[u].y);
          } else {
            *reinterpret_cast<uint2*>(to + u * step * hs + at_a) = va[u];
            *reinterpret_cast<uint2*>(to + u * step * hs + at_b) = vb[u];
          }
        }
      }
    }
    // the next batch: of this part, the other, the next token
    g += U * p.split;
    if (!k && g >= groups0) g = g1;
    if (g >= groups) g = share, j += j_step;
    more = j < n_tokens && g < groups;
    if (more) fetch();
  }
}

template <int LPR, bool PAGED, bool ADJ>
cudaError_t rope_launch_t(RopeParams p, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / LPR;
  const int groups = (p.part[0].heads + RPW - 1) / RPW + (p.part[1].heads + RPW - 1) / RPW;
  p.inv_d = 1.f / (float)p.d;
  // Few tokens: a token's heads go to several warps, while those are at most 24 an SM, fewer than
  // run at once (32: 1003 tokens of 40 heads 7.3 us instead of 6.4): 2 or 4 of a block, or more blocks a
  // token. Many: a warp takes several tokens where they have few heads, for at least two batches of loads.
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
