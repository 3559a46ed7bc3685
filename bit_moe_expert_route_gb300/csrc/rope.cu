// Norms of each head's queries and keys, their rotation by position, and the writing of
// new keys and values to a paged cache.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pairs (a, b) of y turned by position * freq
//
// A warp takes one token's heads, or every split-th group of them: a lane holds 8
// elements (16 bytes) of a head, a head takes d / 8 lanes (rounded up to 8, 16 or 32),
// so that a warp's load is 1, 2 or 4 whole heads. The angles go by the token and the lane
// alone: a warp makes its 8 sines and cosines a lane once and keeps them in registers
// over the heads. Bound by HBM for many tokens, by one chain of load - sum - store for
// few.
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

MOE_DEVINL void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The sequence of token t: the last b with starts[b] <= t, B if that is none's; a warp
// looks at 32 places a step.
MOE_DEVINL int find_sequence(const int32_t* starts, int B, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B + 1;  // starts[lo - 1] <= t, starts[lo + n] > t
  while (n > 0) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = at < lo + n && starts[at] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // (rising: the first c lanes)
    if (c == 0) {
      n = 0;
    } else {
      const int end = lo + n;
      lo += (c - 1) * step + 1;
      n = min(step - 1, end - lo);
    }
  }
  return lo - 1;
}

template <int LPR, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr int RPW = 32 / LPR;  // heads a warp holds
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int64_t w = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t token = w / p.split;
  const int first = (int)(w - token * p.split);
  if (token >= p.T) return;
  const int t = (int)token;
  const int lane = threadIdx.x & 31, c = lane % LPR, sub = lane / LPR;
  const bool active = c * 8 < p.d;

  int64_t row = t, place = 0;  // source row; the place in the cache
  int position = 0;
  if constexpr (PAGED) {
    const int b = find_sequence(p.starts, p.B, t);
    if (b < 0 || b >= p.B) return;  // no sequence's
    const int from = p.starts[b];
    if (t < from || t >= p.starts[b + 1]) return;  // (only where starts do not rise)
    const int64_t at = (int64_t)max(p.lens[b], 0) + ((int64_t)t - from);
    const int64_t index = at >> p.page_log2;
    if (index >= p.width) return;
    const int page = p.table[b * p.ld_table + index];
    if (p.rows) row = p.rows[t];
    if (page < 0 || page >= p.n_pages || row < 0 || row >= p.n_rows) return;
    place = page * p.page_stride + (at & ((1 << p.page_log2) - 1)) * p.position_stride;
    position = (int)at;
  }

  // cos and sin of this lane's pairs (adjacent: 4, else 8; a lane of the second
  // elements has its partners' angles, with the sign of its sine)
  float cs[8], sn[8];
  const int turning = p.adjacent ? p.pairs / 4 : p.pairs / 8;  // lanes of (first) elements
  const bool second = !p.adjacent && c >= turning;
  const bool turns = c < (p.adjacent ? turning : 2 * turning);
  if (p.pairs > 0) {
    int at[MOE_ROPE_MAX_AXES] = {position, 0, 0, 0};
    if (p.positions) {
#pragma unroll
      for (int a = 0; a < MOE_ROPE_MAX_AXES; ++a)
        if (a < p.n_axes) at[a] = p.positions[a * p.ld_positions + t];
    }
    const int i0 = p.adjacent ? c * 4 : (second ? c - turning : c) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!turns || (p.adjacent && i >= 4)) {
        cs[i] = 1.f, sn[i] = 0.f;
        continue;
      }
      const int pair = i0 + i;
      int axis = 0;
      if (p.n_axes > 1) {
        if (p.cyclic) {
          axis = pair % p.n_axes;
          if (pair >= p.n_axes * (axis == 0 ? p.pairs : axis == 1 ? p.sections[1] : axis == 2 ? p.sections[2] : p.sections[3])) axis = 0;
        } else {
          axis = (pair >= p.sections[0]) + (pair >= p.sections[0] + p.sections[1]) +
                 (pair >= p.sections[0] + p.sections[1] + p.sections[2]);
        }
      }
      const int pos = axis == 0 ? at[0] : axis == 1 ? at[1] : axis == 2 ? at[2] : at[3];
      const float freq = p.freqs[pair];
      const uint64_t turn = turns_per_position(freq) * (uint64_t)(int64_t)pos;
      const int32_t left = (int32_t)(uint32_t)((turn + 0x80000000ull) >> 32);  // of a turn, in 2^-32
      sincospif((float)left * 4.656612873077393e-10f, &sn[i], &cs[i]);         // 2^-31
      const float bad = freq - freq;  // NaN for a frequency that is not finite
      cs[i] += bad;
      sn[i] = second ? sn[i] + bad : -(sn[i] + bad);
    }
  }
  const int partner = (lane & ~(LPR - 1)) + (!turns ? c : second ? c - turning : c + turning);

  const int groups0 = (p.part[0].heads + RPW - 1) / RPW, groups = groups0 + (p.part[1].heads + RPW - 1) / RPW;
  constexpr int U = 4;  // heads (or groups of them) in flight
#pragma unroll 1
  for (int g0 = first; g0 < groups; g0 += U * p.split) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * p.split, k = g < groups0 ? 0 : 1, head = (k ? g - groups0 : g) * RPW + sub;
      v[u] = make_uint4(0, 0, 0, 0);
      if (g < groups && active && head < p.part[k].heads)
        v[u] = *reinterpret_cast<const uint4*>(p.part[k].src + row * p.part[k].ld + (int64_t)head * p.d + c * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * p.split, k = g < groups0 ? 0 : 1, head = (k ? g - groups0 : g) * RPW + sub;
      if (g >= groups) break;  // (g is the warp's)
      const bool in = active && head < p.part[k].heads;
      uint4 out = v[u];
      const uint16_t* weight = p.part[k].weight;
      if (weight || p.part[k].turn) {
        float x[8];
        unpack8(v[u], x);
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          float eps = p.eps;
          const bool over = !(ss <= 3.4e38f);
          if (__any_sync(0xffffffffu, over)) {  // squares past fp32: of a row 2^-70 of this one
            float s2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float y = x[i] * 8.470329472543003e-22f;
              s2 = fmaf(y, y, s2);
              if (over) x[i] = y;
            }
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, off);
            if (over) ss = s2, eps = 0.f;
          }
          const float inv = 1.f / sqrtf(ss / (float)p.d + eps);
          float wt[8];
          uint4 wv = make_uint4(0, 0, 0, 0);
          if (active) wv = *reinterpret_cast<const uint4*>(weight + c * 8);
          unpack8(wv, wt);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wt[i];
        }
        if (p.part[k].turn) {
          if (p.adjacent) {
            if (turns) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = fmaf(b, sn[i], a * cs[i]);  // (sn is -sin)
                x[2 * i + 1] = fmaf(b, cs[i], -a * sn[i]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float other = __shfl_sync(0xffffffffu, x[i], partner);
              if (turns) x[i] = fmaf(other, sn[i], x[i] * cs[i]);
            }
          }
        }
        out = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      }
      if (in) {
        const int64_t to = PAGED ? place + head * p.head_stride : row * p.part[k].ld_dst + (int64_t)head * p.d;
        *reinterpret_cast<uint4*>(p.part[k].dst + to + c * 8) = out;
      }
    }
  }
}

template <int LPR, bool PAGED>
cudaError_t rope_launch_t(RopeParams p, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / LPR, kWarps = kRopeThreads / 32;
  const int groups = (p.part[0].heads + RPW - 1) / RPW + (p.part[1].heads + RPW - 1) / RPW;
  // Few tokens: their heads go to several warps, up to four warps a scheduler.
  p.split = (int)std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)sms * 16 / p.T));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.T * p.split + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<LPR, PAGED>, p);
}

template <bool PAGED>
cudaError_t rope_launch_p(const RopeParams& p, int sms, cudaStream_t s) {
  if (p.d <= 64) return rope_launch_t<8, PAGED>(p, sms, s);
  if (p.d <= 128) return rope_launch_t<16, PAGED>(p, sms, s);
  return rope_launch_t<32, PAGED>(p, sms, s);
}

}  // namespace

cudaError_t rope_launch(const RopeParams& p, int sms, cudaStream_t s) {
  return p.starts ? rope_launch_p<true>(p, sms, s) : rope_launch_p<false>(p, sms, s);
}

}  // namespace moe
