// Residual addition, root-mean-square norm and an 8-bit output with a scale
// per token, in one pass over the row.
//
//   r = bf16(x + residual), u = r w, a = max |u|, rms = sqrt(mean r^2 + eps)
//   q = round(u top / a), scale = a / (top rms)      (top = 127 or 448)
//
// The root mean square cancels out of q: only the scale needs it, so one
// reduction carries both the largest |u| and the sum of squares, and the
// codes follow from values that stayed in registers. u is a product of two
// bf16 values, exact in fp32; u * (top / a) in fp32 is within 3 * 2^-24 of the
// exact quotient (relative), so only a quotient that near a rounding border is
// compared with it exactly: every code is the correctly rounded one. (Products of a
// row whose a is below 2^-80 may fall below fp32's normal range, and top / a may
// pass it: such a row finds its a again with exponents apart, and its quotients from
// products lifted by a's exponent.)
//
// Bound by HBM: 7 bytes an element (x, residual in; residual, q out), 9 with
// the bf16 values: 32768 rows of 2048 in 93 us with the values, 6.5 TB/s (95% of
// the measured copy). A row belongs to G threads of NV 16-byte vectors each,
// whole warps, joined by one barrier.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kNormThreads = 256;  // a block's threads where a row needs no more

MOE_DEVINL void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Adding this and taking it away rounds |t| < 2^22 to a whole number (its low
// byte, in two's complement, ends in the sum's), or |t| < 2^13 to a multiple
// of 2^-9 (the spacing of e4m3 below 2^-6).
constexpr float kRoundInt = 12582912.f;  // 1.5 * 2^23
constexpr float kRoundSub = 24576.f;     // 1.5 * 2^14

// Whether the fp32 quotient t may round to another code than the exact one
// (its error is below 3 * 2^-24 |t|). True for a NaN.
MOE_DEVINL bool near_border_int8(float t) {
  const float n = (t + kRoundInt) - kRoundInt;
  return !(fabsf(t - n) < 0.5f - 4e-5f);  // |t| <= 127: error below 2.4e-5
}
MOE_DEVINL bool near_border_e4m3(float t) {
  // normal values keep 3 of the 23 fraction bits: near when the other 20 are
  // within 8 of half
  const bool cut = ((__float_as_uint(t) & 0xFFFFFu) - 0x7FFF8u) <= 16u;
  const float n = (t + kRoundSub) - kRoundSub;
  const bool sub = !(fabsf(t - n) < 0x1p-10f - 1e-8f);
  return fabsf(t) >= 0x1p-6f ? cut : sub;
}

// Rows whose a is below this are done with exponents apart.
constexpr float kTiny = 0x1p-80f;

// |f w| as a whole number that rises with it: its exponent, then the 15 bits after
// the leading one (a product of two bf16 values has 16 bits). 0 for 0.
MOE_DEVINL uint32_t product_key(float f, float w) {
  int ef, ew, ep;
  const float p = frexpf(fabsf(frexpf(f, &ef) * frexpf(w, &ew)), &ep);  // exact, in [1/2, 1)
  return p > 0.f ? (uint32_t)(ef + ew + ep + 512) << 15 | ((uint32_t)(p * 65536.f) - 32768u) : 0u;
}
MOE_DEVINL int key_exponent(uint32_t key) { return (int)(key >> 15) - 512; }
MOE_DEVINL float key_fraction(uint32_t key) { return (float)((key & 32767u) + 32768u) * 0x1p-16f; }
// The products f w 2^-exponent of a vector.
struct Products8 {
  float u[8];
};
__device__ __noinline__ Products8 lifted(uint4 r, uint4 weight, int exponent) {
  float f[8], w[8];
  unpack8(r, f);
  unpack8(weight, w);
  Products8 c;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int ef, ew;
    const float p = frexpf(f[e], &ef) * frexpf(w[e], &ew);
    c.u[e] = ldexpf(p, ef + ew - exponent);
  }
  return c;
}
// The largest product_key of a vector.
__device__ __noinline__ uint32_t largest_key(uint4 r, uint4 weight) {
  float f[8], w[8];
  unpack8(r, f);
  unpack8(weight, w);
  uint32_t key = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) key = max(key, product_key(f[e], w[e]));
  return key;
}

// A vector with a quotient near a border: the quotients moved to the border's
// right side (or onto it: a tie). u and a have 16 significant bits, so
// top |u| and border * a (borders have 8 bits at most) are exact in fp32 and
// their comparison is the exact quotient's with the border. Out of line, for
// the instruction cache: it is rarely taken.
// (exponent < 0: a tiny row, whose a and products are lifted by 2^-exponent. a = 0: no quotients.)
struct Quotients8 {
  float t[8];
};
template <bool E4M3>
__device__ __noinline__ Quotients8 settle(uint4 r, uint4 weight, float a, int exponent) {
  constexpr float kTop = E4M3 ? 448.f : 127.f;
  // far from fp32's ends, by an exact factor: neither product overflows or loses bits
  const float lift = exponent < 0 ? 1.f : a < 1e-20f ? 0x1p64f : a > 1e20f ? 0x1p-64f : 1.f, al = a * lift;
  Products8 c;
  if (exponent < 0) {  // (a lifted product that is rounded, below 2^-126, is far below any code's border)
    c = lifted(r, weight, exponent);
  } else {
    float f[8], w[8];
    unpack8(r, f);
    unpack8(weight, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) c.u[e] = f[e] * w[e] * lift;
  }
  Quotients8 q;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float u = c.u[e];
    float t = a > 0.f ? u * (kTop / al) : 0.f;
    if (a > 0.f && (E4M3 ? near_border_e4m3(t) : near_border_int8(t))) {
      const float b = fabsf(t);
      float border, below, above;  // the border and values that round to either side of it
      if (!E4M3 || b < 0x1p-6f) {
        const float unit = E4M3 ? 0x1p-9f : 1.f;
        below = floorf(b / unit) * unit;
        above = below + unit;
        border = below + 0.5f * unit;
      } else {
        const uint32_t mid = (__float_as_uint(b) & ~0xFFFFFu) | 0x80000u;
        border = __uint_as_float(mid);
        below = __uint_as_float(mid - 1);
        above = __uint_as_float(mid + 1);
      }
      const float exact = kTop * fabsf(u), at = border * al;
      t = copysignf(exact < at ? below : exact > at ? above : border, t);
    }
    q.t[e] = t;
  }
  return q;
}

// A barrier of row `sub`'s G threads, G > 32: at most four rows a block. (A barrier
// number that is not a constant would reserve all 16 for the block, and four blocks
// would fill an SM: 32768 rows of 2048 118 us against 106.)
static_assert(kNormThreads / 64 <= 4, "a constant for each row");
MOE_DEVINL void row_barrier(int sub, int G) {
  if (sub == 0) asm volatile("bar.sync 1, %0;" ::"r"(G) : "memory");
  if (sub == 1) asm volatile("bar.sync 2, %0;" ::"r"(G) : "memory");
  if (sub == 2) asm volatile("bar.sync 3, %0;" ::"r"(G) : "memory");
  if (sub == 3) asm volatile("bar.sync 4, %0;" ::"r"(G) : "memory");
}

template <int NV, bool E4M3>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p, int G) {
  // G threads a row (whole warps), blockDim / G rows a block
  const int sub = threadIdx.x / G, lt = threadIdx.x % G;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / G) + sub;
  const int nvec = p.d / 8;
  const bool live = row < p.T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  uint4 r[NV];
  const int64_t base = row * p.d;
  float ss = 0.f, a = 0.f;
  if (live) {
    const uint16_t* xr = p.x + row * p.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lt + i * G;
      r[i] = v < nvec ? *reinterpret_cast<const uint4*>(xr + 8 * v) : make_uint4(0, 0, 0, 0);
    }
    if (p.residual) {
      uint4 s[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lt + i * G;
        s[i] = v < nvec ? *reinterpret_cast<const uint4*>(p.residual + base + 8 * v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[8], g[8];
        unpack8(r[i], f);
        unpack8(s[i], g);
        r[i] = make_uint4(pack_bf16(f[0] + g[0], f[1] + g[1]), pack_bf16(f[2] + g[2], f[3] + g[3]),
                          pack_bf16(f[4] + g[4], f[5] + g[5]), pack_bf16(f[6] + g[6], f[7] + g[7]));
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lt + i * G;
      if (v < nvec) {
        if (p.residual_out) *reinterpret_cast<uint4*>(p.residual_out + base + 8 * v) = r[i];
        float f[8], w[8], s8 = 0.f;
        unpack8(r[i], f);
        unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight) + v), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s8 = fmaf(f[e], f[e], s8);
          a = max_nan(a, fabsf(f[e] * w[e]));
        }
        ss += s8;
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, off);
    a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, off));
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, first = sub * (G / 32);
  if (G > 32) {  // the same for the whole block: every thread takes the barrier
    __shared__ float sh[2][32];
    if (lane == 0) {
      sh[0][warp] = ss;
      sh[1][warp] = a;
    }
    __syncthreads();
    ss = 0.f;
    a = 0.f;
    for (int w = first; w < first + G / 32; ++w) {
      ss += sh[0][w];
      a = max_nan(a, sh[1][w]);
    }
  }
  int exponent = 0;  // of a tiny row (< 0): its a is a 2^exponent from here on
  if (a < kTiny) {  // (the same for the row's threads; rows past the end take it too)
    uint32_t key = 0;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lt + i * G;
        if (v < nvec) key = max(key, largest_key(r[i], __ldg(reinterpret_cast<const uint4*>(p.weight) + v)));
      }
    }
    key = __reduce_max_sync(0xffffffffu, key);
    if (G > 32) {
      __shared__ uint32_t sh_key[32];
      if (lane == 0) sh_key[warp] = key;
      row_barrier(sub, G);
      for (int w = first; w < first + G / 32; ++w) key = max(key, sh_key[w]);
    }
    a = key ? key_fraction(key) : 0.f;
    exponent = key_exponent(key);
  }
  if (!live) return;
  constexpr float kTop = E4M3 ? 448.f : 127.f, kMax = 3.402823466e38f;
  const float nan = __int_as_float(0x7fc00000);
  // a NaN or an infinity in the row shows in the sum of squares, one in the
  // products (a weight's, or an overflow) in a
  const bool fine = ss <= kMax && a <= kMax;
  float scale = fine ? a / kTop / sqrtf(ss / (float)p.d + p.eps) : nan;
  if (exponent < 0) scale = ldexpf(scale, exponent);
  if (lt == 0) p.scale[row] = scale;
  // Rows without a usable fp32 quotient (zeros, values that are not finite,
  // and tiny rows) are settled apart, as NaNs.
  if (!fine) a = 0.f;
  const float inv = exponent == 0 && a > 0.f ? kTop / a : nan;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = lt + i * G;
    if (v < nvec) {
      float f[8], w[8], t[8];
      const uint4 weight = __ldg(reinterpret_cast<const uint4*>(p.weight) + v);
      unpack8(r[i], f);
      unpack8(weight, w);
      bool near = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[e] = (f[e] * w[e]) * inv;
        near |= E4M3 ? near_border_e4m3(t[e]) : near_border_int8(t[e]);
      }
      if (near) {
        const Quotients8 c = settle<E4M3>(r[i], weight, a, exponent);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = c.t[e];
      }
      uint32_t word[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (E4M3) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * h], t[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * h + 2], t[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
          word[h] = lo | (hi << 16);
        } else {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float s = t[4 * h + e] + kRoundInt;
            b[e] = __float_as_uint(s);
            t[4 * h + e] = s - kRoundInt;
          }
          word[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
      }
      *reinterpret_cast<uint2*>(p.q + base + 8 * v) = make_uint2(word[0], word[1]);
      if (p.values) {
        if constexpr (E4M3) {  // what the codes stand for
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
            const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            t[2 * h] = v2.x;
            t[2 * h + 1] = v2.y;
          }
        }
        *reinterpret_cast<uint4*>(p.values + base + 8 * v) =
            make_uint4(pack_bf16(t[0] * scale, t[1] * scale), pack_bf16(t[2] * scale, t[3] * scale),
                       pack_bf16(t[4] * scale, t[5] * scale), pack_bf16(t[6] * scale, t[7] * scale));
      }
    }
  }
}

template <int NV, bool E4M3>
cudaError_t norm_launch_nv(const NormParams& p, cudaStream_t s) {
  const int G = ((p.d / 8 + NV - 1) / NV + 31) / 32 * 32;  // a row's threads: whole warps, at most 1024
  const int rows = G < kNormThreads ? kNormThreads / G : 1, threads = rows * G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + (int64_t)rows - 1) / rows));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_kernel<NV, E4M3>, p, G);
}

}  // namespace

cudaError_t norm_launch(const NormParams& p, int sms, cudaStream_t s) {
  const int nvec = p.d / 8;
  // Two vectors a thread: 32768 rows of 2048 with bf16 values take 94 us, against
  // 105 with four and 118 with eight (fewer warps fit, and each keeps fewer rows'
  // phases apart). One where the rows are few, for latency.
  if ((int64_t)p.T * ((nvec + 1) / 2) < (int64_t)sms * 512 && nvec <= 1024)
    return p.e4m3 ? norm_launch_nv<1, true>(p, s) : norm_launch_nv<1, false>(p, s);
  return p.e4m3 ? norm_launch_nv<2, true>(p, s) : norm_launch_nv<2, false>(p, s);
}

}  // namespace moe
