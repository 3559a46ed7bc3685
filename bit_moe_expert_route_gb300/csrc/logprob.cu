// Log probabilities of given tokens, entropy and top alternatives from logits,
// each logit read once.
//
//   lse = ref + log S, S = sum exp(z - ref);  logprob = z_id - lse
//   H = log S - U / S, U = sum exp(z - ref) (z - ref)
//
// Every thread keeps its own reference `ref`, sum S and weighted sum U over the
// 16-byte vectors it reads. ref starts at the largest logit of the thread's
// first vectors and moves only when a logit passes it by more than kLazy: sums
// of fp32 need no nearer reference, and the rescale is almost never taken. The
// row's sums are moved to the largest logit at the end, where neither
// difference cancels. z - ref is taken in natural units before the
// multiplication by log2 e, so that large logits lose nothing to the
// constant's rounding. bf16 logits enter a mixed-precision add as they are, and
// two elements at a time go through the packed fp32 multiply, add and fused
// multiply-add: about four instructions an element with its ex2.
//
// Top k (k <= 32): a warp holds its best 32 in order, one a lane, and inserts
// what reaches the block's threshold, a lower bound of the row's k-th best. It
// starts from the thread maxima of the block's first pass, so that only a few
// elements a pass ever reach the insertion. Ties go to the lower index: entries
// are 64-bit keys (value in order, then the index reversed), and an element
// equal to the threshold is still inserted.
//
// Many rows: one block a row (short rows: one warp). Few rows: a cluster of 2, 4
// or 8 blocks shares a row and the first block merges their states from
// distributed shared memory, so one launch suffices at every size.
//
// 2048 rows of 131072 bf16 logits: 84 us without alternatives (6.4 TB/s, 94% of
// the measured copy), 95 with 8, 125 with 32; bound by HBM, then by instruction
// issue (72% active with 8). 48 rows of 100003 fp32 logits with 20: 17.5 us, of
// which 8 without alternatives: the merges' and insertions' latency.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kLpWarps = 8;
constexpr int kLpThreads = 32 * kLpWarps;
constexpr float kLazy = 20.f;  // e^20: fp32 sums hold it easily
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;


// The order of a logit among the top alternatives: larger value, larger rank;
// NaN below every number (rank 1), 0 = no element.
MOE_DEVINL uint32_t rank_of(float z) { return z != z ? 1u : order_key(z); }
MOE_DEVINL uint64_t key_of(float z, int index) {
  return ((uint64_t)rank_of(z) << 32) | (uint32_t)(~index);
}

// A thread's sums over its elements.
struct Sums {
  float ref, S, U;  // S = sum exp(z - ref), U = sum exp(z - ref) (z - ref)
  float top;        // the largest logit (NaN if one is)
};

// Moves (S, U) to another reference (both finite).
MOE_DEVINL void rebase(Sums& s, float ref) {
  const float d = s.ref - ref, f = exp2f(d * kLog2e);
  // e (z - ref') = f e_old ((z - ref) + d); f = 0 far below leaves nothing
  s.U = f > 0.f ? f * fmaf(s.S, d, s.U) : 0.f * s.U;
  s.S *= f;
  s.ref = ref;
}
MOE_DEVINL void merge(Sums& a, Sums b) {
  const float ref = fmaxf(a.ref, b.ref);
  rebase(a, ref);
  rebase(b, ref);
  a.S += b.S;
  a.U += b.U;
  a.top = max_nan(a.top, b.top);
}

// The best 32 of two descending lists of 32 (one entry a lane), descending.
MOE_DEVINL uint64_t merge32(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = a > r ? a : r;  // the upper half of a bitonic sequence
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, a, off);
    const bool upper = (lane & off) == 0;
    a = (a > o) == upper ? a : o;
  }
  return a;
}
// 32 values (one a lane) into descending order.
MOE_DEVINL uint32_t sort32(uint32_t a, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int off = size / 2; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, a, off);
      const bool keep_max = ((lane & off) == 0) == ((lane & size) == 0);
      a = keep_max ? max(a, o) : min(a, o);
    }
  return a;
}

// Elements of a 16-byte vector.
template <bool F32>
constexpr int kVecElems = F32 ? 4 : 8;
template <bool F32>
MOE_DEVINL uint4 none_vec() {  // -infinity throughout
  constexpr uint32_t w = F32 ? 0xFF800000u : 0xFF80FF80u;
  return make_uint4(w, w, w, w);
}

// The vector of the row's elements first .. first + E - 1 (16-byte aligned);
// those outside [0, V) as -infinity. A vector inside is one 16-byte load.
template <bool F32>
MOE_DEVINL uint4 load_vec(const void* row, int64_t first, int V) {
  constexpr int E = kVecElems<F32>;
  const float* f = static_cast<const float*>(row);
  const uint16_t* h = static_cast<const uint16_t*>(row);
  if (first >= 0 && first + E <= V) {
    if constexpr (F32) return __ldg(reinterpret_cast<const uint4*>(f + first));
    return __ldg(reinterpret_cast<const uint4*>(h + first));
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F32) {
      w[i] = first + i >= 0 && first + i < V ? __float_as_uint(f[first + i]) : 0xFF800000u;
    } else {
      const int64_t a = first + 2 * i, b = a + 1;
      const uint32_t x = a >= 0 && a < V ? h[a] : 0xFF80u;
      const uint32_t y = b >= 0 && b < V ? h[b] : 0xFF80u;
      w[i] = x | (y << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kUnroll = 4;  // vectors a thread holds at a time

// The largest element of the thread's vectors (NaN if one is).
template <bool F32, int N>
MOE_DEVINL float largest(const uint4* v) {
  if constexpr (F32) {
    float m = __uint_as_float(v[0].x);
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = max_nan(max_nan(m, max_nan(__uint_as_float(v[i].x), __uint_as_float(v[i].y))),
                  max_nan(__uint_as_float(v[i].z), __uint_as_float(v[i].w)));
    return m;
  } else {
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(v);
    __nv_bfloat162 m = b[0];
#pragma unroll
    for (int i = 1; i < 4 * N; ++i) m = __hmax2_nan(m, b[i]);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
    return max_nan(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
}

// z - ref of a vector's elements. bf16 logits go through the mixed-precision
// add, which takes them from their half of the word as they are.
template <bool F32>
MOE_DEVINL void distances(const uint4& v, float nref, float2 (&d)[kVecElems<F32> / 2]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      d[i] = __fadd2_rn(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), make_float2(nref, nref));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
          "add.rn.f32.bf16 %0, lo, %3;\n\tadd.rn.f32.bf16 %1, hi, %3;\n\t}"
          : "=f"(d[i].x), "=f"(d[i].y)
          : "r"(u[i]), "f"(nref));
  }
}

// Adds the thread's vectors, whose largest element is m.
template <bool F32>
MOE_DEVINL void add_vecs(Sums& s, const uint4 (&v)[kUnroll], float m) {
  constexpr int E = kVecElems<F32>;
  s.top = max_nan(s.top, m);
  if (m > s.ref + kLazy) rebase(s, m);  // (+infinity ends as NaN, as it should)
  const float2 c = make_float2(kLog2e, kLog2e);
  float2 S[2] = {}, U[2] = {};
#pragma unroll
  for (int k = 0; k < kUnroll; ++k) {
    float2 d[E / 2];
    distances<F32>(v[k], -s.ref, d);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 x = __fmul2_rn(d[i], c);
      const float2 e = make_float2(ex2(x.x), ex2(x.y));
      S[i & 1] = __fadd2_rn(S[i & 1], e);
      U[i & 1] = __ffma2_rn(e, d[i], U[i & 1]);
    }
  }
  s.S += (S[0].x + S[0].y) + (S[1].x + S[1].y);
  float u = (U[0].x + U[0].y) + (U[1].x + U[1].y);
  if (u != u) {  // -infinity among them (0 * infinity): its weight is 0, and so is 0 * (a finite distance)
    u = 0.f;
#pragma unroll 1
    for (int k = 0; k < kUnroll; ++k) {
      uint4 w = v[0];
#pragma unroll
      for (int q = 1; q < kUnroll; ++q) w = q == k ? v[q] : w;
      float2 d[E / 2];
      distances<F32>(w, -s.ref, d);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        u = fmaf(ex2(d[i].x * kLog2e), max_nan(d[i].x, kLowest), u);
        u = fmaf(ex2(d[i].y * kLog2e), max_nan(d[i].y, kLowest), u);
      }
    }
  }
  s.U += u;
}

struct LpShared {
  uint64_t list[kLpWarps][32];
  Sums sums[kLpWarps];
  uint64_t row_list[32];  // the block's results, read by the cluster's first block
  Sums row_sums;
  uint4 scratch[kLpWarps][kUnroll];  // a lane's vectors, looked at by its warp
  uint32_t kth[kLpWarps], qth[kLpWarps];  // the ranks of each warp's k-th and q-th best so far
};

// The best 32 of n lists in shared memory (n a power of two <= 8) into
// list[0]: halving, one warp a pair. The whole block calls it.
MOE_DEVINL void merge_lists(uint64_t (*list)[32], int n, int warp, int lane) {
  for (; n > 1; n >>= 1) {
    __syncthreads();
    if (warp < n / 2) list[warp][lane] = merge32(list[warp][lane], list[warp + n / 2][lane], lane);
  }
  __syncthreads();
}

MOE_DEVINL float remote_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Sums of the first n lanes, joined in every lane (n a power of two).
MOE_DEVINL void join_lanes(Sums& s, int n) {
  for (int off = n / 2; off > 0; off >>= 1) {
    Sums o;
    o.ref = __shfl_xor_sync(0xffffffffu, s.ref, off);
    o.S = __shfl_xor_sync(0xffffffffu, s.S, off);
    o.U = __shfl_xor_sync(0xffffffffu, s.U, off);
    o.top = __shfl_xor_sync(0xffffffffu, s.top, off);
    merge(s, o);
  }
}

// W warps a row: 8 (a block's, or a cluster's of such blocks), or 1 (eight rows
// a block, with no barrier).
template <bool F32, bool TOP, int W>
__global__ void __launch_bounds__(kLpThreads, 4) logprob_kernel(const LogprobParams p) {
  constexpr int E = kVecElems<F32>, T = 32 * W;
  __shared__ LpShared sh;
  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = W == 1 ? 0 : warp, tid = wr * 32 + lane;  // in the row
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * kLpWarps + warp : blockIdx.x / ranks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (W == 1 && row >= p.N) return;
  const char* base = static_cast<const char*>(p.logits) + row * p.ld * (F32 ? 4 : 2);
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15) / (F32 ? 4 : 2));
  // the row's vectors, the first one starting `lead` elements before it, in
  // contiguous parts for the cluster's blocks
  const int nvec = (lead + p.V + E - 1) / E, part = (nvec + (int)ranks - 1) / (int)ranks;
  const int v0 = (int)rank * part, v1 = min(nvec, v0 + part);
  Sums s;
  s.ref = kLowest;
  s.S = 0.f;
  s.U = 0.f;
  s.top = -INFINITY;
  uint64_t mine = 0;  // this lane's entry of the warp's list, 0 = none
  uint32_t bar = 0;   // the rank that an element has to reach, and its value
  float bar_z = -INFINITY;
  // Two bounds of the row's k-th best from below, which need no list but a
  // warp's own and may be read while others raise theirs: any warp's k-th best
  // (near for small k), and, with n warps' q-th best places, q n >= k, the least
  // of those (near for large k). n counts warps whose lanes all have elements.
  const int full = W == 1 ? 1 : min(W, max(1, (v1 - v0) / 32)), q = TOP ? (p.k + full - 1) / full : 1;
  auto shared_bar = [&]() {
    const int w = lane & (W - 1);
    const uint32_t kth = *reinterpret_cast<volatile uint32_t*>(&sh.kth[w]), qth = *reinterpret_cast<volatile uint32_t*>(&sh.qth[w]);
    return max(__reduce_max_sync(0xffffffffu, kth), __reduce_min_sync(0xffffffffu, w < full ? qth : 0xFFFFFFFFu));
  };
  // vectors [in0, in1) lie inside the row: a pass of only those is plain loads
  const int in0 = lead ? 1 : 0, in1 = (lead + p.V) / E;
  const uint4* vecs = reinterpret_cast<const uint4*>(base - lead * (F32 ? 4 : 2));
  auto load = [&](int v, uint4 (&w)[kUnroll]) {
    if (v >= in0 && v + kUnroll * T <= min(v1, in1)) {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) w[i] = __ldg(vecs + v + tid + i * T);
    } else {
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int vi = v + i * T + tid;
        w[i] = vi < v1 ? load_vec<F32>(base, (int64_t)vi * E - lead, p.V) : none_vec<F32>();
      }
    }
  };
  uint4 w[kUnroll];
  load(v0, w);
#pragma unroll 1
  for (int v = v0; v < v1; v += kUnroll * T) {
    uint4 next[kUnroll];
    load(v + kUnroll * T, next);  // in flight while these are summed
    const float m = largest<F32, kUnroll>(w);
    if (v == v0) {
      s.ref = fminf(fmaxf(m, kLowest), -kLowest);  // (NaN: the lowest)
      if (TOP) {
        // the k-th largest of the threads' maxima bounds the k-th largest element
        // from below. A thread without elements counts as nothing (rank 0).
        const uint32_t sorted = sort32(v + tid < v1 ? rank_of(m) : 0u, lane);
        if constexpr (W == 1) {
          bar = __shfl_sync(0xffffffffu, sorted, p.k - 1);
        } else {
          sh.list[warp][lane] = ((uint64_t)sorted << 32);
          merge_lists(sh.list, kLpWarps, warp, lane);
          bar = (uint32_t)(sh.list[0][p.k - 1] >> 32);
          if (lane == 0) sh.kth[warp] = sh.qth[warp] = bar;
          __syncthreads();
        }
        bar_z = bar > 1 ? key_value(bar) : -INFINITY;
      }
    }
    add_vecs<F32>(s, w, m);
    // (a NaN hides the other elements: those are looked at)
    if (TOP && __any_sync(0xffffffffu, !(m < bar_z))) {
      if (W > 1) bar = max(bar, shared_bar());
      unsigned hit = __ballot_sync(0xffffffffu, m != m || rank_of(m) >= bar);
      while (hit) {  // one lane's vectors at a time, through shared memory: an element a lane
        const int src = __ffs(hit) - 1;
        hit &= hit - 1;
        if (lane == src) {
#pragma unroll
          for (int i = 0; i < kUnroll; ++i) sh.scratch[warp][i] = w[i];
        }
        __syncwarp();
        const int vi = v + (lane / E) * T + wr * 32 + src;
        const int64_t index = (int64_t)vi * E - lead + lane % E;
        uint64_t key = 0;
        if (lane < kUnroll * E && vi < v1 && index >= 0 && index < p.V) {
          const float z = F32 ? reinterpret_cast<const float*>(sh.scratch[warp])[lane & 15]
                              : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(sh.scratch[warp])[lane]);
          key = key_of(z, (int)index);
        }
        unsigned todo = __ballot_sync(0xffffffffu, key != 0 && (uint32_t)(key >> 32) >= bar);
        while (todo) {
          const uint64_t c = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
          todo &= todo - 1;
          const int at = __popc(__ballot_sync(0xffffffffu, mine > c));  // entries above it
          const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
          if (lane == at) mine = c;
          else if (lane > at) mine = up;
        }
      }
      // the warp's own places may raise the threshold
      const uint32_t place = (uint32_t)(mine >> 32);
      bar = max(bar, __shfl_sync(0xffffffffu, place, p.k - 1));
      if constexpr (W > 1) {
        if (lane == q - 1 && place > sh.qth[warp]) *reinterpret_cast<volatile uint32_t*>(&sh.qth[warp]) = place;
        if (lane == p.k - 1 && place > sh.kth[warp]) *reinterpret_cast<volatile uint32_t*>(&sh.kth[warp]) = place;
      }
      bar_z = bar > 1 ? key_value(bar) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) w[i] = next[i];
  }
  join_lanes(s, 32);
  uint64_t best = mine;  // lane i: the row's i-th
  if constexpr (W > 1) {
    // the block's sums and list, in warp 0
    if (lane == 0) sh.sums[warp] = s;
    if (TOP) {
      sh.list[warp][lane] = mine;
      merge_lists(sh.list, kLpWarps, warp, lane);
    } else {
      __syncthreads();
    }
    if (warp == 0) {
      s = sh.sums[lane & (kLpWarps - 1)];
      join_lanes(s, kLpWarps);
      if (TOP) best = sh.list[0][lane];
    }
    if (ranks > 1) {
      if (warp == 0) {
        if (lane == 0) sh.row_sums = s;
        if (TOP) sh.row_list[lane] = best;
      }
      cluster_sync();
      if (rank == 0) {
        if (TOP) {
          if (warp < (int)ranks) {
            uint64_t e;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(e) : "r"(remote_addr(&sh.row_list[lane], warp)) : "memory");
            sh.list[warp][lane] = e;
          }
          merge_lists(sh.list, (int)ranks, warp, lane);
        }
        if (warp == 0) {
          const uint32_t a = remote_addr(&sh.row_sums, lane & (ranks - 1));
          s.ref = remote_f32(a);
          s.S = remote_f32(a + 4);
          s.U = remote_f32(a + 8);
          s.top = remote_f32(a + 12);
          join_lanes(s, (int)ranks);
          if (TOP) best = sh.list[0][lane];
        }
      }
      cluster_sync();  // the other blocks' shared memory stays until the first has read it
      if (rank != 0) return;
    }
    if (warp != 0) return;
  }
  const bool none = s.top == -INFINITY;   // nothing but -infinity
  const bool bad = !(s.top <= -kLowest);  // +infinity or NaN
  const float nan = __int_as_float(0x7fc00000);
  if (!bad && !none) rebase(s, s.top);
  const float logS = logf(s.S);
  auto log_p = [&](float z) {
    if (bad) return nan;
    return none || z == -INFINITY ? -INFINITY : (z - s.ref) - logS;
  };
  if (lane == 0 && p.logprob) {
    const int id = p.ids[row];
    float lp = nan;
    if (id >= 0 && id < p.V)
      lp = log_p(F32 ? reinterpret_cast<const float*>(base)[id]
                     : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(base)[id]));
    p.logprob[row] = lp;
  }
  if (lane == 1 && p.entropy) p.entropy[row] = bad ? nan : none ? 0.f : fmaxf(logS - s.U / s.S, 0.f);
  if (TOP && lane < p.k) {
    p.top_ids[row * p.k + lane] = (int)~(uint32_t)best;
    p.top_logprobs[row * p.k + lane] = log_p(key_value((uint32_t)(best >> 32)));
  }
}

template <bool F32, bool TOP, int W>
cudaError_t logprob_launch_t(const LogprobParams& p, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(W == 1 ? ((int64_t)p.N + kLpWarps - 1) / kLpWarps : (int64_t)p.N * cluster));
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<F32, TOP, W>, p);
}
template <bool F32>
cudaError_t logprob_launch_w(const LogprobParams& p, bool warp_rows, int cluster, cudaStream_t s) {
  if (warp_rows) return p.k ? logprob_launch_t<F32, true, 1>(p, 1, s) : logprob_launch_t<F32, false, 1>(p, 1, s);
  return p.k ? logprob_launch_t<F32, true, 8>(p, cluster, s) : logprob_launch_t<F32, false, 8>(p, cluster, s);
}

}  // namespace

cudaError_t logprob_launch(const LogprobParams& p, int sms, cudaStream_t s) {
  // Short rows: a warp each, of one pass over its lanes' vectors, or of up to
  // eight where there are rows enough for every multiprocessor's warps.
  const int64_t pass = (int64_t)32 * kUnroll * (p.f32 ? 4 : 8);
  const bool warp_rows = p.V <= pass || (p.V <= 8 * pass && (int64_t)p.N >= (int64_t)sms * 16);
  // Else a block each, or more while the grid leaves multiprocessors short of 4
  // blocks and each block keeps two vectors a thread.
  int cluster = 1;
  while (cluster < 8 && (int64_t)p.N * cluster * 2 <= (int64_t)sms * 4 && p.V >= cluster * 2 * 4 * pass) cluster *= 2;
  return p.f32 ? logprob_launch_w<true>(p, warp_rows, cluster, s) : logprob_launch_w<false>(p, warp_rows, cluster, s);
}

}  // namespace moe
