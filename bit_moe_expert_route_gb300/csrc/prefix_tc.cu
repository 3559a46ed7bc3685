// Attention over a shared prefix for many query rows (more than 32 a KV head):
// the partial states of prefix.cu from tcgen05 products.
//
// A CTA takes one KV head, 128 query rows and one slice of the prefix. Per tile
// of KT keys:  S = Q K^T (both in shared memory) into tensor memory; softmax
// weights P = 2^(scale S - m) from there into the same columns of tensor memory
// as bf16; O += P V with P as the MMA's A operand and O kept in tensor memory
// through the slice. One thread issues the scores' products, another the
// outputs', three tiles behind at most, so the tensor core works while the softmax
// warps do (with two tiles' columns 64 sequences over 32768 positions, 2 KV heads
// of 256, took 49.5 us, with three 44.6).
//
// K and V tiles come by TMA into one ring of slots in the order in which the
// products use them (K0 K1 V0 K2 V1 ...); V is read as it lies (MN-major
// operand, no transpose). Every query row of a KV head's sequences shares
// these tiles. At head size 256 with 512 rows a tile of 64 keys takes 1.1 us
// (about 2050 cycles), 1824 of them the MMAs' (16 of N = 64 at their least time
// of 50, 8 of N = 256 at 128). Few rows and a long prefix are bound by HBM: 128
// rows, 8 KV heads of 128, 131072 positions in 91 us, 5.9 TB/s. (Asking L2 for
// tiles ahead of the ring made it a third more.)
//
// The weights enter the second product as two bf16 parts, as in prefix.cu: one
// part alone carries its roundings to the output, as much again as the output's
// own (2.3e-3 of the 2-norm in all, against 1.7e-3), and its weights do not sum to
// l. That costs 64 sequences over 32768 positions, 2 KV heads of 256, 39.3 -> 44.6
// us, 8 KV heads of 128 (4 query heads each) 36.3 -> 48.1.
//
// The reference m moves only when a score passes it by 2^8; then the warp waits
// for the products before and rescales its rows of O in tensor memory.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTcRows = 128;
constexpr int kTcThreads = 256;  // warp 0 TMA, warps 1 and 2 MMA, warp 3 the ticket, warps 4-7 softmax
constexpr float kLazyLog2 = 8.f;

template <int D>
struct TcCfg {
  static constexpr int KT = D == 256 ? 64 : 128;    // keys a tile
  static constexpr int kSlot = KT * D * 2;          // K or V of a tile
  static constexpr int kSlots = D == 256 ? 5 : D == 128 ? 6 : 8;
  static constexpr int kQ = kTcRows * D * 2;
  static constexpr int kBufs = 3;                   // tiles between their scores and their outputs
  static constexpr int kOffSlots = kQ;
  static constexpr int kOffBar = kOffSlots + kSlots * kSlot;
  static constexpr int kBars = 2 * kSlots + 1 + 3 * kBufs + 1;
  static constexpr int kSmem = kOffBar + 8 * kBars + 16 + 1024;
  // tensor memory: O, then the score buffers; a tile's weights take the columns of
  // its scores (two bf16 a column: the first parts, then the second)
  static constexpr int kColS = D;
  static_assert(kColS + kBufs * KT <= 512, "tensor memory exceeded");
  static_assert(kSmem <= 232448, "shared memory exceeded");
  static_assert(kTcRows * (D * 4 + 16) <= kSlots * kSlot, "the output's rows do not fit the ring");
};

struct TcArgs {
  CUtensorMap tm_k, tm_v;  // [P][Hkv d], box 64 x KT
  PrefixParams p;
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) prefix_tc_kernel(const __grid_constant__ TcArgs args) {
  using C = TcCfg<D>;
  constexpr int KT = C::KT, NS = C::kSlots, NB = C::kBufs;
  const PrefixParams& p = args.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [NS] a slot's tile has landed
  uint64_t* empty = full + NS;                                      // [NS] its products are done
  uint64_t* q_full = empty + NS;                                    // [1]
  uint64_t* s_full = q_full + 1;                                    // [NB] scores are complete
  uint64_t* p_full = s_full + NB;                                   // [NB] weights are written, over the scores
  uint64_t* pv_done = p_full + NB;                                  // [NB] their product is complete: the columns are free
  uint64_t* drain = pv_done + NB;                                   // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, R = p.B * G, tiles = (R + kTcRows - 1) / kTcRows;
  const int h = blockIdx.x % p.Hkv, tile = (blockIdx.x / p.Hkv) % tiles, split = blockIdx.x / (p.Hkv * tiles);
  const int row0 = tile * kTcRows, k0 = split * p.prefix_slice, k1 = min(p.P, k0 + p.prefix_slice);
  const int n = (k1 - k0 + KT - 1) / KT;  // key tiles, at least 1

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(q_full, 4);
    for (int i = 0; i < NB; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&args.tm_k);
    tma_prefetch_desc(&args.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;

  if (warp == 3) {  // for the blocks that run beside this kernel (prefix.cu)
    if (blockIdx.x == 0 && lane == 0) release_ticket(p.ticket_word, p.ticket);
  } else if (warp == 0) {
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_last();  // the other row tiles read the same tiles
      int slot = 0, phase = 1, loads = 0;
      bool alive = true;
      auto load = [&](const CUtensorMap* tm, int key) {
        if (!mbar_wait(&empty[slot], phase, abort_flag, p.status, 81)) return false;
        mbar_arrive_expect_tx(&full[slot], C::kSlot);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)  // positions past the prefix's end read as zeros
          tma_load_2d(smem + C::kOffSlots + slot * C::kSlot + c * (KT * 128), tm, h * D + c * 64, key, &full[slot], policy);
        ++loads;
        if (++slot == NS) slot = 0, phase ^= 1;
        return true;
      };
      alive = load(&args.tm_k, k0);
      for (int i = 0; i < n && alive; ++i) {
        if (i + 1 < n) alive = load(&args.tm_k, k0 + (i + 1) * KT);
        if (alive) alive = load(&args.tm_v, k0 + i * KT);
      }
      // every load lands before the CTA ends, also when another role gave up
      volatile int drained = 0;
      for (int j = loads > NS ? loads - NS : 0; j < loads; ++j)
        mbar_wait(&full[j % NS], (j / NS) & 1, &drained, p.status, 82);
    }
  } else if (warp == 1 || warp == 2) {
    // Warp 1 issues the scores' products, warp 2 the outputs': what one does
    // between two tiles (waits, commits) runs beside the other's MMAs.
    if (lane == 0) {
      const uint32_t slots = smem_u32(smem + C::kOffSlots);
      int slot = 0, phase = 0, buf = 0, turn = 0;
      auto advance = [&](int by) {
        if ((slot += by) >= NS) slot -= NS, phase ^= 1;
        if (++buf == NB) buf = 0, turn ^= 1;
      };
      if (warp == 1) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(kTcRows, KT);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(smem));
        bool alive = mbar_wait(q_full, 0, abort_flag, p.status, 84);
        for (int i = 0; i < n && alive; ++i) {
          // the columns hold the weights of NB tiles before until their product is complete
          if ((i >= NB && !mbar_wait(&pv_done[buf], turn ^ 1, abort_flag, p.status, 91)) ||
              !mbar_wait(&full[slot], phase, abort_flag, p.status, 83))
            break;
          tc_fence_after();
          const uint64_t k_desc = smem_desc_sw128(slots + slot * C::kSlot);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(tmem + C::kColS + buf * KT, q_desc + ((c * (kTcRows * 128) + kk * 32) >> 4),
                          k_desc + ((c * (KT * 128) + kk * 32) >> 4), idesc_s, (c | kk) != 0);
          tc_commit(&empty[slot]);
          tc_commit(&s_full[buf]);
          advance(i == 0 ? 1 : 2);  // K0 K1 V0 K2 V1 ...
        }
      } else {
        constexpr uint32_t idesc_o = idesc_bf16_f32(kTcRows, D) | (1u << 16);  // B (V) is MN-major
        slot = n > 1 ? 2 : 1;
        for (int i = 0; i < n; ++i) {
          if (!mbar_wait(&full[slot], phase, abort_flag, p.status, 86) ||
              !mbar_wait(&p_full[buf], turn, abort_flag, p.status, 85))
            break;
          tc_fence_after();
          const uint64_t v_desc = smem_desc_mn(slots + slot * C::kSlot, KT * 128);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              tc_mma_ts(tmem, tmem + C::kColS + buf * KT + part * (KT / 2) + kk * 8, v_desc + ((kk * 2048) >> 4), idesc_o,
                        (i | kk | part) != 0);
          tc_commit(&empty[slot]);
          tc_commit(&pv_done[buf]);
          advance(i + 2 < n ? 2 : 1);  // the last V follows the one before it
        }
      }
      volatile int drained = 0;
      tc_commit(drain);  // all MMAs complete before tensor memory is freed
      mbar_wait(drain, 0, &drained, p.status, 87);
    }
  } else if (warp >= 4) {
    const int quarter = warp & 3, r = quarter * 32 + lane;  // this thread's row of the tile
    auto query_row = [&](int row) { return (int64_t)(row / G) * p.Hq + h * G + row % G; };  // of B Hq
    {  // the queries into the swizzled K-major operand; rows past the end as zeros
      constexpr int kChunks = D / 8;
#pragma unroll 4
      for (int k = 0; k < kChunks; ++k) {  // all in flight at once
        const int i = threadIdx.x - 128 + k * 128, row = i / kChunks, c = i % kChunks;
        const bool in = row0 + row < R;
        cp_async_16(smem_u32(smem + (c / 8) * (kTcRows * 128) + sw128_offset(row, c % 8)),
                    p.q + (in ? query_row(row0 + row) * D + c * 8 : 0), in ? 16u : 0u);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      warp_arrive(q_full);
    }
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    float m = -INFINITY, l = 0.f;
    bool alive = true;
    int buf = 0, turn = 0, last = 0, last_turn = 0;  // of this tile and of the one before
    for (int i = 0; i < n; ++i) {
      if (!(alive = warp_wait(&s_full[buf], turn, abort_flag, p.status, 88))) break;
      tc_fence_after();
      uint32_t s[KT / 32][32];
#pragma unroll
      for (int c = 0; c < KT / 32; ++c) tmem_ld_32x32b_x32(tmem + lanes + C::kColS + buf * KT + c * 32, s[c]);
      tc_wait_ld();
      const int left = k1 - (k0 + i * KT);  // keys of this tile inside the slice
      if (left < KT) {
#pragma unroll
        for (int c = 0; c < KT / 32; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c * 32 + j >= left) s[c][j] = 0xFF800000u;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < KT / 32; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[c][j]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      if (__any_sync(0xffffffffu, top > m + kLazyLog2)) {
        const float nm = fmaxf(m, top), f = nm == -INFINITY ? 1.f : ex2(m - nm);  // (m -infinity: 0)
        l *= f;
        m = nm;
        if (i > 0) {
          // O is whole once the product before is complete
          if (!(alive = warp_wait(&pv_done[last], last_turn, abort_flag, p.status, 89))) break;
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
      const float2 sc = make_float2(p.scale_log2, p.scale_log2), nr = make_float2(-ref, -ref);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < KT / 32; ++c) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1])), sc, nr);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          sum = __fadd2_rn(sum, e);
          split_bf16(e.x, e.y, hi[j], lo[j]);
        }
        const uint32_t col = tmem + lanes + C::kColS + buf * KT + c * 16;
        tmem_st_32x32b_x16(col, hi);
        tmem_st_32x32b_x16(col + KT / 2, lo);
      }
      l += sum.x + sum.y;
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&p_full[buf]);
      last = buf, last_turn = turn;
      if (++buf == NB) buf = 0, turn ^= 1;
    }
    // the slice's state: every product is complete with the last one
    const bool mine = row0 + r < R;
    const int64_t at = (int64_t)split * p.B * p.Hq + (mine ? query_row(row0 + r) : 0);
    if (alive) alive = warp_wait(&pv_done[last], last_turn, abort_flag, p.status, 90);
    if (!alive) {  // after a wait that ran out: a state that makes the row NaN, beside the status
      if (mine) p.part_ml[at] = make_float2(0.f, __int_as_float(0x7fc00000));
    } else {
      tc_fence_after();
      if (l != l && m == -INFINITY) m = 0.f;  // nothing but NaN: not a state without positions
      if (mine) p.part_ml[at] = make_float2(m, l);
      // through shared memory (the ring is free: every product is complete), so
      // that a row goes out as one copy; rows 16 bytes further apart than they
      // are long keep eight lanes' stores in different banks
      float* out = reinterpret_cast<float*>(smem + C::kOffSlots + r * (D * 4 + 16));
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(tmem + lanes + c, o);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(out + c + 4 * j) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      }
      fence_proxy_async_smem();
      if (mine) {
        bulk_store(p.part_o + at * D, out, D * 4);
        bulk_commit();
        bulk_wait_all();  // (before the CTA's shared memory goes)
      }
    }
  }
  __syncwarp();  // the single-lane roles join their warps
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

bool encode_cache(CUtensorMap* tm, const uint16_t* base, const PrefixParams& p, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)p.Hkv * p.d, (cuuint64_t)p.P};
  const cuuint64_t strides[1] = {(cuuint64_t)p.ld_prefix * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t prefix_tc_launch_t(const PrefixParams& p, cudaStream_t s) {
  using C = TcCfg<D>;
  TcArgs args;
  memset(&args, 0, sizeof args);
  args.p = p;
  if (!encode_cache(&args.tm_k, p.kp, p, C::KT) || !encode_cache(&args.tm_v, p.vp, p, C::KT)) return cudaErrorInvalidValue;
  static SharedMemoryOptIn opt_in;
  if (const cudaError_t err = opt_in(prefix_tc_kernel<D>, C::kSmem); err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.prefix_blocks);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_tc_kernel<D>, args);
}

}  // namespace

cudaError_t prefix_tc_launch(const PrefixParams& p, cudaStream_t s) {
  if (p.d == 256) return prefix_tc_launch_t<256>(p, s);
  if (p.d == 128) return prefix_tc_launch_t<128>(p, s);
  return prefix_tc_launch_t<64>(p, s);
}

}  // namespace moe
