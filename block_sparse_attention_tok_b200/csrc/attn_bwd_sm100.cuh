// Gradient of the block-sparse attention over kept tiles, for sm_100a.
//
// With P_tu = exp(s q_t . k_u - lse_t) over the kept pairs, dP_tu = do_t . v_u and
// delta_t = sum_c do_tc o_tc (which is sum_u P_tu dP_tu):
//   dS = P * (dP - delta),  dv_u = sum_t P_tu do_t,  dk_u = s sum_t dS_tu q_t,
//   dq_t = s sum_u dS_tu k_u.
// P is recomputed from lse, so nothing of the forward pass's tiles is kept.
//
// Two passes over the kept tiles instead of one with an atomic sum: dkv_kernel holds a KV block
// and walks the query blocks that keep it (4 products a tile), dq_kernel holds a query block
// and walks its KV blocks (3 products a tile). That is 7 products where 5 would do, but every
// output element has one writer and a fixed order of additions, so the same inputs give the
// same bits, as in the forward pass; the one-pass form would also add 64 KB of fp32 reductions
// a tile (about twice what the tile reads) and has no room for them in tensor memory.
//
// Both kernels: persistent, one CTA per SM, 8 softmax warps (two per TMEM lane quarter, each
// pair splitting the 128 columns of a tile), a TMA warp, an MMA warp. A thread keeps half a row
// of P in fp32 registers between the two halves of its work (P from S, dS from dP).
// P and dS are rounded to bf16 as operands of the tensor cores (half a step, 2^-9 of the value
// on average, as the forward pass rounds P); all sums are fp32.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace sparstar {

template <int D, int B>
struct BwdConfig {
  static_assert(D == 64 || D == 128, "head_dim must be 64 or 128");
  static_assert(B == 64 || B == 128, "block must be 64 or 128");
  static constexpr int kBlocksPerTile = 128 / B;       // list entries per 128-row tile
  static constexpr int kChunks = D / 64;               // 128-byte swizzle chunks per row
  static constexpr uint32_t kChunkBytes = 128 * 128;   // 128 rows x 128 bytes
  static constexpr uint32_t kBoxBytes = B * 128;
  static constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
  // The walked operand that two products of a tile use far apart (Q for dK, K for dQ) gets
  // three stages, the other one two: with two held tiles that fills 224 of 227 KB at D = 128.
  static constexpr int kStagesA = 3, kStagesB = 2;
  static constexpr int kStagesStat = 2;
  static constexpr uint32_t kStatBytes = 2 * 128 * 4;  // lse and delta of 128 query rows
  static constexpr int kThreads = 384;
  static constexpr int kSoftmaxThreads = 256;
  static constexpr int kLoadWarp = 8;
  static constexpr int kMmaWarp = 9;
  static constexpr int kRegsSoftmax = 208, kRegsProducer = 80;
  static constexpr int kRegsNeeded = 256 * kRegsSoftmax + 128 * kRegsProducer;
  static constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
  static_assert(kRegsNeeded <= kThreads * kLaunchRegs, "setmaxnreg split above the launch allocation");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSmemBytes = (2 + kStagesA + kStagesB) * kTileBytes + kStagesStat * kStatBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false);
  static constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, true);
};

struct BwdParams {
  const int32_t* idx;      // [H, nqb, kmax] kept KV blocks (dq)
  const int32_t* cnt;      // [H, nqb]
  const int32_t* col_row;  // [H, nqb * kmax] query blocks of each KV block (dkv)
  const int32_t* col_at;   // [H, nkb + 1] first entry of each KV block in col_row
  const float* lse2;       // [H, nqb * B] lse * log2(e), +inf past n_q
  const float* delta;      // [H, nqb * B], 0 past n_q
  __nv_bfloat16 *dq, *dk, *dv;
  unsigned* status;
  int64_t n_q, n_kv;
  int nqb, nkb, kmax, n_items;
  float scale, scale_log2;
};

__device__ __forceinline__ int bwd_count(int c, int kmax) { return c < 1 ? 1 : c > kmax ? kmax : c; }
__device__ __forceinline__ int bwd_block(int j, int n) { return j < 0 ? 0 : j >= n ? n - 1 : j; }

// An untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Barriers of both kernels (dkv names in comments; dq: A = K, B = V, held = Q and dO).
struct BwdBars {
  uint64_t a_full[3], a_empty[3];   // walked operand of two products (Q)
  uint64_t b_full[2], b_empty[2];   // the other walked operand (dO)
  uint64_t st_full[2], st_empty[2]; // lse and delta of the walked rows (dkv only)
  uint64_t held_full, held_empty;   // the held pair of tiles (K, V)
  uint64_t s_full[2], p_full;       // S ready / P written
  uint64_t dp_full, dp_read;        // dP ready / dP taken into registers (dq only)
  uint64_t ds_full, acc_full, drain;
  uint32_t tmem;
  uint32_t abort_flag;
};
static_assert(sizeof(BwdBars) <= 1024, "barrier block");

__device__ __forceinline__ void bwd_bars_init(BwdBars* b) {
  for (int i = 0; i < 3; ++i) {
    mbar_init(&b->a_full[i], 1);
    mbar_init(&b->a_empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&b->b_full[i], 1);
    mbar_init(&b->b_empty[i], 1);
    mbar_init(&b->st_full[i], 1);
    mbar_init(&b->st_empty[i], 1);
    mbar_init(&b->s_full[i], 1);
  }
  mbar_init(&b->held_full, 1);
  mbar_init(&b->held_empty, 1);
  mbar_init(&b->p_full, 256);
  mbar_init(&b->dp_full, 1);
  mbar_init(&b->dp_read, 256);
  mbar_init(&b->ds_full, 256);
  mbar_init(&b->acc_full, 1);
  mbar_init(&b->drain, 1);
  b->abort_flag = 0u;
  fence_barrier_init();
}

// A bounded wait that only lets copies in flight land (their barrier may never complete when
// the CTA gave up before they were issued).
__device__ __forceinline__ void bwd_drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kWaitLimitNs) {
  }
}

// The last use of stage `st` of a ring of `stages` after `uses` loads: waits for it to land.
__device__ __forceinline__ void bwd_drain_ring(uint64_t* full, uint32_t stages, uint32_t uses) {
  for (uint32_t st = 0; st < stages; ++st)
    if (uses > st) bwd_drain(&full[st], ((uses - 1 - st) / stages) & 1u);
}

// Column of the A operand (packed bf16 pairs) of 16-row step kk: each half of a tile's columns
// is written over the start of its own half of the fp32 tile, so that no warp overwrites what
// its partner still reads.
__device__ __forceinline__ uint32_t bwd_a_col(int kk) { return static_cast<uint32_t>((kk >> 2) * 64 + (kk & 3) * 8); }

// 64 fp32 values -> bf16 pairs -> 32 TMEM columns.
__device__ __forceinline__ void bwd_store_half(uint32_t taddr, const float (&x)[64]) {
  uint32_t pk[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
  tmem_st32(taddr, pk);
}

__device__ __forceinline__ void bwd_load_half(uint32_t taddr, uint32_t (&r)[2][32]) {
  tmem_ld32(taddr, r[0]);
  tmem_ld32(taddr + 32, r[1]);
  tmem_wait_ld();
}

// An accumulator row of N fp32 columns times `f`, as bf16, to `dst` where `put`.
template <int N>
__device__ __forceinline__ void bwd_store_row(uint32_t taddr, __nv_bfloat16* dst, bool put, float f) {
#pragma unroll 1
  for (int c = 0; c < N / 32; ++c) {
    uint32_t ov[32];
    tmem_ld32(taddr + 32 * c, ov);
    tmem_wait_ld();
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * f, __uint_as_float(ov[2 * e + 1]) * f);
    if (put) {
      uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * c);
#pragma unroll
      for (int v = 0; v < 4; ++v) __stcs(d4 + v, make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]));
    }
  }
}

// ------------------------------------------------------------------------ dK and dV
//
// Tensor memory: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [384,384+D): rows are KV tokens.
// Tile n of an item (KV block, query blocks that keep it), in the MMA warp's issue order:
//   dV += P^T(n) dO(n);  S^T(n+1) = K Q(n+1)^T;  dK += dS^T(n) Q(n);  dP^T(n+1) = V dO(n+1)^T.
// The softmax warps work on dS(n) while dV(n) and S(n+1) run, and on P(n+1) while dK(n) and
// dP(n+1) run, so S, dP and the two accumulators need one buffer each (all 512 columns).
// S(n+1) may overwrite P(n): tcgen05.mma of one thread run in order.
template <int D, int B>
__global__ void __launch_bounds__(BwdConfig<D, B>::kThreads, 1)
    attn_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const BwdParams p) {
  using C = BwdConfig<D, B>;
  constexpr int BPT = C::kBlocksPerTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* k_tile = smem;
  uint8_t* v_tile = smem + C::kTileBytes;
  uint8_t* q_ring = smem + 2 * C::kTileBytes;
  uint8_t* do_ring = q_ring + C::kStagesA * C::kTileBytes;
  uint8_t* st_ring = do_ring + C::kStagesB * C::kTileBytes;
  BwdBars* bars = reinterpret_cast<BwdBars*>(st_ring + C::kStagesStat * C::kStatBytes);
  volatile uint32_t* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The swizzled tiles need a 1024-byte aligned base, which this kernel's shared memory has
  // (it declares no static array); were it ever otherwise, nothing is computed and it is reported.
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) bwd_bars_init(bars);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  constexpr uint32_t kS = 0, kDP = 128, kDV = 256, kDK = 384;

  struct Item {
    int h, j, n_ent, n_tiles;
    const int32_t* rows;
  };
  auto get = [&](int item) {
    Item it;
    it.h = item / p.nkb;
    it.j = item - it.h * p.nkb;
    const int32_t* at = p.col_at + static_cast<int64_t>(it.h) * (p.nkb + 1) + it.j;
    const int a = __ldg(at), b = __ldg(at + 1);
    it.n_ent = b - a;
    it.n_tiles = (it.n_ent + BPT - 1) / BPT;
    it.rows = p.col_row + static_cast<int64_t>(it.h) * p.nqb * p.kmax + a;
    return it;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsProducer));
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        const uint64_t pol_held = l2_policy_evict_first(), pol_walk = l2_policy_evict_last();
        uint32_t t = 0, held = 0;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
          const Item it = get(item);
          if (it.n_tiles == 0) continue;
          ok = mbar_wait(&bars->held_empty, (held & 1u) ^ 1u, abort_flag, p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars->held_full, 2 * C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            tma_load_3d_hint(smem_u32(k_tile) + c * C::kChunkBytes, &tm_k, &bars->held_full, c * 64, it.j * B, it.h,
                             pol_held);
            tma_load_3d_hint(smem_u32(v_tile) + c * C::kChunkBytes, &tm_v, &bars->held_full, c * 64, it.j * B, it.h,
                             pol_held);
          }
          ++held;
          for (int n = 0; n < it.n_tiles; ++n, ++t) {
            int qb[BPT];
#pragma unroll
            for (int b = 0; b < BPT; ++b) {
              const int e = n * BPT + b;
              qb[b] = __ldg(it.rows + (e < it.n_ent ? e : n * BPT));
            }
            const uint32_t sa = t % C::kStagesA, sb = t % C::kStagesB;
            ok = mbar_wait(&bars->st_empty[sb], ((t / 2) & 1u) ^ 1u, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx(&bars->st_full[sb], C::kStatBytes);
            const uint32_t st = smem_u32(st_ring) + sb * C::kStatBytes;
#pragma unroll
            for (int b = 0; b < BPT; ++b) {
              const int64_t at = (static_cast<int64_t>(it.h) * p.nqb + qb[b]) * B;
              bulk_load(st + b * B * 4, p.lse2 + at, B * 4, &bars->st_full[sb]);
              bulk_load(st + 512 + b * B * 4, p.delta + at, B * 4, &bars->st_full[sb]);
            }
            ok = mbar_wait(&bars->a_empty[sa], ((t / C::kStagesA) & 1u) ^ 1u, abort_flag, p.status);
            if (!ok) {
              bwd_drain(&bars->st_full[sb], (t / 2) & 1u);
              break;
            }
            mbar_arrive_expect_tx(&bars->a_full[sa], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int b = 0; b < BPT; ++b)
                tma_load_3d_hint(smem_u32(q_ring) + sa * C::kTileBytes + c * C::kChunkBytes + b * C::kBoxBytes, &tm_q,
                                 &bars->a_full[sa], c * 64, qb[b] * B, it.h, pol_walk);
            ok = mbar_wait(&bars->b_empty[sb], ((t / 2) & 1u) ^ 1u, abort_flag, p.status);
            if (!ok) {
              bwd_drain(&bars->st_full[sb], (t / 2) & 1u);
              bwd_drain(&bars->a_full[sa], (t / C::kStagesA) & 1u);
              break;
            }
            mbar_arrive_expect_tx(&bars->b_full[sb], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int b = 0; b < BPT; ++b)
                tma_load_3d_hint(smem_u32(do_ring) + sb * C::kTileBytes + c * C::kChunkBytes + b * C::kBoxBytes, &tm_do,
                                 &bars->b_full[sb], c * 64, qb[b] * B, it.h, pol_walk);
          }
        }
        // every copy lands before the CTA exits (matters only after an abort)
        if (held > 0) bwd_drain(&bars->held_full, (held - 1) & 1u);
        bwd_drain_ring(bars->st_full, 2, t);
        bwd_drain_ring(bars->a_full, C::kStagesA, t);
        bwd_drain_ring(bars->b_full, C::kStagesB, t);
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status));
      };
      const uint64_t k_desc = smem_desc_sw128(smem_u32(k_tile), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(v_tile), 16, 1024);
      const uint64_t q_desc = smem_desc_sw128(smem_u32(q_ring), 16, 1024);
      const uint64_t do_desc = smem_desc_sw128(smem_u32(do_ring), 16, 1024);
      const uint64_t q_mn = smem_desc_sw128(smem_u32(q_ring), C::kChunkBytes, 1024);
      const uint64_t do_mn = smem_desc_sw128(smem_u32(do_ring), C::kChunkBytes, 1024);
      auto product = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
          mma_ss(d, a + off, b + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
      };
      auto gather = [&](uint32_t d, uint32_t a, uint64_t b, bool add) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(d, a + bwd_a_col(kk), b + ((kk * 2048) >> 4), C::kIdescAcc, (add || kk > 0) ? 1u : 0u);
      };
      uint32_t t = 0, held = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t u) -> bool {
        const uint32_t sa = u % C::kStagesA;
        if (!wait_all(&bars->a_full[sa], (u / C::kStagesA) & 1u)) return false;
        if (elect_one()) {
          product(tmem + kS, k_desc, q_desc + ((sa * C::kTileBytes) >> 4));
          mma_commit(&bars->s_full[0]);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](uint32_t u, bool last) -> bool {
        const uint32_t sb = u % C::kStagesB;
        if (!wait_all(&bars->b_full[sb], (u / C::kStagesB) & 1u)) return false;
        if (elect_one()) {
          product(tmem + kDP, v_desc, do_desc + ((sb * C::kTileBytes) >> 4));
          mma_commit(&bars->dp_full);
          if (last) mma_commit(&bars->held_empty);
        }
        __syncwarp();
        return true;
      };
      for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
        const Item it = get(item);
        if (it.n_tiles == 0) continue;
        ok = wait_all(&bars->held_full, held & 1u);
        if (!ok) break;
        ++held;
        ok = issue_s(t) && issue_dp(t, it.n_tiles == 1);
        for (int n = 0; ok && n < it.n_tiles; ++n, ++t) {
          const bool last = n == it.n_tiles - 1;
          const uint32_t sa = t % C::kStagesA, sb = t % C::kStagesB;
          if (!(ok = wait_all(&bars->p_full, t & 1u))) break;
          tc_fence_after();
          if (elect_one()) {
            gather(tmem + kDV, tmem + kS, do_mn + ((sb * C::kTileBytes) >> 4), n > 0);
            mma_commit(&bars->b_empty[sb]);
          }
          __syncwarp();
          if (!last && !(ok = issue_s(t + 1))) break;
          if (!(ok = wait_all(&bars->ds_full, t & 1u))) break;
          tc_fence_after();
          if (elect_one()) {
            gather(tmem + kDK, tmem + kDP, q_mn + ((sa * C::kTileBytes) >> 4), n > 0);
            mma_commit(&bars->a_empty[sa]);
            mma_commit(&bars->st_empty[sb]);
            if (last) mma_commit(&bars->acc_full);
          }
          __syncwarp();
          if (!last && !(ok = issue_dp(t + 1, n == it.n_tiles - 2))) break;
        }
      }
      if (elect_one()) mma_commit(&bars->drain);
      __syncwarp();
      bwd_drain(&bars->drain, 0);
      __syncwarp();
    }  // warps 10 and 11 only complete the warpgroup
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // ---------------------------------------------------------- P, dS and the epilogue
    const int half = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;  // KV token of the block
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_off + kS + 64 * half, t_dp = tmem + lane_off + kDP + 64 * half;
    uint32_t t = 0, done = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status));
    };
    for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
      const Item it = get(item);
      const int64_t tok = static_cast<int64_t>(it.j) * B + row;
      const bool put = row < B && tok < p.n_kv;
      __nv_bfloat16* dst = (half == 0 ? p.dv : p.dk) + (static_cast<int64_t>(it.h) * p.n_kv + tok) * D;
      if (it.n_tiles == 0) {  // a block that no query block keeps
        if (put)
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      // With 64-token blocks rows 64-127 belong to the next KV block: computed, never stored.
      const bool idle = B < 128 && wq * 32 >= B;
      for (int n = 0; n < it.n_tiles; ++n, ++t) {
        const uint32_t sb = t & 1u;
        const float4* lse = reinterpret_cast<const float4*>(st_ring + sb * C::kStatBytes + half * 256);
        const float4* del = reinterpret_cast<const float4*>(st_ring + sb * C::kStatBytes + 512 + half * 256);
        if (!(ok = wait_all(&bars->st_full[sb], (t >> 1) & 1u))) break;
        if (!(ok = wait_all(&bars->s_full[0], t & 1u))) break;
        if (idle) {
          // whatever S and dP left there stands in for P and dS of rows that are dropped
          mbar_arrive(&bars->p_full);
          if (!(ok = wait_all(&bars->dp_full, t & 1u))) break;
          mbar_arrive(&bars->ds_full);
          continue;
        }
        tc_fence_after();
        uint32_t r[2][32];
        float pr[64];
        bwd_load_half(t_s, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 l = lse[e];
          const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * e + i;
            pr[c] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][c & 31]), p.scale_log2, -lv[i]));
          }
        }
        if (BPT > 1 && half == 1 && 2 * n + 1 >= it.n_ent) {  // odd last entry: its half repeats a block
#pragma unroll
          for (int c = 0; c < 64; ++c) pr[c] = 0.f;
        }
        bwd_store_half(t_s, pr);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full);
        if (!(ok = wait_all(&bars->dp_full, t & 1u))) break;
        tc_fence_after();
        bwd_load_half(t_dp, r);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float4 l = del[e];
          const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * e + i;
            pr[c] *= __uint_as_float(r[c >> 5][c & 31]) - lv[i];
          }
        }
        bwd_store_half(t_dp, pr);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);
      }
      if (!ok) break;
      if (!(ok = wait_all(&bars->acc_full, done & 1u))) break;
      ++done;
      tc_fence_after();
      if (!idle) bwd_store_row<D>(tmem + lane_off + (half == 0 ? kDV : kDK), dst, put, half == 0 ? 1.f : p.scale);
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------------ dQ
//
// Tensor memory: S of even and odd tiles [0,128), [128,256), dP [256,384), dQ [384,384+D): rows are
// query tokens. Issue order per tile n: S(n+1) = Q K(n+1)^T; dP(n+1) = dO V(n+1)^T once dP(n) is in
// registers; dQ += dS(n) K(n), with dS(n) over S(n). The softmax warps never wait for a product
// that starts after their own previous step.
template <int D, int B>
__global__ void __launch_bounds__(BwdConfig<D, B>::kThreads, 1)
    attn_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const BwdParams p) {
  using C = BwdConfig<D, B>;
  constexpr int BPT = C::kBlocksPerTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* q_tile = smem;
  uint8_t* do_tile = smem + C::kTileBytes;
  uint8_t* k_ring = smem + 2 * C::kTileBytes;
  uint8_t* v_ring = k_ring + C::kStagesA * C::kTileBytes;
  BwdBars* bars = reinterpret_cast<BwdBars*>(v_ring + C::kStagesB * C::kTileBytes);
  volatile uint32_t* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) bwd_bars_init(bars);
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  constexpr uint32_t kS = 0, kDP = 256, kDQ = 384;

  auto tiles_of = [&](int item, int* n_ent) {
    *n_ent = bwd_count(__ldg(p.cnt + item), p.kmax);
    return (*n_ent + BPT - 1) / BPT;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsProducer));
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        const uint64_t pol_held = l2_policy_evict_first(), pol_walk = l2_policy_evict_last();
        uint32_t t = 0, held = 0;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
          const int h = item / p.nqb, qb = item - h * p.nqb;
          int n_ent;
          const int n_tiles = tiles_of(item, &n_ent);
          const int32_t* list = p.idx + static_cast<int64_t>(item) * p.kmax;
          ok = mbar_wait(&bars->held_empty, (held & 1u) ^ 1u, abort_flag, p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(&bars->held_full, 2 * C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            tma_load_3d_hint(smem_u32(q_tile) + c * C::kChunkBytes, &tm_q, &bars->held_full, c * 64, qb * B, h,
                             pol_held);
            tma_load_3d_hint(smem_u32(do_tile) + c * C::kChunkBytes, &tm_do, &bars->held_full, c * 64, qb * B, h,
                             pol_held);
          }
          ++held;
          for (int n = 0; n < n_tiles; ++n, ++t) {
            int jb[BPT];
#pragma unroll
            for (int b = 0; b < BPT; ++b) {
              const int e = n * BPT + b;
              jb[b] = bwd_block(__ldg(list + (e < n_ent ? e : n * BPT)), p.nkb);
            }
            const uint32_t sa = t % C::kStagesA, sb = t % C::kStagesB;
            ok = mbar_wait(&bars->a_empty[sa], ((t / C::kStagesA) & 1u) ^ 1u, abort_flag, p.status);
            if (!ok) break;
            mbar_arrive_expect_tx(&bars->a_full[sa], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int b = 0; b < BPT; ++b)
                tma_load_3d_hint(smem_u32(k_ring) + sa * C::kTileBytes + c * C::kChunkBytes + b * C::kBoxBytes, &tm_k,
                                 &bars->a_full[sa], c * 64, jb[b] * B, h, pol_walk);
            ok = mbar_wait(&bars->b_empty[sb], ((t / C::kStagesB) & 1u) ^ 1u, abort_flag, p.status);
            if (!ok) {
              bwd_drain(&bars->a_full[sa], (t / C::kStagesA) & 1u);
              break;
            }
            mbar_arrive_expect_tx(&bars->b_full[sb], C::kTileBytes);
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
              for (int b = 0; b < BPT; ++b)
                tma_load_3d_hint(smem_u32(v_ring) + sb * C::kTileBytes + c * C::kChunkBytes + b * C::kBoxBytes, &tm_v,
                                 &bars->b_full[sb], c * 64, jb[b] * B, h, pol_walk);
          }
        }
        if (held > 0) bwd_drain(&bars->held_full, (held - 1) & 1u);
        bwd_drain_ring(bars->a_full, C::kStagesA, t);
        bwd_drain_ring(bars->b_full, C::kStagesB, t);
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status));
      };
      const uint64_t q_desc = smem_desc_sw128(smem_u32(q_tile), 16, 1024);
      const uint64_t do_desc = smem_desc_sw128(smem_u32(do_tile), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_u32(k_ring), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_u32(v_ring), 16, 1024);
      const uint64_t k_mn = smem_desc_sw128(smem_u32(k_ring), C::kChunkBytes, 1024);
      auto product = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
          mma_ss(d, a + off, b + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
      };
      uint32_t t = 0, held = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t u) -> bool {
        const uint32_t sa = u % C::kStagesA;
        if (!wait_all(&bars->a_full[sa], (u / C::kStagesA) & 1u)) return false;
        if (elect_one()) {
          product(tmem + kS + 128u * (u & 1u), q_desc, k_desc + ((sa * C::kTileBytes) >> 4));
          mma_commit(&bars->s_full[u & 1u]);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](uint32_t u, bool last) -> bool {
        const uint32_t sb = u % C::kStagesB;
        if (u > 0 && !wait_all(&bars->dp_read, (u - 1) & 1u)) return false;
        if (!wait_all(&bars->b_full[sb], (u / C::kStagesB) & 1u)) return false;
        tc_fence_after();
        if (elect_one()) {
          product(tmem + kDP, do_desc, v_desc + ((sb * C::kTileBytes) >> 4));
          mma_commit(&bars->dp_full);
          mma_commit(&bars->b_empty[sb]);
          if (last) mma_commit(&bars->held_empty);
        }
        __syncwarp();
        return true;
      };
      for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
        int n_ent;
        const int n_tiles = tiles_of(item, &n_ent);
        ok = wait_all(&bars->held_full, held & 1u);
        if (!ok) break;
        ++held;
        ok = issue_s(t) && issue_dp(t, n_tiles == 1);
        for (int n = 0; ok && n < n_tiles; ++n, ++t) {
          const bool last = n == n_tiles - 1;
          if (!last && !(ok = issue_s(t + 1) && issue_dp(t + 1, n == n_tiles - 2))) break;
          if (!(ok = wait_all(&bars->ds_full, t & 1u))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = t % C::kStagesA;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + kDQ, tmem + kS + 128u * (t & 1u) + bwd_a_col(kk),
                     k_mn + ((sa * C::kTileBytes + kk * 2048) >> 4), C::kIdescAcc, (n > 0 || kk > 0) ? 1u : 0u);
            mma_commit(&bars->a_empty[sa]);
            if (last) mma_commit(&bars->acc_full);
          }
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit(&bars->drain);
      __syncwarp();
      bwd_drain(&bars->drain, 0);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // ---------------------------------------------------------- dS and the epilogue
    const int half = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;  // query token of the block
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    uint32_t t = 0, done = 0;
    bool ok = true;
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status));
    };
    const bool ragged_kv = p.n_kv % B != 0;
    const bool idle = B < 128 && wq * 32 >= B;
    for (int item = blockIdx.x; ok && item < p.n_items; item += gridDim.x) {
      const int h = item / p.nqb, qb = item - h * p.nqb;
      int n_ent;
      const int n_tiles = tiles_of(item, &n_ent);
      const int32_t* list = p.idx + static_cast<int64_t>(item) * p.kmax;
      const int64_t tok = static_cast<int64_t>(qb) * B + row;
      float neg_lse = 0.f, delta = 0.f;
      if (row < B) {
        const int64_t at = (static_cast<int64_t>(h) * p.nqb + qb) * B + row;
        neg_lse = -__ldg(p.lse2 + at);
        delta = __ldg(p.delta + at);
      }
      for (int n = 0; n < n_tiles; ++n, ++t) {
        const uint32_t t_s = tmem + lane_off + kS + 128u * (t & 1u) + 64 * half;
        const uint32_t t_dp = tmem + lane_off + kDP + 64 * half;
        // valid columns of this half of the tile
        int nv = 64;
        if (BPT > 1 && half == 1 && 2 * n + 1 >= n_ent) nv = 0;  // odd last entry: its half repeats a block
        if (ragged_kv && nv > 0) {
          const int j = bwd_block(__ldg(list + (BPT > 1 ? 2 * n + half : n)), p.nkb);
          if (j == p.nkb - 1) {
            const int64_t left = p.n_kv - static_cast<int64_t>(j) * B - (BPT > 1 ? 0 : 64 * half);
            nv = left < 0 ? 0 : left < 64 ? static_cast<int>(left) : 64;
          }
        }
        if (!(ok = wait_all(&bars->s_full[t & 1u], (t >> 1) & 1u))) break;
        if (idle) {
          if (!(ok = wait_all(&bars->dp_full, t & 1u))) break;
          mbar_arrive(&bars->dp_read);
          mbar_arrive(&bars->ds_full);
          continue;
        }
        tc_fence_after();
        uint32_t r[2][32];
        float pr[64];
        bwd_load_half(t_s, r);
#pragma unroll
        for (int c = 0; c < 64; ++c)
          pr[c] = ex2_approx(fmaf(__uint_as_float(r[c >> 5][c & 31]), p.scale_log2, neg_lse));
        if (nv < 64) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= nv) pr[c] = 0.f;
        }
        if (!(ok = wait_all(&bars->dp_full, t & 1u))) break;
        tc_fence_after();
        bwd_load_half(t_dp, r);
        tc_fence_before();
        mbar_arrive(&bars->dp_read);
#pragma unroll
        for (int c = 0; c < 64; ++c) pr[c] *= __uint_as_float(r[c >> 5][c & 31]) - delta;
        bwd_store_half(t_s, pr);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);
      }
      if (!ok) break;
      if (!(ok = wait_all(&bars->acc_full, done & 1u))) break;
      ++done;
      tc_fence_after();
      const bool put = row < B && tok < p.n_q;
      if (!idle)
        bwd_store_row<D / 2>(tmem + lane_off + kDQ + (D / 2) * half,
                             p.dq + (static_cast<int64_t>(h) * p.n_q + tok) * D + (D / 2) * half, put, p.scale);
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------------ row statistics
//
// lse2 = lse log2(e) and delta = do . o of every query row, padded to whole blocks (+inf and 0
// past n_q: such a row's P is 0), so that a block's statistics are one aligned copy. One read of
// o and do, D / 8 lanes a row. Memory-bound and small beside the products.
template <int D>
__global__ void __launch_bounds__(256)
    bwd_rows_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ d_o,
                    const float* __restrict__ lse, int64_t n_q, int64_t n_pad, float* __restrict__ lse2,
                    float* __restrict__ delta) {
  constexpr int G = D / 8;
  const int l = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G;
  const int64_t h = blockIdx.y;
  float s = 0.f;
  if (row < n_q) {
    const int64_t at = (h * n_q + row) * D + 8 * l;
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(o + at));
    const uint4 b = __ldcs(reinterpret_cast<const uint4*>(d_o + at));
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
      s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
    }
  }
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  if (l == 0 && row < n_pad) {
    lse2[h * n_pad + row] = row < n_q ? __ldg(lse + h * n_q + row) * 1.4426950408889634f : INFINITY;
    delta[h * n_pad + row] = s;
  }
}

// ------------------------------------------------------------------------ transposed lists
//
// Query blocks of each KV block, ascending, from the kept lists: a counting sort that is stable
// by rows. Rows are cut into chunks of kMaskRows; each (chunk, head) counts its entries per KV
// block, the counts are scanned over chunks and blocks, and each (chunk, head) places its rows
// one after another. A block listed twice in a row is placed twice (the forward pass attends to
// it twice). Out-of-range entries are clamped as the forward pass clamps them, and recorded.
constexpr int kMaskRows = 32;
constexpr int kMaskMaxBlocks = 49152;  // KV blocks at most: one 4-byte counter each in shared memory

__global__ void __launch_bounds__(256)
    mask_count_kernel(const int32_t* __restrict__ idx, const int32_t* __restrict__ cnt, int nqb, int nkb, int kmax,
                      int32_t* __restrict__ chunk_cnt, unsigned* status) {
  extern __shared__ int32_t hist[];
  const int chunk = blockIdx.x, h = blockIdx.y;
  for (int j = threadIdx.x; j < nkb; j += blockDim.x) hist[j] = 0;
  __syncthreads();
  const int r1 = min(nqb, (chunk + 1) * kMaskRows);
  for (int i = chunk * kMaskRows; i < r1; ++i) {
    const int64_t at = static_cast<int64_t>(h) * nqb + i;
    const int c0 = __ldg(cnt + at), c = bwd_count(c0, kmax);
    if (c != c0 && threadIdx.x == 0) atomicOr(status, kStatusBounds);
    for (int e = threadIdx.x; e < c; e += blockDim.x) {
      const int j0 = __ldg(idx + at * kmax + e), j = bwd_block(j0, nkb);
      if (j != j0) atomicOr(status, kStatusBounds);
      atomicAdd(&hist[j], 1);
    }
  }
  __syncthreads();
  int32_t* out = chunk_cnt + (static_cast<int64_t>(h) * gridDim.x + chunk) * nkb;
  for (int j = threadIdx.x; j < nkb; j += blockDim.x) out[j] = hist[j];
}

// One CTA per head: chunk_cnt becomes each chunk's first place within a KV block, col_at the
// block's first place within the head.
__global__ void __launch_bounds__(1024)
    mask_scan_kernel(int nkb, int n_chunks, int32_t* __restrict__ chunk_cnt, int32_t* __restrict__ col_at) {
  __shared__ int32_t warp_sum[32];
  __shared__ int32_t base;
  const int h = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int32_t* cc = chunk_cnt + static_cast<int64_t>(h) * n_chunks * nkb;
  int32_t* at = col_at + static_cast<int64_t>(h) * (nkb + 1);
  if (threadIdx.x == 0) base = 0;
  for (int j0 = 0; j0 < nkb; j0 += 1024) {
    const int j = j0 + threadIdx.x;
    int total = 0;
    if (j < nkb)
      for (int c = 0; c < n_chunks; ++c) {
        const int v = cc[static_cast<int64_t>(c) * nkb + j];
        cc[static_cast<int64_t>(c) * nkb + j] = total;
        total += v;
      }
    int incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sum[w] = incl;
    __syncthreads();
    if (w == 0) {
      int v = warp_sum[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, off);
        if (lane >= off) v += u;
      }
      warp_sum[lane] = v;
    }
    __syncthreads();
    const int before = base + (w > 0 ? warp_sum[w - 1] : 0) + incl - total;
    if (j < nkb) at[j] = before;
    __syncthreads();
    if (threadIdx.x == 1023) base = before + total;
    __syncthreads();
  }
  if (threadIdx.x == 0) at[nkb] = base;
}

__global__ void __launch_bounds__(256)
    mask_fill_kernel(const int32_t* __restrict__ idx, const int32_t* __restrict__ cnt, int nqb, int nkb, int kmax,
                     const int32_t* __restrict__ chunk_cnt, const int32_t* __restrict__ col_at,
                     int32_t* __restrict__ col_row) {
  extern __shared__ int32_t place[];
  const int chunk = blockIdx.x, h = blockIdx.y;
  const int32_t* cc = chunk_cnt + (static_cast<int64_t>(h) * gridDim.x + chunk) * nkb;
  const int32_t* at = col_at + static_cast<int64_t>(h) * (nkb + 1);
  for (int j = threadIdx.x; j < nkb; j += blockDim.x) place[j] = at[j] + cc[j];
  int32_t* out = col_row + static_cast<int64_t>(h) * nqb * kmax;
  const int r1 = min(nqb, (chunk + 1) * kMaskRows);
  for (int i = chunk * kMaskRows; i < r1; ++i) {
    __syncthreads();  // rows in order
    const int64_t row = static_cast<int64_t>(h) * nqb + i;
    const int c = bwd_count(__ldg(cnt + row), kmax);
    for (int e = threadIdx.x; e < c; e += blockDim.x)
      out[atomicAdd(&place[bwd_block(__ldg(idx + row * kmax + e), nkb)], 1)] = i;
  }
}

}  // namespace sparstar
