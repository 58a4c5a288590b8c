// Gradient of the block-sparse attention over kept tiles, for sm_100a.
//
// With P_tu = exp(s q_t . k_u - lse_t) over the kept pairs, dP_tu = do_t . v_u and
// delta_t = sum_c do_tc o_tc (which is sum_u P_tu dP_tu):
//   dS = P * (dP - delta),  dv_u = sum_t P_tu do_t,  dk_u = s sum_t dS_tu q_t,
//   dq_t = s sum_u dS_tu k_u.
// P is recomputed from lse, so nothing of the forward pass's tiles is kept.
//
// Two passes over the kept tiles instead of one with an atomic sum: a dK/dV item holds a KV block
// and walks the query blocks that keep it (4 products a tile), a dQ item holds a query block
// and walks its KV blocks (3 products a tile). That is 7 products where 5 would do, but every
// output element has one writer and a fixed order of additions, so the same inputs give the
// same bits, as in the forward pass; the one-pass form would also add 64 KB of fp32 reductions
// a tile, as much as a dK/dV tile reads of Q and dO, and its fifth product would have to take turns
// with S: S, dP, dV and dK fill tensor memory. A form that stores dS for the dQ items has not been built.
//
// One persistent kernel does both, one CTA per SM: 8 softmax warps (two per TMEM lane quarter,
// each pair splitting the 128 columns of a tile), a TMA warp, an MMA warp. A thread keeps half a
// row of P in fp32 registers between the two halves of its work (P from S, dS from dP).
// P and dS are rounded to bf16 as operands of the tensor cores (each off by at most 2^-8 of its
// value, as the forward pass rounds P); all sums are fp32.
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
  static constexpr int kLoadWarp = 8;
  static constexpr int kMmaWarp = 9;
  static constexpr int kRegsSoftmax = 200, kRegsProducer = 96;
  static constexpr int kRegsNeeded = 256 * kRegsSoftmax + 128 * kRegsProducer;
  static constexpr int kLaunchRegs = (65536 / kThreads) & ~7;
  static_assert(kRegsNeeded <= kThreads * kLaunchRegs, "setmaxnreg split above the launch allocation");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kSmemBytes = (2 + kStagesA + kStagesB) * kTileBytes + kStagesStat * kStatBytes + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false);
  static constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, true);
};

// A run of a long list, one of `n` from parts[base] on.
struct BwdPart {
  int32_t item, first, count, base, n;
};
constexpr int kBwdMaxParts = 296;  // two for each of 148 SMs: see the choice of part_ent

struct BwdParams {
  const int32_t* idx;      // [H, nqb, kmax] kept KV blocks (dq)
  const int32_t* cnt;      // [H, nqb]
  const int32_t* col_row;  // [H, nqb * kmax] query blocks of each KV block (dkv)
  const int32_t* col_at;   // [H, nkb + 1] first entry of each KV block in col_row
  const float* neg_lse2;   // [H, nqb * B] -lse log2(e), -inf past n_q
  const float* neg_delta;  // [H, nqb * B] -delta, 0 past n_q
  __nv_bfloat16 *dq, *dk, *dv;
  unsigned* status;
  int* next;               // item counter (0 at launch), and how many parts there are
  const struct BwdPart* parts;  // parts of long lists
  float* part_sum;         // [parts][dV, dK][B][D]
  int* part_done;          // [parts][8]: how many parts of a list a softmax warp has stored (0 at launch)
  int part_ent;            // entries of a part at most; longer lists are split
  int64_t n_q, n_kv;
  int nqb, nkb, kmax;
  int n_dkv, n_dq;         // items of either kind
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

// Tensor maps of q, do, k, v: boxes of one block (walked), and of 128 rows (held).
struct BwdMaps {
  CUtensorMap walk[4], held[4];
};

// Barriers of one kind of items (dK/dV names in comments; dQ: a = K, b = V, held = Q and dO).
struct BwdPhaseBars {
  uint64_t a_full[3], a_empty[3];    // walked operand of two products (Q)
  uint64_t b_full[2], b_empty[2];    // the other walked operand (dO)
  uint64_t st_full[2], st_empty[2];  // lse and delta of the walked rows (dK/dV only)
  uint64_t held_full, held_empty;    // the held pair of tiles (K, V)
  uint64_t s_full, p_full;           // S ready / P written (dK/dV only)
  uint64_t dp_full, ds_full;         // dP ready / dS written
  uint64_t hold_tm, s_read;          // Q and dO in tensor memory / S taken into registers (dQ only)
  uint64_t acc_full;
};

struct BwdBars {
  BwdPhaseBars dkv, dq;
  uint64_t item_full[2], item_empty[2];
  uint64_t smem_free, tmem_free, drain;
  int32_t item[2], n_ent[2], part[2];
  uint32_t tmem;
  uint32_t abort_flag;
};
static_assert(sizeof(BwdBars) <= 1024, "barrier block");

__device__ __forceinline__ void bwd_bars_init(BwdBars* bars) {
  for (BwdPhaseBars* b : {&bars->dkv, &bars->dq}) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&b->a_full[i], 1);
      mbar_init(&b->a_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->b_full[i], 1);
      mbar_init(&b->b_empty[i], 1);
      mbar_init(&b->st_full[i], 1);
      mbar_init(&b->st_empty[i], 1);
    }
    mbar_init(&b->s_full, 1);
    mbar_init(&b->held_full, 1);
    mbar_init(&b->held_empty, b == &bars->dkv ? 1 : 8);  // by the products, or by the warps that copy it
    mbar_init(&b->p_full, 8);  // one arrival per softmax warp, here and below
    mbar_init(&b->dp_full, 1);
    mbar_init(&b->ds_full, 8);
    mbar_init(&b->hold_tm, 8);
    mbar_init(&b->s_read, 8);
    mbar_init(&b->acc_full, 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bars->item_full[i], 1);
    mbar_init(&bars->item_empty[i], 9);  // the MMA warp and 8 softmax warps
  }
  mbar_init(&bars->smem_free, 1);
  mbar_init(&bars->tmem_free, 8);
  mbar_init(&bars->drain, 1);
  bars->abort_flag = 0u;
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

// 64 fp32 values (as pairs of neighbours) -> bf16 pairs -> 32 TMEM columns.
__device__ __forceinline__ void bwd_store_half(uint32_t taddr, const float2 (&x)[32]) {
  uint32_t pk[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) pk[e] = pack_bf16x2(x[e].x, x[e].y);
  tmem_st32(taddr, pk);
}

// Columns 2e and 2e + 1 of half a row.
__device__ __forceinline__ float2 bwd_pair(const uint32_t (&r)[2][32], int e) {
  return make_float2(__uint_as_float(r[e >> 4][(2 * e) & 31]), __uint_as_float(r[e >> 4][(2 * e + 1) & 31]));
}

// P of a pair of columns: exp2(s * scale - lse2).
__device__ __forceinline__ float2 bwd_exp(float2 s, float2 scale, float2 neg_lse) {
  const float2 x = __ffma2_rn(s, scale, neg_lse);
  return make_float2(ex2_approx(x.x), ex2_approx(x.y));
}

__device__ __forceinline__ void bwd_load_half(uint32_t taddr, uint32_t (&r)[2][32]) {
  tmem_ld32(taddr, r[0]);
  tmem_ld32(taddr + 32, r[1]);
  tmem_wait_ld();
}

// 32 columns of a warp's 32 rows, a row a lane as bf16 pairs, to `dst` (the first row's columns; rows
// `stride` elements apart, `rows` of them to be written). Four lanes swap their 16-byte units first, so that
// a store covers 64 bytes of 8 rows instead of 16 bytes of 32, which the load/store unit takes a row at a time.
// With it and the parts' sums in whole lines 8 heads of 4,096 queries take 72 us instead of 92 us, 2 heads of
// 18,432 203 us instead of 219 us.
__device__ __forceinline__ void bwd_put32(const uint32_t (&pk)[16], __nv_bfloat16* dst, int stride, int rows) {
  const int lane = threadIdx.x & 31;
  uint32_t u[4][4];
#pragma unroll
  for (int e = 0; e < 16; ++e) u[e >> 2][e & 3] = pk[e];
#pragma unroll
  for (int m = 0; m < 4; m += 2)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? u[m][w] : u[m + 1][w], 1);
      if (lane & 1)
        u[m][w] = got;
      else
        u[m + 1][w] = got;
    }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, (lane & 2) ? u[x][w] : u[x + 2][w], 2);
      if (lane & 2)
        u[x][w] = got;
      else
        u[x + 2][w] = got;
    }
#pragma unroll
  for (int v = 0; v < 4; ++v) {  // now unit lane % 4 of the v-th of the four lanes' rows
    const int row = (lane & ~3) + v;
    if (row < rows)
      __stcs(reinterpret_cast<uint4*>(dst + static_cast<int64_t>(row) * stride + 8 * (lane & 3)),
             make_uint4(u[v][0], u[v][1], u[v][2], u[v][3]));
  }
}

// N fp32 columns of a warp's 32 accumulator rows times `f`, as bf16, to `dst` (see bwd_put32).
template <int N>
__device__ __forceinline__ void bwd_store_rows(uint32_t taddr, __nv_bfloat16* dst, int stride, int rows, float f) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t ov[32], pk[16];
    tmem_ld32(taddr + c, ov);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * f, __uint_as_float(ov[2 * e + 1]) * f);
    bwd_put32(pk, dst + c, stride, rows);
  }
}

// The same columns in fp32 to a part's room for this warp: [N / 4][32 lanes][4].
template <int N>
__device__ __forceinline__ void bwd_store_part(uint32_t taddr, float* dst) {
  float4* d4 = reinterpret_cast<float4*>(dst) + (threadIdx.x & 31);
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    uint32_t ov[32];
    tmem_ld32(taddr + c, ov);
    tmem_wait_ld();
#pragma unroll
    for (int v = 0; v < 8; ++v)
      __stcg(d4 + (c / 4 + v) * 32, make_float4(__uint_as_float(ov[4 * v]), __uint_as_float(ov[4 * v + 1]),
                                                __uint_as_float(ov[4 * v + 2]), __uint_as_float(ov[4 * v + 3])));
  }
}

// The sum of n parts' columns, `step` floats apart, in order, times `f`, as bf16, to `dst`.
template <int N>
__device__ __forceinline__ void bwd_sum_parts(const float* src, int n, int64_t step, __nv_bfloat16* dst, int stride,
                                              int rows, float f) {
#pragma unroll 1
  for (int c = 0; c < N; c += 32) {
    float4 a[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) a[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const float4* s4 = reinterpret_cast<const float4*>(src + i * step) + c * 8 + (threadIdx.x & 31);
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float4 x = __ldcg(s4 + v * 32);
        a[v].x += x.x, a[v].y += x.y, a[v].z += x.z, a[v].w += x.w;
      }
    }
    uint32_t pk[16];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      pk[2 * v] = pack_bf16x2(a[v].x * f, a[v].y * f);
      pk[2 * v + 1] = pack_bf16x2(a[v].z * f, a[v].w * f);
    }
    bwd_put32(pk, dst + c, stride, rows);
  }
}

// ------------------------------------------------------------------------ the kernel
//
// Items: every (head, KV block) for dK and dV, then every (head, query block) for dQ, taken in
// order from a counter, so that a CTA whose list was short takes the next item sooner and the
// dQ items fill the end of the dK/dV ones. Lists of KV blocks differ in length by a factor of ten (every
// query block keeps the text blocks): one with more entries than an SM's share of all is split into parts
// that go first, each storing its fp32 sums; the warp that stores a row range last adds the parts up in
// order (4 heads, 4,133 queries in 64-token blocks: 67 us, 82 us without; 1 head, 8,192 queries: 65 us,
// 112 us). The load thread takes the items and hands them to the other warps through two slots.
//
// dK, dV. Tensor memory: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [384,384+D): rows are KV
// tokens. Issue order for tile n of an item:
//   dV += P^T(n) dO(n);  S^T(n+1) = K Q(n+1)^T;  dK += dS^T(n) Q(n);  dP^T(n+1) = V dO(n+1)^T.
// The softmax warps work on dS(n) while dV(n) and S(n+1) run, and on P(n+1) while dK(n) and
// dP(n+1) run, so S, dP and the two accumulators need one buffer each (all 512 columns).
// S(n+1) may overwrite P(n): tcgen05.mma of one thread run in order.
//
// dQ. Tensor memory: S [0,128), dP [128,256), Q and dO as bf16 pairs [256,256+D), dQ [384,384+D): rows
// are query tokens. Issue order per tile n:
//   S(n+1) = Q K(n+1)^T once S(n) is in registers;  dQ += dS(n) K(n);  dP(n+1) = dO V(n+1)^T,
// with dS(n) over dP(n), in its halves' own columns. The exponentials of tile n+1 run beside dQ(n) and
// dP(n+1). Q and dO are operands of every tile: from tensor memory they cost no shared-memory
// bandwidth, which a product with both operands in shared memory takes whole (128 bytes a cycle) while
// the tiles' copies need a share of it. Four heads of the 720p final scale, back to back at the power
// cap: 5.98 ms, with Q and dO read from shared memory 6.16 ms. K and V of the dK/dV items find no room
// there beside two accumulators; steps of 64 query rows would make it, but their barriers cost more
// (6.32 ms against 5.91 ms on the same GPU).
//
// Between the two a CTA hands its shared memory over when its last dK/dV product is done and its
// tensor memory when the last dV and dK rows have been read.
template <int D, int B>
__global__ void __launch_bounds__(BwdConfig<D, B>::kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ BwdMaps maps, const BwdParams p) {
  using C = BwdConfig<D, B>;
  constexpr int BPT = C::kBlocksPerTile;
  constexpr uint32_t TB = C::kTileBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* held0 = smem;                                // K, or Q
  uint8_t* held1 = smem + TB;                           // V, or dO
  uint8_t* ring_a = smem + 2 * TB;                      // Q, or K
  uint8_t* ring_b = ring_a + C::kStagesA * TB;          // dO, or V
  uint8_t* st_ring = ring_b + C::kStagesB * TB;         // lse and delta of the walked query rows
  BwdBars* bars = reinterpret_cast<BwdBars*>(st_ring + C::kStagesStat * C::kStatBytes);
  BwdPhaseBars* bk = &bars->dkv;
  BwdPhaseBars* bq = &bars->dq;
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
  griddep_wait();  // row statistics, lists and the item counter come from the kernels before
  const int n_all = p.n_dkv + p.n_dq;
  constexpr uint32_t kS = 0, kDPk = 128, kDV = 256, kDK = 384;  // dK, dV items
  constexpr uint32_t kDPq = 128, kQ = 256, kDO = 256 + D / 2, kDQ = 384;  // dQ items

  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, p.status));
  };
  // The k-th item of this CTA, for the warps that do not take it themselves.
  auto next_item = [&](uint32_t k, int* item, int* n_ent, int* part) -> bool {
    if (!wait_all(&bars->item_full[k & 1u], (k >> 1) & 1u)) return false;
    *item = *const_cast<volatile int32_t*>(&bars->item[k & 1u]);
    *n_ent = *const_cast<volatile int32_t*>(&bars->n_ent[k & 1u]);
    *part = *const_cast<volatile int32_t*>(&bars->part[k & 1u]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[k & 1u]);
    return true;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsProducer));
    if (warp == C::kLoadWarp) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        const uint64_t pol_held = l2_policy_evict_first(), pol_walk = l2_policy_evict_last();
        uint32_t tk = 0, tq = 0, hk = 0, hq = 0;  // tiles and held pairs loaded in either phase
        // A tile of one operand, from the blocks blk[0..BPT).
        auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, const int (&blk)[BPT], int h) {
          mbar_arrive_expect_tx(bar, TB);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
            for (int b = 0; b < BPT; ++b)
              tma_load_3d_hint(smem_u32(dst) + c * C::kChunkBytes + b * C::kBoxBytes, map, bar, c * 64, blk[b] * B, h,
                               pol_walk);
        };
        auto load_held = [&](BwdPhaseBars* pb, uint32_t n, const CUtensorMap* m0, const CUtensorMap* m1, int blk,
                             int h) -> bool {
          if (!mbar_wait(&pb->held_empty, (n & 1u) ^ 1u, abort_flag, p.status)) return false;
          mbar_arrive_expect_tx(&pb->held_full, 2 * TB);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            tma_load_3d_hint(smem_u32(held0) + c * C::kChunkBytes, m0, &pb->held_full, c * 64, blk * B, h, pol_held);
            tma_load_3d_hint(smem_u32(held1) + c * C::kChunkBytes, m1, &pb->held_full, c * 64, blk * B, h, pol_held);
          }
          return true;
        };
        bool ok = true, in_dq = false;
        const int n_parts = __ldg(p.next + 1);
        int drawn = atomicAdd(p.next, 1);
        for (uint32_t k = 0; ok; ++k) {
          int item, n_ent, h, blk;
          const int32_t* list;
          // The parts of long lists, then the other items in order.
          for (;; drawn = atomicAdd(p.next, 1)) {
            const bool part = drawn < n_parts;
            item = part ? __ldg(&p.parts[drawn].item) : drawn - n_parts;
            n_ent = h = blk = 0;
            list = nullptr;
            if (item >= p.n_dkv) break;
            h = item / p.nkb;
            blk = item - h * p.nkb;
            const int32_t* at = p.col_at + static_cast<int64_t>(h) * (p.nkb + 1) + blk;
            const int a = __ldg(at);
            n_ent = __ldg(at + 1) - a;
            list = p.col_row + static_cast<int64_t>(h) * p.nqb * p.kmax + a;
            if (part) {
              list += __ldg(&p.parts[drawn].first);
              n_ent = __ldg(&p.parts[drawn].count);
            } else if (n_ent > p.part_ent) {
              continue;
            }
            break;
          }
          if (item >= p.n_dkv && item < n_all) {
            const int iq = item - p.n_dkv;
            h = iq / p.nqb;
            blk = iq - h * p.nqb;
            n_ent = bwd_count(__ldg(p.cnt + iq), p.kmax);
            list = p.idx + static_cast<int64_t>(iq) * p.kmax;
          }
          const int n_tiles = (n_ent + BPT - 1) / BPT;
          const int part = drawn < n_parts ? drawn : -1;
          int taken = -1;  // the item after this one, drawn in time: at once, or with this one's last tile
          if (n_tiles == 0 && item < n_all) taken = atomicAdd(p.next, 1);
          if (!mbar_wait(&bars->item_empty[k & 1u], ((k >> 1) & 1u) ^ 1u, abort_flag, p.status)) break;
          *const_cast<volatile int32_t*>(&bars->item[k & 1u]) = item;
          *const_cast<volatile int32_t*>(&bars->n_ent[k & 1u]) = n_ent;
          *const_cast<volatile int32_t*>(&bars->part[k & 1u]) = part;
          mbar_arrive(&bars->item_full[k & 1u]);
          if (item >= n_all) break;
          if (item < p.n_dkv) {
            if (n_tiles > 0) {
              if (!(ok = load_held(bk, hk, &maps.held[2], &maps.held[3], blk, h))) break;
              ++hk;
            }
            for (int n = 0; n < n_tiles; ++n, ++tk) {
              if (n == n_tiles - 1) taken = atomicAdd(p.next, 1);
              int qb[BPT];
#pragma unroll
              for (int b = 0; b < BPT; ++b) {
                const int e = n * BPT + b;
                qb[b] = __ldg(list + (e < n_ent ? e : n * BPT));
              }
              const uint32_t sa = tk % C::kStagesA, sb = tk % C::kStagesB;
              if (!(ok = mbar_wait(&bk->st_empty[sb], ((tk / 2) & 1u) ^ 1u, abort_flag, p.status))) break;
              mbar_arrive_expect_tx(&bk->st_full[sb], C::kStatBytes);
              const uint32_t st = smem_u32(st_ring) + sb * C::kStatBytes;
#pragma unroll
              for (int b = 0; b < BPT; ++b) {
                const int64_t at = (static_cast<int64_t>(h) * p.nqb + qb[b]) * B;
                bulk_load(st + b * B * 4, p.neg_lse2 + at, B * 4, &bk->st_full[sb]);
                bulk_load(st + 512 + b * B * 4, p.neg_delta + at, B * 4, &bk->st_full[sb]);
              }
              if (!(ok = mbar_wait(&bk->a_empty[sa], ((tk / C::kStagesA) & 1u) ^ 1u, abort_flag, p.status))) {
                bwd_drain(&bk->st_full[sb], (tk / 2) & 1u);
                break;
              }
              load_tile(ring_a + sa * TB, &maps.walk[0], &bk->a_full[sa], qb, h);
              if (!(ok = mbar_wait(&bk->b_empty[sb], ((tk / C::kStagesB) & 1u) ^ 1u, abort_flag, p.status))) {
                bwd_drain(&bk->st_full[sb], (tk / 2) & 1u);
                bwd_drain(&bk->a_full[sa], (tk / C::kStagesA) & 1u);
                break;
              }
              load_tile(ring_b + sb * TB, &maps.walk[1], &bk->b_full[sb], qb, h);
            }
          } else {
            if (!in_dq) {  // the last dK/dV product has read its tiles
              in_dq = true;
              if (!(ok = mbar_wait(&bars->smem_free, 0u, abort_flag, p.status))) break;
            }
            if (!(ok = load_held(bq, hq, &maps.held[0], &maps.held[1], blk, h))) break;
            ++hq;
            for (int n = 0; n < n_tiles; ++n, ++tq) {
              if (n == n_tiles - 1) taken = atomicAdd(p.next, 1);
              int jb[BPT];
#pragma unroll
              for (int b = 0; b < BPT; ++b) {
                const int e = n * BPT + b;
                jb[b] = bwd_block(__ldg(list + (e < n_ent ? e : n * BPT)), p.nkb);
              }
              const uint32_t sa = tq % C::kStagesA, sb = tq % C::kStagesB;
              if (!(ok = mbar_wait(&bq->a_empty[sa], ((tq / C::kStagesA) & 1u) ^ 1u, abort_flag, p.status))) break;
              load_tile(ring_a + sa * TB, &maps.walk[2], &bq->a_full[sa], jb, h);
              if (!(ok = mbar_wait(&bq->b_empty[sb], ((tq / C::kStagesB) & 1u) ^ 1u, abort_flag, p.status))) {
                bwd_drain(&bq->a_full[sa], (tq / C::kStagesA) & 1u);
                break;
              }
              load_tile(ring_b + sb * TB, &maps.walk[3], &bq->b_full[sb], jb, h);
            }
          }
          drawn = taken;
        }
        // every copy lands before the CTA exits (matters only after an abort)
        if (hk > 0) bwd_drain(&bk->held_full, (hk - 1) & 1u);
        if (hq > 0) bwd_drain(&bq->held_full, (hq - 1) & 1u);
        bwd_drain_ring(bk->st_full, 2, tk);
        bwd_drain_ring(bk->a_full, C::kStagesA, tk);
        bwd_drain_ring(bk->b_full, C::kStagesB, tk);
        bwd_drain_ring(bq->a_full, C::kStagesA, tq);
        bwd_drain_ring(bq->b_full, C::kStagesB, tq);
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // K-major views of every tile, and the MN-major ones of the walked tiles
      const uint64_t h0 = smem_desc_sw128(smem_u32(held0), 16, 1024);
      const uint64_t h1 = smem_desc_sw128(smem_u32(held1), 16, 1024);
      const uint64_t ra = smem_desc_sw128(smem_u32(ring_a), 16, 1024);
      const uint64_t rb = smem_desc_sw128(smem_u32(ring_b), 16, 1024);
      const uint64_t ra_mn = smem_desc_sw128(smem_u32(ring_a), C::kChunkBytes, 1024);
      const uint64_t rb_mn = smem_desc_sw128(smem_u32(ring_b), C::kChunkBytes, 1024);
      auto product = [&](uint32_t d, uint64_t a, uint64_t b) {  // 128 x 128 over D
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
          mma_ss(d, a + off, b + off, C::kIdescS, kk > 0 ? 1u : 0u);
        }
      };
      auto gather = [&](uint32_t d, uint32_t a, uint64_t b, bool add) {  // 128 x D over 128 rows
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(d, a + bwd_a_col(kk), b + ((kk * 2048) >> 4), C::kIdescAcc, (add || kk > 0) ? 1u : 0u);
      };
      auto stage_of = [&](uint32_t st) { return static_cast<uint64_t>((st * TB) >> 4); };
      uint32_t tk = 0, tq = 0, hk = 0, hq = 0;
      bool ok = true, in_dq = false;
      auto k_issue_s = [&](uint32_t u) -> bool {
        const uint32_t sa = u % C::kStagesA;
        if (!wait_all(&bk->a_full[sa], (u / C::kStagesA) & 1u)) return false;
        if (elect_one()) {
          product(tmem + kS, h0, ra + stage_of(sa));
          mma_commit(&bk->s_full);
        }
        __syncwarp();
        return true;
      };
      auto k_issue_dp = [&](uint32_t u, bool last) -> bool {
        const uint32_t sb = u % C::kStagesB;
        if (!wait_all(&bk->b_full[sb], (u / C::kStagesB) & 1u)) return false;
        if (elect_one()) {
          product(tmem + kDPk, h1, rb + stage_of(sb));
          mma_commit(&bk->dp_full);
          if (last) mma_commit(&bk->held_empty);
        }
        __syncwarp();
        return true;
      };
      auto product_t = [&](uint32_t d, uint32_t a, uint64_t b) {  // the same, A in tensor memory
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ts(d, a + 8 * kk, b + (((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4), C::kIdescS, kk > 0 ? 1u : 0u);
      };
      auto q_issue_s = [&](uint32_t u) -> bool {
        const uint32_t sa = u % C::kStagesA;
        if (!wait_all(&bq->a_full[sa], (u / C::kStagesA) & 1u)) return false;
        if (elect_one()) {
          product_t(tmem + kS, tmem + kQ, ra + stage_of(sa));
          mma_commit(&bq->s_full);
        }
        __syncwarp();
        return true;
      };
      auto q_issue_dp = [&](uint32_t u) -> bool {
        const uint32_t sb = u % C::kStagesB;
        if (!wait_all(&bq->b_full[sb], (u / C::kStagesB) & 1u)) return false;
        if (elect_one()) {
          product_t(tmem + kDPq, tmem + kDO, rb + stage_of(sb));
          mma_commit(&bq->dp_full);
          mma_commit(&bq->b_empty[sb]);
        }
        __syncwarp();
        return true;
      };
      for (uint32_t k = 0; ok; ++k) {
        int item, n_ent, part;
        if (!next_item(k, &item, &n_ent, &part) || item >= n_all) break;
        const int n_tiles = (n_ent + BPT - 1) / BPT;
        if (item < p.n_dkv) {
          if (n_tiles == 0) continue;
          if (!(ok = wait_all(&bk->held_full, hk & 1u))) break;
          ++hk;
          ok = k_issue_s(tk) && k_issue_dp(tk, n_tiles == 1);
          for (int n = 0; ok && n < n_tiles; ++n, ++tk) {
            const bool last = n == n_tiles - 1;
            const uint32_t sa = tk % C::kStagesA, sb = tk % C::kStagesB;
            if (!(ok = wait_all(&bk->p_full, tk & 1u))) break;
            tc_fence_after();
            if (elect_one()) {
              gather(tmem + kDV, tmem + kS, rb_mn + stage_of(sb), n > 0);
              mma_commit(&bk->b_empty[sb]);
            }
            __syncwarp();
            if (!last && !(ok = k_issue_s(tk + 1))) break;
            if (!(ok = wait_all(&bk->ds_full, tk & 1u))) break;
            tc_fence_after();
            if (elect_one()) {
              gather(tmem + kDK, tmem + kDPk, ra_mn + stage_of(sa), n > 0);
              mma_commit(&bk->a_empty[sa]);
              mma_commit(&bk->st_empty[sb]);
              if (last) mma_commit(&bk->acc_full);
            }
            __syncwarp();
            if (!last && !(ok = k_issue_dp(tk + 1, n == n_tiles - 2))) break;
          }
        } else {
          if (!in_dq) {
            in_dq = true;
            if (elect_one()) mma_commit(&bars->smem_free);
            __syncwarp();
            if (!(ok = wait_all(&bars->tmem_free, 0u))) break;
            tc_fence_after();
          }
          if (!(ok = wait_all(&bq->hold_tm, hq & 1u))) break;
          ++hq;
          tc_fence_after();
          ok = q_issue_s(tq) && q_issue_dp(tq);
          for (int n = 0; ok && n < n_tiles; ++n, ++tq) {
            const bool last = n == n_tiles - 1;
            if (!last) {
              if (!(ok = wait_all(&bq->s_read, tq & 1u))) break;
              tc_fence_after();
              if (!(ok = q_issue_s(tq + 1))) break;
            }
            if (!(ok = wait_all(&bq->ds_full, tq & 1u))) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t sa = tq % C::kStagesA;
              gather(tmem + kDQ, tmem + kDPq, ra_mn + stage_of(sa), n > 0);
              mma_commit(&bq->a_empty[sa]);
              if (last) mma_commit(&bq->acc_full);
            }
            __syncwarp();
            if (!last && !(ok = q_issue_dp(tq + 1))) break;
          }
        }
      }
      if (elect_one()) mma_commit(&bars->drain);
      __syncwarp();
      bwd_drain(&bars->drain, 0);
      __syncwarp();
    }  // warps 10 and 11 only complete the warpgroup
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // ---------------------------------------------------------- P, dS and the epilogues
    // One arrival for the warp, after every lane's accesses.
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int half = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;  // row of the held block: KV token, or query token
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    // With 64-token blocks rows 64-127 of a held tile belong to the next block: whatever stands
    // in their rows of P and dS only reaches accumulator rows that are never stored.
    const bool idle = B < 128 && wq * 32 >= B;
    const bool ragged_kv = p.n_kv % B != 0;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t tk = 0, tq = 0, hq = 0, dk_done = 0, dq_done = 0;
    bool ok = true, in_dq = false;
    for (uint32_t k = 0; ok; ++k) {
      int item, n_ent, part;
      if (!next_item(k, &item, &n_ent, &part) || item >= n_all) break;
      const int n_tiles = (n_ent + BPT - 1) / BPT;
      if (item < p.n_dkv) {
        const int h = item / p.nkb, blk = item - h * p.nkb;
        const int64_t tok = static_cast<int64_t>(blk) * B, left = p.n_kv - tok;
        const int rows = left < B ? static_cast<int>(left) : B;  // of this block
        __nv_bfloat16* dst = (half == 0 ? p.dv : p.dk) + (static_cast<int64_t>(h) * p.n_kv + tok) * D;
        if (n_tiles == 0) {  // a block that no query block keeps
          for (int c = row; c < rows * (D / 8); c += 128) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0u, 0u, 0u, 0u);
          continue;
        }
        dst += wq * 32 * D;
        const uint32_t t_s = tmem + lane_off + kS + 64 * half, t_dp = tmem + lane_off + kDPk + 64 * half;
        for (int n = 0; n < n_tiles; ++n, ++tk) {
          const uint32_t sb = tk & 1u;
          const float4* lse = reinterpret_cast<const float4*>(st_ring + sb * C::kStatBytes + half * 256);
          const float4* del = reinterpret_cast<const float4*>(st_ring + sb * C::kStatBytes + 512 + half * 256);
          if (!(ok = wait_all(&bk->st_full[sb], (tk >> 1) & 1u))) break;
          if (!(ok = wait_all(&bk->s_full, tk & 1u))) break;
          if (idle) {
            arrive(&bk->p_full);
            if (!(ok = wait_all(&bk->dp_full, tk & 1u))) break;
            arrive(&bk->ds_full);
            continue;
          }
          tc_fence_after();
          uint32_t r[2][32];
          float2 pr[32];
          bwd_load_half(t_s, r);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float4 l = lse[e];
            pr[2 * e] = bwd_exp(bwd_pair(r, 2 * e), scale2, make_float2(l.x, l.y));
            pr[2 * e + 1] = bwd_exp(bwd_pair(r, 2 * e + 1), scale2, make_float2(l.z, l.w));
          }
          if (BPT > 1 && half == 1 && 2 * n + 1 >= n_ent) {  // odd last entry: its half repeats a block
#pragma unroll
            for (int e = 0; e < 32; ++e) pr[e] = make_float2(0.f, 0.f);
          }
          bwd_store_half(t_s, pr);
          tmem_wait_st();
          arrive(&bk->p_full);
          if (!(ok = wait_all(&bk->dp_full, tk & 1u))) break;
          tc_fence_after();
          bwd_load_half(t_dp, r);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float4 l = del[e];
            pr[2 * e] = __fmul2_rn(pr[2 * e], __fadd2_rn(bwd_pair(r, 2 * e), make_float2(l.x, l.y)));
            pr[2 * e + 1] = __fmul2_rn(pr[2 * e + 1], __fadd2_rn(bwd_pair(r, 2 * e + 1), make_float2(l.z, l.w)));
          }
          bwd_store_half(t_dp, pr);
          tmem_wait_st();
          arrive(&bk->ds_full);
        }
        if (!ok) break;
        if (!(ok = wait_all(&bk->acc_full, dk_done & 1u))) break;
        ++dk_done;
        tc_fence_after();
        const uint32_t acc = tmem + lane_off + (half == 0 ? kDV : kDK);
        const float f = half == 0 ? 1.f : p.scale;
        if (!idle && part < 0) bwd_store_rows<D>(acc, dst, D, rows - wq * 32, f);
        if (!idle && part >= 0) {
          // The warp's rows of this part, and, where it is the last of the list's parts to store them, the
          // sum of all parts in their order. No one waits for another.
          const BwdPart bp = p.parts[part];
          const int64_t room = (half * B + wq * 32) * D;  // of this warp in a part's sums
          bwd_store_part<D>(acc, p.part_sum + static_cast<int64_t>(part) * 2 * B * D + room);
          __threadfence();
          __syncwarp();
          int before = 0;
          if (lane == 0) before = atomicAdd(p.part_done + bp.base * 8 + warp, 1);
          if (__shfl_sync(0xFFFFFFFFu, before, 0) == bp.n - 1) {
            __threadfence();
            bwd_sum_parts<D>(p.part_sum + static_cast<int64_t>(bp.base) * 2 * B * D + room, bp.n,
                             static_cast<int64_t>(2) * B * D, dst, D, rows - wq * 32, f);
          }
        }
        tc_fence_before();
      } else {
        const int iq = item - p.n_dkv, h = iq / p.nqb, blk = iq - h * p.nqb;
        if (!in_dq) {
          in_dq = true;
          arrive(&bars->tmem_free);
          if (!(ok = wait_all(&bars->tmem_free, 0u))) break;  // Q and dO go where others read dV
          tc_fence_after();
        }
        const int32_t* list = p.idx + static_cast<int64_t>(iq) * p.kmax;
        float2 neg_lse = make_float2(0.f, 0.f), neg_delta = make_float2(0.f, 0.f);
        if (row < B) {
          const int64_t at = static_cast<int64_t>(iq) * B + row;
          neg_lse.x = neg_lse.y = __ldg(p.neg_lse2 + at);
          neg_delta.x = neg_delta.y = __ldg(p.neg_delta + at);
        }
        // Q (first half of the warps) and dO (second half) from shared to tensor memory, a row a thread.
        // The products of the item before have read the old ones: its accumulator was waited for.
        if (!(ok = wait_all(&bq->held_full, hq & 1u))) break;
        ++hq;
        if (!idle) {
          const uint8_t* src = (half == 0 ? held0 : held1) + row * 128;
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + c * C::kChunkBytes + ((u ^ (row & 7)) << 4));
              w[4 * u] = x.x, w[4 * u + 1] = x.y, w[4 * u + 2] = x.z, w[4 * u + 3] = x.w;
            }
            tmem_st32(tmem + lane_off + (half == 0 ? kQ : kDO) + 32 * c, w);
          }
          tmem_wait_st();
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // reads are done before the next copy lands
        arrive(&bq->held_empty);
        arrive(&bq->hold_tm);
        const uint32_t t_s = tmem + lane_off + kS + 64 * half, t_dp = tmem + lane_off + kDPq + 64 * half;
        for (int n = 0; n < n_tiles; ++n, ++tq) {
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
          if (!(ok = wait_all(&bq->s_full, tq & 1u))) break;
          if (idle) {
            arrive(&bq->s_read);
            if (!(ok = wait_all(&bq->dp_full, tq & 1u))) break;
            arrive(&bq->ds_full);
            continue;
          }
          tc_fence_after();
          uint32_t r[2][32];
          float2 pr[32];
          bwd_load_half(t_s, r);
          arrive(&bq->s_read);
#pragma unroll
          for (int e = 0; e < 32; ++e) pr[e] = bwd_exp(bwd_pair(r, e), scale2, neg_lse);
          if (nv < 64) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (2 * e >= nv) pr[e].x = 0.f;
              if (2 * e + 1 >= nv) pr[e].y = 0.f;
            }
          }
          if (!(ok = wait_all(&bq->dp_full, tq & 1u))) break;
          tc_fence_after();
          bwd_load_half(t_dp, r);
#pragma unroll
          for (int e = 0; e < 32; ++e) pr[e] = __fmul2_rn(pr[e], __fadd2_rn(bwd_pair(r, e), neg_delta));
          bwd_store_half(t_dp, pr);
          tmem_wait_st();
          arrive(&bq->ds_full);
        }
        if (!ok) break;
        if (!(ok = wait_all(&bq->acc_full, dq_done & 1u))) break;
        ++dq_done;
        tc_fence_after();
        if (!idle) {
          const int64_t tok = static_cast<int64_t>(blk) * B + wq * 32, left = p.n_q - tok;
          bwd_store_rows<D / 2>(tmem + lane_off + kDQ + (D / 2) * half,
                                p.dq + (static_cast<int64_t>(h) * p.n_q + tok) * D + (D / 2) * half, D,
                                left < 32 ? static_cast<int>(left) : 32, p.scale);
        }
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------------ preparation
//
// bwd_prep_kernel, in one launch:
//   rows: -lse log2(e) and -delta = -do . o of every query row, padded to whole blocks (-inf and 0
//   past n_q: such a row's P is 0), so that a block's statistics are one aligned copy. One read of
//   o and do, D / 8 lanes a row; memory-bound.
//   masks: for each (chunk of 32 query-block rows, head), one word per KV block with the rows that
//   keep it. A chunk where a row lists a block twice is noted in `twice`, and its words are how often
//   each block is listed instead (the forward pass attends to it twice, so it counts twice).
// bwd_lists_kernel, one CTA per head: the query blocks of each KV block, ascending. Counts are
// scanned over chunks and blocks, then every word places its rows. The rows of a chunk with a block
// listed twice are placed from their lists, by one warp, row after row, each block's place counting up;
// which lane takes which of a row's equal entries changes nothing (1 head, 1,000 rows of 200 of 2,000
// blocks, one of them repeated in every chunk: the call takes 2.06 ms, 1.91 ms where none is; with a search
// of the chunk's lists for every block 47 ms). Out-of-range entries are clamped as the forward pass clamps
// them, and recorded.
constexpr int kMaskRows = 32;
constexpr int kMaskMaxBlocks = 49152;  // KV blocks at most: one 4-byte word each in shared memory

struct BwdPrep {
  const __nv_bfloat16 *o, *d_o;
  const float* lse;
  const int32_t *idx, *cnt;
  float *neg_lse2, *neg_delta;
  uint32_t* words;   // [H, chunks, nkb] the rows that keep a block, or (twice) how often it is listed
  int32_t* place;    // [H, chunks, nkb] place of each word's first (twice: next) row within its KV block
  int32_t* twice;    // [H, chunks]
  int32_t *col_at, *col_row;
  BwdPart* parts;
  int* next;       // the item counter, and the number of parts
  int* part_done;  // [kBwdMaxParts][8]
  unsigned* status;
  int part_ent;
  int64_t n_q, n_pad;
  int heads, nqb, nkb, kmax, n_chunks;
};

template <int D>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const BwdPrep p) {
  extern __shared__ uint32_t words[];
  __shared__ int32_t counts[kMaskRows];
  __shared__ int32_t twice;
  griddep_launch_dependents();
  const int n_mask = p.n_chunks * p.heads;
  if (blockIdx.x == 0) {  // the counters of this call
    if (threadIdx.x < 2) p.next[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < kBwdMaxParts * 8; i += 256) p.part_done[i] = 0;
  }
  if (static_cast<int>(blockIdx.x) < n_mask) {
    const int h = blockIdx.x / p.n_chunks, chunk = blockIdx.x - h * p.n_chunks;
    const int64_t row0 = static_cast<int64_t>(h) * p.nqb + chunk * kMaskRows;
    const int rows = min(kMaskRows, p.nqb - chunk * kMaskRows);
    for (int j = threadIdx.x; j < p.nkb; j += 256) words[j] = 0u;
    if (threadIdx.x < rows) {
      const int c0 = __ldg(p.cnt + row0 + threadIdx.x), c = bwd_count(c0, p.kmax);
      if (c != c0) atomicOr(p.status, kStatusBounds);
      counts[threadIdx.x] = c;
    }
    if (threadIdx.x == 0) twice = 0;
    __syncthreads();
    // f(row, block) of every entry, four in flight per thread
    const uint32_t kmax = p.kmax, total = rows * kmax;  // at most nqb * kmax: 31 bits
    auto entries = [&](auto f) {
      for (uint32_t i0 = threadIdx.x; i0 < total; i0 += 4 * 256) {
        int j[4], r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t i = i0 + u * 256;
          r[u] = i < total ? static_cast<int>(i / kmax) : -1;
          if (r[u] >= 0 && static_cast<int>(i - r[u] * kmax) < counts[r[u]])
            j[u] = __ldg(p.idx + row0 * p.kmax + i);
          else
            r[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r[u] >= 0) f(r[u], j[u]);
      }
    };
    entries([&](int r, int j) {
      const int jc = bwd_block(j, p.nkb);
      if (jc != j) atomicOr(p.status, kStatusBounds);
      if ((atomicOr(&words[jc], 1u << r) >> r) & 1u) twice = 1;
    });
    __syncthreads();
    if (twice) {
      for (int j = threadIdx.x; j < p.nkb; j += 256) words[j] = 0u;
      __syncthreads();
      entries([&](int, int j) { atomicAdd(&words[bwd_block(j, p.nkb)], 1u); });
      __syncthreads();
    }
    uint32_t* out = p.words + static_cast<int64_t>(blockIdx.x) * p.nkb;
    for (int j = threadIdx.x; j < p.nkb; j += 256) out[j] = words[j];
    if (threadIdx.x == 0) p.twice[blockIdx.x] = twice;
    return;
  }
  constexpr int G = D / 8, kRows = 256 / G;
  const int l = threadIdx.x % G;
  const int64_t tiles = (p.n_pad + kRows - 1) / kRows, all = tiles * p.heads;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) - n_mask; t < all; t += gridDim.x - n_mask) {
    const int64_t h = t / tiles, row = (t - h * tiles) * kRows + threadIdx.x / G;
    float s = 0.f;
    if (row < p.n_q) {
      const int64_t at = (h * p.n_q + row) * D + 8 * l;
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p.o + at));
      const uint4 b = __ldcs(reinterpret_cast<const uint4*>(p.d_o + at));
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
        s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
      }
    }
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (l == 0 && row < p.n_pad) {
      p.neg_lse2[h * p.n_pad + row] =
          row < p.n_q ? __ldg(p.lse + h * p.n_q + row) * -1.4426950408889634f : -INFINITY;
      p.neg_delta[h * p.n_pad + row] = -s;
    }
  }
}

__global__ void __launch_bounds__(1024) bwd_lists_kernel(const BwdPrep p) {
  __shared__ int32_t warp_sum[32];
  __shared__ int32_t base;
  griddep_launch_dependents();
  griddep_wait();
  const int h = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t* words = p.words + static_cast<int64_t>(h) * p.n_chunks * p.nkb;
  int32_t* place = p.place + static_cast<int64_t>(h) * p.n_chunks * p.nkb;
  const int32_t* twice = p.twice + static_cast<int64_t>(h) * p.n_chunks;
  int32_t* at = p.col_at + static_cast<int64_t>(h) * (p.nkb + 1);
  int32_t* rows = p.col_row + static_cast<int64_t>(h) * p.nqb * p.kmax;
  if (threadIdx.x == 0) base = 0;
  for (int j0 = 0; j0 < p.nkb; j0 += 1024) {
    const int j = j0 + threadIdx.x;
    int total = 0;
    if (j < p.nkb)
      for (int c0 = 0; c0 < p.n_chunks; c0 += 8) {
        uint32_t x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = c0 + u < p.n_chunks ? words[static_cast<int64_t>(c0 + u) * p.nkb + j] : 0u;
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (c0 + u < p.n_chunks) {
            place[static_cast<int64_t>(c0 + u) * p.nkb + j] = total;
            total += twice[c0 + u] ? static_cast<int>(x[u]) : __popc(x[u]);
          }
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
    if (j < p.nkb) at[j] = before;
    __syncthreads();
    if (threadIdx.x == 1023) base = before + total;
    __syncthreads();
  }
  if (threadIdx.x == 0) at[p.nkb] = base;
  __syncthreads();
  for (int j = threadIdx.x; j < p.nkb; j += 1024) {
    const int len = at[j + 1] - at[j];
    if (len > p.part_ent) {
      const int n = (len + p.part_ent - 1) / p.part_ent, base_part = atomicAdd(p.next + 1, n);
      for (int k = 0, first = 0; k < n; ++k) {  // as even as whole entries allow
        const int count = (len - first + n - k - 1) / (n - k);
        p.parts[base_part + k] = BwdPart{h * p.nkb + j, first, count, base_part, n};
        first += count;
      }
    }
  }
  const int64_t n_words = static_cast<int64_t>(p.n_chunks) * p.nkb;
  for (int64_t i = threadIdx.x; i < n_words; i += 1024) {
    const int chunk = static_cast<int>(i / p.nkb), j = static_cast<int>(i - static_cast<int64_t>(chunk) * p.nkb);
    if (twice[chunk]) continue;
    uint32_t word = words[i];
    int32_t* out = rows + at[j] + place[i];
    for (; word != 0u; word &= word - 1u) *out++ = chunk * kMaskRows + __ffs(word) - 1;
  }
  for (int chunk = w; chunk < p.n_chunks; chunk += 32) {
    if (!twice[chunk]) continue;
    const int r1 = min(p.nqb, (chunk + 1) * kMaskRows);
    int32_t* next = place + static_cast<int64_t>(chunk) * p.nkb;
    for (int i = chunk * kMaskRows; i < r1; ++i) {
      const int64_t row = static_cast<int64_t>(h) * p.nqb + i;
      const int c = bwd_count(__ldg(p.cnt + row), p.kmax);
#pragma unroll 4
      for (int e = lane; e < c; e += 32) {
        const int j = bwd_block(__ldg(p.idx + row * p.kmax + e), p.nkb);
        rows[at[j] + atomicAdd(next + j, 1)] = i;
      }
      __syncwarp();  // the next row's places come behind this one's
    }
  }
}

}  // namespace sparstar
