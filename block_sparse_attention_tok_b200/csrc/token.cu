// One query token per sequence over a K/V cache: block means, selection, attention.
//
// Per (sequence, key head), with G = heads_q / heads_k query heads that share the key head:
//   score_j = (sum_g q_g) . mean_j      of every block j between the forced ones (fp64: the rank
//                                       of two near scores must not hang on a summation order),
//   kept    = the first n_sink and last n_recent blocks and the best others up to `keep`,
//   o_g     = sum over the kept tokens u of softmax_u(s q_g . k_u) v_u,  lse_g.
// The mean of the G queries ranks as their sum does, so this is the block score of the scale's
// selection with the G heads as the query block.
//
// token_kernel is one launch for all of it. A cluster of C CTAs serves one (sequence, key head):
// each CTA attends to every C-th kept block, and the partial results (max, sum, o of G rows) are
// merged through distributed shared memory: no workspace, no atomics, the same order of additions
// every time. Up to 160 candidates (one a thread) every CTA scores and ranks all of them for itself;
// more are scored by all CTAs into the first one's shared memory, which ranks and writes the list.
// Bound: memory (4 bytes a scored mean value, 4 bytes a kept K/V value, read once). K and V tiles
// come by TMA into a ring of shared-memory stages; the products use mma.sync on 16 rows (G real
// ones): one tile of 64 KB takes the SM about 2,700 cycles to receive and its 256 products a
// fifth of that, so tcgen05 (128 rows, a tensor memory round trip) would save nothing.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "host.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace sparstar {
namespace {

constexpr int kTokThreads = 160;      // 4 product warps and a TMA warp
constexpr int kTokMaxGroup = 16;      // query heads of one key head
constexpr int kTokMaxBlocks = 16384;  // blocks of one sequence whose scores fit shared memory
constexpr int kDigitBins = 256;       // radix select: 8 bits a pass
constexpr int kGather = 128;          // a bucket of at most this many keys is ranked directly

template <int D>
struct TokConfig {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kChunkBytes = 128 * 128;
  static constexpr uint32_t kTileBytes = kChunks * kChunkBytes;  // 128 tokens
  static constexpr int kStages = D == 128 ? 3 : 6;               // 96 KB: two CTAs an SM
  static constexpr uint32_t kRingBytes = kStages * kTileBytes;
};

struct TokParams {
  const __nv_bfloat16* q;   // [B, Hq, d]
  const float* means;       // [B, Hk, nb_cap, d]
  const int32_t* kv_len;    // [B]
  int32_t* idx;             // [B, Hk, keep]
  int32_t* cnt;             // [B, Hk]
  __nv_bfloat16* o;         // [B, Hq, d]
  float* lse;               // [B, Hq] or nullptr
  unsigned* status;
  int64_t capacity;
  int hk, group, nb_cap, keep, n_sink, n_recent;
  float scale_log2;
  uint32_t union_bytes;     // shared memory that scores and ring share
};

// Shared memory behind the ring and the scores.
struct TokFixed {
  uint64_t full[6], empty[6];
  double score[kTokThreads];    // few candidates: scored and ranked by every CTA for itself
  int32_t chosen[kTokThreads];
  int32_t warp_tot[kTokThreads / 32];
  uint32_t abort_flag;
};

// Order-preserving key of a score: NaN lowest, -0 = +0.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (isnan(s)) return 0ull;
  const unsigned long long b = __double_as_longlong(s + 0.0);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared state of the ranking, behind the scores.
struct RankState {
  int32_t hist[kDigitBins];
  unsigned long long keys[kGather];
  int32_t warp_tot[2][kTokThreads / 32];
  unsigned long long cut;
  int32_t need, bucket, count, eq;
};

// Ranks scores[0, n) and writes the `take` best as base + position, ascending, to out. One CTA,
// all threads. Equal scores go to the lower position.
__device__ void rank_and_write(const double* scores, int n, int take, int base, int32_t* out, RankState* st) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  // Radix select of the take-th largest key, from the top digit down, until the bucket that
  // holds it is taken whole or small enough to be ranked by counting.
  unsigned long long prefix = 0ull, mask = 0ull;
  int need = take;
  unsigned long long cut = 0ull;
  int eq = 0;  // how many keys equal to `cut` are taken
  bool done = false, whole = false;  // whole: every key with the cut's looked-at digits is taken
  constexpr int bins = kDigitBins;
  for (int shift = 56; !done; shift -= 8) {
    for (int i = tid; i < bins; i += kTokThreads) st->hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTokThreads) {
      const unsigned long long key = score_key(scores[i]);
      if ((key & mask) == prefix) atomicAdd(&st->hist[(key >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    if (w == 0) {  // the digit at which the count from the top reaches `need`
      constexpr int per = bins / 32;
      int sum = 0;
      for (int i = 0; i < per; ++i) sum += st->hist[bins - 1 - (lane * per + i)];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
      }
      int above = incl - sum;
      if (above < need && need <= incl) {
        for (int i = 0;; ++i) {
          const int b = bins - 1 - (lane * per + i), c = st->hist[b];
          if (above + c >= need) {
            st->bucket = b;
            st->count = c;
            st->need = need - above;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    prefix |= static_cast<unsigned long long>(st->bucket) << shift;
    mask |= static_cast<unsigned long long>(bins - 1) << shift;
    need = st->need;
    const int count = st->count;
    if (count == need) {
      cut = prefix;
      eq = count;
      done = whole = true;
    } else if (shift == 0) {  // equal keys, of which `need` are taken
      cut = prefix;
      eq = need;
      done = true;
    } else if (count <= kGather) {
      __syncthreads();
      if (tid == 0) st->count = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kTokThreads) {
        const unsigned long long key = score_key(scores[i]);
        if ((key & mask) == prefix) st->keys[atomicAdd(&st->count, 1)] = key;
      }
      __syncthreads();
      if (tid < count) {
        const unsigned long long key = st->keys[tid];
        int above = 0, same = 0;
        for (int i = 0; i < count; ++i) {
          above += st->keys[i] > key;
          same += st->keys[i] == key;
        }
        if (above < need && need <= above + same) {  // equal keys write equal values
          st->cut = key;
          st->eq = need - above;
        }
      }
      __syncthreads();
      cut = st->cut;
      eq = st->eq;
      done = true;
    }
    __syncthreads();
  }
  int placed = 0, eq_seen = 0;
  for (int i0 = 0; i0 < n; i0 += kTokThreads) {
    const int i = i0 + tid;
    const unsigned long long key = i < n ? score_key(scores[i]) : 0ull;
    const bool same = i < n && (whole ? (key & mask) == prefix : key == cut);
    const bool more = i < n && !same && key > cut;
    const unsigned bs = __ballot_sync(0xFFFFFFFFu, same);
    if (lane == 0) st->warp_tot[0][w] = __popc(bs);
    __syncthreads();
    int before = eq_seen + __popc(bs & ((1u << lane) - 1u));
    for (int x = 0; x < w; ++x) before += st->warp_tot[0][x];
    const bool take_it = more || (same && before < eq);
    const unsigned bt = __ballot_sync(0xFFFFFFFFu, take_it);
    if (lane == 0) st->warp_tot[1][w] = __popc(bt);
    __syncthreads();
    int pos = placed + __popc(bt & ((1u << lane) - 1u));
    for (int x = 0; x < w; ++x) pos += st->warp_tot[1][x];
    if (take_it) out[pos] = base + i;
    for (int x = 0; x < kTokThreads / 32; ++x) {
      eq_seen += st->warp_tot[0][x];
      placed += st->warp_tot[1][x];
    }
    __syncthreads();
  }
}

// Scores of blocks first, first + step, ... below n (8 lanes a block), each to scores[j]: the sum
// over the group's queries, times the block's mean, in fp64.
template <int D>
__device__ __forceinline__ void score_blocks(const __nv_bfloat16* q, int group, const float* means, int n, int first,
                                             int step, double* scores) {
  constexpr int N = D / 32;  // float4 per lane
  const int l = threadIdx.x & 7;
  double qs[4 * N];
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) qs[i] = 0.0;
  for (int g = 0; g < group; ++g)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(q + g * D + 4 * (l + 8 * i)));
      qs[4 * i] += static_cast<double>(__uint_as_float(v.x << 16));
      qs[4 * i + 1] += static_cast<double>(__uint_as_float(v.x & 0xFFFF0000u));
      qs[4 * i + 2] += static_cast<double>(__uint_as_float(v.y << 16));
      qs[4 * i + 3] += static_cast<double>(__uint_as_float(v.y & 0xFFFF0000u));
    }
  const float4* mean = reinterpret_cast<const float4*>(means) + l;
  for (int j0 = first; j0 < n; j0 += step) {
    const int j = j0 + threadIdx.x / 8;
    double s = 0.0;
    if (j < n) {
      float4 m[N];
#pragma unroll
      for (int i = 0; i < N; ++i) m[i] = __ldg(mean + static_cast<int64_t>(j) * (D / 4) + 8 * i);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s = fma(qs[4 * i], static_cast<double>(m[i].x), s);
        s = fma(qs[4 * i + 1], static_cast<double>(m[i].y), s);
        s = fma(qs[4 * i + 2], static_cast<double>(m[i].z), s);
        s = fma(qs[4 * i + 3], static_cast<double>(m[i].w), s);
      }
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (l == 0 && j < n) scores[j] = s;
  }
}

// At most one candidate a thread: its rank is the number of better ones. The chosen positions go,
// ascending, to chosen. One CTA, all threads, scores written before (and synchronised).
__device__ __forceinline__ void rank_few(const double* scores, int n, int take, int32_t* chosen, int32_t* warp_tot) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const unsigned long long key = tid < n ? score_key(scores[tid]) : 0ull;
  int above = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned long long k = score_key(scores[i]);
    above += k > key || (k == key && i < tid);
  }
  const bool take_it = tid < n && above < take;
  const unsigned b = __ballot_sync(0xFFFFFFFFu, take_it);
  if (lane == 0) warp_tot[w] = __popc(b);
  __syncthreads();
  int pos = __popc(b & ((1u << lane) - 1u));
  for (int x = 0; x < w; ++x) pos += warp_tot[x];
  if (take_it) chosen[pos] = tid;
}

// SEL: choose the blocks (idx, cnt are written). ATT: attend to them (with SEL to the chosen
// ones, else to the given idx, cnt). grid (C, Hk, B), clusters of C along x.
template <int D, bool SEL, bool ATT>
__global__ void __launch_bounds__(kTokThreads)
    token_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const TokParams p) {
  using C = TokConfig<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, size = gridDim.x;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = static_cast<int64_t>(b) * p.hk + hk;  // (sequence, key head)
  TokFixed* fix = reinterpret_cast<TokFixed*>(smem + p.union_bytes);
  uint64_t *full = fix->full, *empty = fix->empty;
  volatile uint32_t* abort_flag = &fix->abort_flag;

  int64_t len = __ldg(p.kv_len + b);
  if (len < 0 || len > p.capacity) {
    if (tid == 0 && rank == 0 && hk == 0) atomicOr(p.status, kStatusBounds);
    len = len < 0 ? 0 : p.capacity;
  }
  const int nb = static_cast<int>((len + 127) / 128);
  const __nv_bfloat16* q = p.q + row * p.group * D;
  int32_t* list = p.idx + row * p.keep;

  if (ATT && tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    fix->abort_flag = 0u;
    fence_barrier_init();
  }

  // Where the e-th kept block stands: every block (all), forced and chosen ones (few candidates,
  // ranked by every CTA), or the list that the first CTA wrote.
  const int n_cand = nb - p.n_sink - p.n_recent, take = p.keep - p.n_sink - p.n_recent;
  const bool all = SEL && nb <= p.keep, few = SEL && !all && n_cand <= kTokThreads;
  bool synced = false;
  if (SEL && !all && take > 0) {  // 0 < take < n_cand
    const float* means = p.means + (row * p.nb_cap + p.n_sink) * D;
    if (few) {
      score_blocks<D>(q, p.group, means, n_cand, 0, kTokThreads / 8, fix->score);
      __syncthreads();
      rank_few(fix->score, n_cand, take, fix->chosen, fix->warp_tot);
      __syncthreads();
    } else {
      if (size > 1) cluster.sync();  // the first CTA runs before anyone writes to it
      constexpr int kPer = kTokThreads / 8;  // blocks a CTA scores at a time
      score_blocks<D>(q, p.group, means, n_cand, rank * kPer, size * kPer,
                      cluster.map_shared_rank(reinterpret_cast<double*>(smem), 0));
      if (size > 1)
        cluster.sync();
      else
        __syncthreads();
      if (rank == 0) {
        RankState* st = reinterpret_cast<RankState*>(smem + ((static_cast<size_t>(n_cand) * 8 + 15) & ~15ull));
        rank_and_write(reinterpret_cast<const double*>(smem), n_cand, take, p.n_sink, list + p.n_sink, st);
      }
      if (size > 1) {
        cluster.sync();  // the list is written
        synced = true;
      }
    }
  }
  auto kept_at = [&](int e) {  // SEL, unless the list has it
    return all ? e
               : e < p.n_sink ? e
                              : e >= p.keep - p.n_recent ? nb - p.keep + e : p.n_sink + fix->chosen[e - p.n_sink];
  };
  if (SEL && rank == 0) {
    if (all) {
      for (int e = tid; e < p.keep; e += kTokThreads) list[e] = e < nb ? e : -1;
    } else {
      for (int e = tid; e < p.keep; e += kTokThreads)
        if (few || e < p.n_sink || e >= p.keep - p.n_recent) list[e] = kept_at(e);
    }
    if (tid == 0) p.cnt[row] = all ? nb : p.keep;
  }
  if (!ATT) return;
  if (!synced) __syncthreads();  // barriers, the list of a lone CTA

  int n_ent = SEL ? (nb <= p.keep ? nb : p.keep) : __ldg(p.cnt + row);
  if (!SEL && (n_ent < 0 || n_ent > p.keep)) {
    if (tid == 0 && rank == 0) atomicOr(p.status, kStatusBounds);
    n_ent = n_ent < 0 ? 0 : p.keep;
  }
  const int n_mine = n_ent > rank ? (n_ent - rank + size - 1) / size : 0;
  // Block of this CTA's i-th entry, or -1 (recorded) where it names no block that holds tokens.
  auto block_at = [&](int i, bool report) {
    const int e = rank + i * size;
    const int j = SEL && (all || few || e < p.n_sink || e >= p.keep - p.n_recent)
                      ? kept_at(e)
                      : *const_cast<volatile int32_t*>(list + e);
    if (j < 0 || j >= nb) {
      if (report) atomicOr(p.status, kStatusBounds);
      return -1;
    }
    return j;
  };

  constexpr int NT = D / 8;  // 8-column tiles of o
  float acc[NT][4];
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scores lay where tiles go
      uint32_t it = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_mine; ++i) {
        const int j = block_at(i, true);
        if (j < 0) continue;
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t st = it % C::kStages;
          ok = mbar_wait(&empty[st], ((it / C::kStages) & 1u) ^ 1u, abort_flag, p.status);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[st], C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(smem_u32(smem) + st * C::kTileBytes + c * C::kChunkBytes, kv == 0 ? &tm_k : &tm_v, &full[st],
                        c * 64, j * 128, static_cast<int>(row));
        }
      }
      for (uint32_t st = 0; st < C::kStages; ++st)
        if (it > st) {  // every copy lands before the memory is used for something else
          const unsigned long long t0 = globaltimer_ns();
          while (!mbar_try_wait(&full[st], ((it - 1 - st) / C::kStages) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
          }
        }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ products: 32 tokens of each tile
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + 8 * (e & 1), c = 16 * kk + c2 + 8 * (e >> 1);
        qa[kk][e] = r < p.group ? __ldg(reinterpret_cast<const uint32_t*>(q + r * D + c)) : 0u;
      }
    uint32_t it = 0;
    for (int i = 0; i < n_mine; ++i) {
      const int j = block_at(i, false);
      if (j < 0) continue;
      const int64_t left = len - static_cast<int64_t>(j) * 128;
      const int valid = left < 128 ? static_cast<int>(left) : 128;  // tokens of this block
      uint32_t st = it % C::kStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (it / C::kStages) & 1u, abort_flag, p.status))) break;
      ++it;
      float s[4][4];
      const uint32_t kt = smem_u32(smem) + st * C::kTileBytes;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
        const int r = warp * 32 + nt * 8 + (lane & 7);
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {  // 32 columns: four 16-byte units
          const int u = 4 * k2 + (lane >> 3);
          uint32_t kb[4];
          ldsm4(kt + (u >> 3) * C::kChunkBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4), kb);
          mma16816(s[nt], qa[2 * k2], kb[0], kb[1]);
          mma16816(s[nt], qa[2 * k2 + 1], kb[2], kb[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = warp * 32 + nt * 8 + c2 + (e & 1);
          s[nt][e] = t < valid ? s[nt][e] * p.scale_log2 : -INFINITY;  // a cache row past the end may hold anything
          mx[e >> 1] = fmaxf(mx[e >> 1], s[nt][e]);
        }
      float alpha[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xFFFFFFFFu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xFFFFFFFFu, mx[x], 2));
        const float m_new = fmaxf(m_run[x], mx[x]);
        alpha[x] = m_new == -INFINITY ? 1.f : ex2_approx(m_run[x] - m_new);
        m_run[x] = m_new;
        l_run[x] *= alpha[x];
      }
      uint32_t pa[2][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float base = m_run[x] == -INFINITY ? 0.f : m_run[x];
          const float p0 = ex2_approx(s[nt][2 * x] - base), p1 = ex2_approx(s[nt][2 * x + 1] - base);
          l_run[x] += p0 + p1;
          pa[nt >> 1][2 * (nt & 1) + x] = pack_bf16x2(p0, p1);  // P in bf16, as the block attention rounds it
        }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] *= alpha[e >> 1];
      st = it % C::kStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (it / C::kStages) & 1u, abort_flag, p.status))) break;
      ++it;
      const uint32_t vt = smem_u32(smem) + st * C::kTileBytes;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int t0 = warp * 32 + ks * 16;
        const int r = t0 + (lane & 15);
        // P is 0 past the end, but 0 times what the cache holds there need not be: zero it
        uint32_t keep_lo = 0xFFFFFFFFu, keep_hi = 0xFFFFFFFFu;
        if (t0 + 16 > valid) {
          auto pair = [&](int t) { return (t < valid ? 0xFFFFu : 0u) | (t + 1 < valid ? 0xFFFF0000u : 0u); };
          keep_lo = pair(t0 + c2);
          keep_hi = pair(t0 + 8 + c2);
        }
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          const int u = t + (lane >> 4);
          uint32_t vb[4];
          ldsm4t(vt + (u >> 3) * C::kChunkBytes + r * 128 + (((u & 7) ^ (r & 7)) << 4), vb);
          mma16816(acc[t], pa[ks], vb[0] & keep_lo, vb[1] & keep_hi);
          mma16816(acc[t + 1], pa[ks], vb[2] & keep_lo, vb[3] & keep_hi);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
  }
  __syncthreads();  // the ring is free

  // Partial results: [4 warps][16 rows][D] o, then max and sum, then the CTA's own merged rows.
  constexpr int kPad = D + 4;
  float* po = reinterpret_cast<float*>(smem);
  float* pm = po + 4 * 16 * kPad;     // [4][16]
  float* pl = pm + 64;                // [4][16]
  float* co = pl + 64;                // [16][D]
  float* cm = co + 16 * D;            // [16]
  float* cl = cm + 16;                // [16]
  if (warp < 4) {
    const int g = lane >> 2, c2 = 2 * (lane & 3);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float l = l_run[x];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      const int r = g + 8 * x;
      if ((lane & 3) == 0) {
        pm[warp * 16 + r] = m_run[x];
        pl[warp * 16 + r] = l;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<float2*>(po + (warp * 16 + r) * kPad + 8 * t + c2) =
            make_float2(acc[t][2 * x], acc[t][2 * x + 1]);
    }
  }
  __syncthreads();
  for (int i = tid; i < p.group * D; i += kTokThreads) {
    const int r = i / D, c = i - r * D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, pm[w * 16 + r]);
    float v = 0.f, l = 0.f;
    if (m != -INFINITY) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2_approx(pm[w * 16 + r] - m);
        v = fmaf(f, po[(w * 16 + r) * kPad + c], v);
        l = fmaf(f, pl[w * 16 + r], l);
      }
    }
    co[i] = v;
    if (c == 0) {
      cm[r] = m;
      cl[r] = l;
    }
  }
  if (size > 1)
    cluster.sync();
  else
    __syncthreads();
  for (int i = rank * kTokThreads + tid; i < p.group * D; i += size * kTokThreads) {
    const int r = i / D, c = i - r * D;
    float m = -INFINITY;
    for (int x = 0; x < size; ++x) m = fmaxf(m, cluster.map_shared_rank(cm, x)[r]);
    float v = 0.f, l = 0.f;
    if (m != -INFINITY)
      for (int x = 0; x < size; ++x) {
        const float f = ex2_approx(cluster.map_shared_rank(cm, x)[r] - m);
        v = fmaf(f, cluster.map_shared_rank(co, x)[i], v);
        l = fmaf(f, cluster.map_shared_rank(cl, x)[r], l);
      }
    // a sequence with no kept token: o = 0, lse = -inf
    p.o[row * p.group * D + i] = __float2bfloat16_rn(m == -INFINITY ? 0.f : v / l);
    if (c == 0 && p.lse != nullptr)
      p.lse[row * p.group + r] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
  if (size > 1) cluster.sync();  // nobody leaves while its rows are read
}

// Mean of each 128-token block of a cache row, a last one over the tokens it holds. One CTA per
// (block, key head, sequence): 16-byte loads, fp32 sums in a fixed order. Bound by memory.
template <int D>
__global__ void __launch_bounds__(256)
    block_means_kernel(const __nv_bfloat16* __restrict__ k, const int32_t* __restrict__ kv_len, int64_t capacity,
                       int nb_cap, int tail_only, float* __restrict__ means, unsigned* status) {
  constexpr int kChunks = D / 8, kRowGroups = 256 / kChunks, kRows = 128 / kRowGroups;
  __shared__ float part[8][D];
  const int hk = blockIdx.y, b = blockIdx.z;
  int64_t len = __ldg(kv_len + b);
  if (len < 0 || len > capacity) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && hk == 0) atomicOr(status, kStatusBounds);
    len = len < 0 ? 0 : capacity;
  }
  const int64_t j = tail_only ? (len - 1) / 128 : blockIdx.x;
  if (len == 0 || j * 128 >= len) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(128), len - j * 128));
  const int64_t row = static_cast<int64_t>(b) * gridDim.y + hk;
  const int c = threadIdx.x % kChunks, rg = threadIdx.x / kChunks;
  const __nv_bfloat16* src = k + (row * capacity + j * 128) * D + 8 * c;
  uint4 v[kRows];
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    const int r = rg + m * kRowGroups;
    v[m] = r < n ? __ldcs(reinterpret_cast<const uint4*>(src + r * D)) : make_uint4(0u, 0u, 0u, 0u);
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int m = 0; m < kRows; ++m) {
    const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] += __uint_as_float(w[i] << 16);
      acc[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
#pragma unroll
  for (int off = kChunks; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], off);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < kChunks)
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][lane * 8 + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][threadIdx.x];
    means[(row * nb_cap + j) * D + threadIdx.x] = s / static_cast<float>(n);
  }
}

std::mutex g_attr_mutex;
bool g_attrs_set[kMaxDevices];

uint32_t tok_union_bytes(int d, int64_t nb, bool sel, bool att) {
  const uint32_t ring = att ? (d == 128 ? TokConfig<128>::kRingBytes : TokConfig<64>::kRingBytes) : 0;
  const uint32_t rank = sel ? static_cast<uint32_t>(nb * 8 + 16 + sizeof(RankState)) : 0;
  return ((ring > rank ? ring : rank) + 1023u) & ~1023u;
}

template <int D>
int tok_set_attrs() {
  const uint32_t most = tok_union_bytes(D, kTokMaxBlocks, true, true) + 1024 + sizeof(TokFixed);
  for (auto kernel : {token_kernel<D, true, true>, token_kernel<D, true, false>, token_kernel<D, false, true>})
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return SPARSTAR_ERR_CUDA;
  return SPARSTAR_OK;
}

// CTAs of a cluster: enough to give every SM two CTAs, at most one per two kept blocks.
int tok_cluster(int n_seq, int heads_k, int keep, int sms) {
  int c = 1;
  while (c < 8 && static_cast<int64_t>(n_seq) * heads_k * c < 2 * sms && 4 * c <= keep) c *= 2;
  return c;
}

int tok_sizes(int n_seq, int heads_q, int heads_k, int64_t capacity, int head_dim) {
  if (n_seq < 0 || heads_k < 1 || heads_q < 1 || heads_q % heads_k != 0 || capacity < 1) return SPARSTAR_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return SPARSTAR_ERR_UNSUPPORTED;
  if (n_seq > 65535 || heads_k > 65535 || heads_q / heads_k > kTokMaxGroup || ceil_blocks(capacity) > kTokMaxBlocks ||
      static_cast<int64_t>(n_seq) * heads_k > INT32_MAX)
    return SPARSTAR_ERR_UNSUPPORTED;
  return SPARSTAR_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shared body of the three token entry points.
int token_run(bool sel, bool att, const void* q, const void* k, const void* v, const int32_t* kv_len,
              const float* means, int n_seq, int heads_q, int heads_k, int64_t capacity, int head_dim, int keep,
              int n_sink, int n_recent, float sm_scale, int32_t* idx, int32_t* cnt, void* o, float* lse, void* stream) {
  int rc = tok_sizes(n_seq, heads_q, heads_k, capacity, head_dim);
  if (rc != SPARSTAR_OK) return rc;
  if (keep < 1 || (sel && (n_sink < 0 || n_recent < 1 || n_recent > keep || n_sink > keep - n_recent)))
    return SPARSTAR_ERR_ARG;
  if (!(sm_scale == sm_scale) || std::isinf(sm_scale)) return SPARSTAR_ERR_ARG;
  if (n_seq == 0) return SPARSTAR_OK;
  if (q == nullptr || !aligned16(q) || kv_len == nullptr || !aligned4(kv_len) || idx == nullptr || !aligned4(idx) ||
      cnt == nullptr || !aligned4(cnt))
    return SPARSTAR_ERR_ARG;
  if (sel && (means == nullptr || !aligned16(means))) return SPARSTAR_ERR_ARG;
  if (att && (k == nullptr || !aligned16(k) || v == nullptr || !aligned16(v) || o == nullptr ||
              (reinterpret_cast<uintptr_t>(o) & 1u) != 0 || !aligned4(lse)))
    return SPARSTAR_ERR_ARG;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != SPARSTAR_OK) return rc;
  if (dev->major != 10) return SPARSTAR_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(g_attr_mutex);
    if (!g_attrs_set[dev->index]) {
      if ((rc = tok_set_attrs<128>()) != SPARSTAR_OK || (rc = tok_set_attrs<64>()) != SPARSTAR_OK) return rc;
      g_attrs_set[dev->index] = true;
    }
  }
  CUtensorMap tk = {}, tv = {};
  if (att && ((rc = make_map(&tk, k, capacity, n_seq * heads_k, head_dim)) != SPARSTAR_OK ||
              (rc = make_map(&tv, v, capacity, n_seq * heads_k, head_dim)) != SPARSTAR_OK))
    return rc;
  TokParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.means = means;
  p.kv_len = kv_len;
  p.idx = idx;
  p.cnt = cnt;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.status = dev->status;
  p.capacity = capacity;
  p.hk = heads_k;
  p.group = heads_q / heads_k;
  p.nb_cap = static_cast<int>(ceil_blocks(capacity));
  p.keep = keep;
  p.n_sink = n_sink;
  p.n_recent = n_recent;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.union_bytes = tok_union_bytes(head_dim, p.nb_cap, sel && p.nb_cap > keep, att);
  const unsigned c = static_cast<unsigned>(tok_cluster(n_seq, heads_k, keep, dev->sms));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, static_cast<unsigned>(heads_k), static_cast<unsigned>(n_seq));
  cfg.blockDim = dim3(kTokThreads);
  cfg.dynamicSmemBytes = p.union_bytes + 1024 + sizeof(TokFixed);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, tk, tv, p); };
  cudaError_t err;
  if (head_dim == 128)
    err = sel && att ? launch(token_kernel<128, true, true>)
                     : sel ? launch(token_kernel<128, true, false>) : launch(token_kernel<128, false, true>);
  else
    err = sel && att ? launch(token_kernel<64, true, true>)
                     : sel ? launch(token_kernel<64, true, false>) : launch(token_kernel<64, false, true>);
  return err == cudaSuccess ? launch_status() : (cudaGetLastError(), SPARSTAR_ERR_CUDA);
}

}  // namespace
}  // namespace sparstar

using namespace sparstar;

extern "C" {

int sparstar_block_means(const void* k, const int32_t* kv_len, int n_seq, int heads_k, int64_t capacity, int head_dim,
                         int tail_only, float* means, void* stream) {
  int rc = tok_sizes(n_seq, heads_k, heads_k, capacity, head_dim);
  if (rc != SPARSTAR_OK) return rc;
  if (n_seq == 0) return SPARSTAR_OK;
  if (k == nullptr || !aligned16(k) || kv_len == nullptr || !aligned4(kv_len) || means == nullptr || !aligned4(means))
    return SPARSTAR_ERR_ARG;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != SPARSTAR_OK) return rc;
  if (dev->major != 10) return SPARSTAR_ERR_UNSUPPORTED;
  const int nb = static_cast<int>(ceil_blocks(capacity));
  const dim3 grid(static_cast<unsigned>(tail_only ? 1 : nb), static_cast<unsigned>(heads_k),
                  static_cast<unsigned>(n_seq));
  const auto* kb = static_cast<const __nv_bfloat16*>(k);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (head_dim == 128)
    block_means_kernel<128><<<grid, 256, 0, st>>>(kb, kv_len, capacity, nb, tail_only, means, dev->status);
  else
    block_means_kernel<64><<<grid, 256, 0, st>>>(kb, kv_len, capacity, nb, tail_only, means, dev->status);
  return launch_status();
}

int sparstar_token_select(const void* q, const float* means, const int32_t* kv_len, int n_seq, int heads_q, int heads_k,
                          int64_t capacity, int head_dim, int keep, int n_sink, int n_recent, int32_t* idx,
                          int32_t* cnt, void* stream) {
  return token_run(true, false, q, nullptr, nullptr, kv_len, means, n_seq, heads_q, heads_k, capacity, head_dim, keep,
                   n_sink, n_recent, 0.f, idx, cnt, nullptr, nullptr, stream);
}

int sparstar_token_attn(const void* q, const void* k, const void* v, const int32_t* kv_len, int n_seq, int heads_q,
                        int heads_k, int64_t capacity, int head_dim, const int32_t* idx, const int32_t* cnt, int keep,
                        float sm_scale, void* o, float* lse, void* stream) {
  return token_run(false, true, q, k, v, kv_len, nullptr, n_seq, heads_q, heads_k, capacity, head_dim, keep, 0, 1,
                   sm_scale, const_cast<int32_t*>(idx), const_cast<int32_t*>(cnt), o, lse, stream);
}

int sparstar_token_forward(const void* q, const void* k, const void* v, const int32_t* kv_len, const float* means,
                           int n_seq, int heads_q, int heads_k, int64_t capacity, int head_dim, int keep, int n_sink,
                           int n_recent, float sm_scale, int32_t* idx, int32_t* cnt, void* o, float* lse,
                           void* stream) {
  return token_run(true, true, q, k, v, kv_len, means, n_seq, heads_q, heads_k, capacity, head_dim, keep, n_sink,
                   n_recent, sm_scale, idx, cnt, o, lse, stream);
}

}  // extern "C"
