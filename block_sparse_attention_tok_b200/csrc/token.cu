// One query token per sequence over a K/V cache: block means, selection, attention.
//
// Per (sequence, key head), with G = heads_q / heads_k query heads that share the key head:
//   score_j = (sum_g q_g) . mean_j      of every block j between the forced ones,
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
// The forced blocks are attended to first: their tiles are on the way while the others are ranked.
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
// Candidates that every CTA ranks for itself by counting, one a thread. With two a thread (up to 320) the
// batch of 48 sequences x 8 key heads with up to 253 took 143 us, so 140 us.
constexpr int kFew = kTokThreads;

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
  uint32_t score_at;        // where scores lie: behind the ring, or (0) in its place where they are many
  uint32_t fixed_at;        // TokFixed, behind both
};

// What a CTA's threads tell one another while ranking.
struct RankShared {
  int32_t tot[2][kTokThreads / 32];
  float most[kTokThreads / 32];
  float cut;
};

// Shared memory behind the ring and the scores.
struct TokFixed {
  uint64_t full[6], empty[6];
  // few candidates: scored and ranked by every CTA for itself
  float2 fast[kFew];
  uint32_t key[kFew];
  double exact[kFew];
  int32_t chosen[kFew], near[kFew];
  RankShared rank;
  uint32_t abort_flag;
};

static_assert(sizeof(TokFixed) <= 6144, "two CTAs an SM");

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

// Shared state of the radix select, behind the scores.
struct RankState {
  int32_t hist[kDigitBins];
  int32_t need, bucket;
};

struct KthKey {
  unsigned long long key;  // the take-th largest key
  int equal;               // how many of the keys equal to it are among the take largest
};

// Radix select over key(0..n), from the digit at `shift` (8 bits) down. One CTA, all threads.
template <typename F>
__device__ KthKey kth_key(int n, int take, int shift, RankState* st, F&& key) {
  const int tid = threadIdx.x, lane = tid & 31;
  unsigned long long prefix = 0ull, mask = 0ull;
  int need = take;
  for (; shift >= 0; shift -= 8) {
    for (int i = tid; i < kDigitBins; i += kTokThreads) st->hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTokThreads) {
      const unsigned long long k = key(i);
      if ((k & mask) == prefix) atomicAdd(&st->hist[(k >> shift) & (kDigitBins - 1)], 1);
    }
    __syncthreads();
    if (tid < 32) {  // the digit at which the count from the top reaches `need`
      constexpr int per = kDigitBins / 32;
      int sum = 0;
      for (int i = 0; i < per; ++i) sum += st->hist[kDigitBins - 1 - (lane * per + i)];
      int incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
      }
      int above = incl - sum;
      if (above < need && need <= incl) {
        for (int i = 0;; ++i) {
          const int b = kDigitBins - 1 - (lane * per + i), c = st->hist[b];
          if (above + c >= need) {
            st->bucket = b;
            st->need = need - above;
            break;
          }
          above += c;
        }
      }
    }
    __syncthreads();
    prefix |= static_cast<unsigned long long>(st->bucket) << shift;
    mask |= static_cast<unsigned long long>(kDigitBins - 1) << shift;
    need = st->need;
    __syncthreads();
  }
  return KthKey{prefix, need};
}

// Scores in two steps. The fp32 score s_j is off the exact S_j by at most E = 2^-18 max_j B_j, B_j the
// sum of the absolute products: 15 roundings of the query sum, the product, 19 of the sum, below
// 36 u = 2^-18.8 of B_j. With t the take-th largest s_j, the take-th largest S_j lies in [t - E, t + E],
// so s_j > t + 2E is in, s_j < t - 2E is out, and only what lies between (usually t's own block) is
// scored again, in fp64, where neighbours need it. Scores that are not finite make E so, and every
// block lies between. (48 sequences x 8 key heads, 297 candidates each: the selection alone takes 22 us,
// with every score in fp64 36 us, most of it conversions of the means.)
// The margin 2E of a largest B, with room for the comparison's rounding and, where products fall below
// the normal range, for the 2^-150 that each may lose there.
__device__ __forceinline__ float score_margin(float most) { return most * (2.25f / 262144.f) + 1e-42f; }

__device__ __forceinline__ uint32_t score_key32(float s) {
  if (isnan(s)) return 0u;
  const uint32_t b = __float_as_uint(s + 0.f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// (s, B) of blocks first, first + 1, ... (8 lanes a block, 20 at a time), the next ones step further on,
// below n.
template <int D>
__device__ __forceinline__ void score_fast(const __nv_bfloat16* q, int group, const float* means, int n, int first,
                                           int step, float2* scores) {
  constexpr int N = D / 32;  // float4 per lane
  const int l = threadIdx.x & 7, mine = threadIdx.x / 8;
  float qs[4 * N], qa[4 * N];
#pragma unroll
  for (int i = 0; i < 4 * N; ++i) qs[i] = qa[i] = 0.f;
  for (int g = 0; g < group; ++g)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(q + g * D + 4 * (l + 8 * i)));
      const float x[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                          __uint_as_float(v.y & 0xFFFF0000u)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qs[4 * i + e] += x[e];
        qa[4 * i + e] += fabsf(x[e]);
      }
    }
  const float4* mean = reinterpret_cast<const float4*>(means) + l;
  // four blocks' means in flight per lane
  for (int j0 = first; j0 < n; j0 += 4 * step) {
    float4 m[4][N];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * step + mine;
#pragma unroll
      for (int i = 0; i < N; ++i)
        m[u][i] = j < n ? __ldg(mean + static_cast<int64_t>(j) * (D / 4) + 8 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u * step + mine;
      if (j0 + u * step >= n) break;
      float s = 0.f, a = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x[4] = {m[u][i].x, m[u][i].y, m[u][i].z, m[u][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(qs[4 * i + e], x[e], s);
          a = fmaf(qa[4 * i + e], fabsf(x[e]), a);
        }
      }
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        a += __shfl_xor_sync(0xFFFFFFFFu, a, off);
      }
      if (l == 0 && j < n) scores[j] = make_float2(s, a);
    }
  }
}

// The fp64 score of one block, by 8 lanes (all of a warp take part).
template <int D>
__device__ double score_exact(const __nv_bfloat16* q, int group, const float* mean) {
  const int l = threadIdx.x & 7;
  double s = 0.0;
  for (int c = 4 * l; c < D; c += 32) {
    const float4 m = __ldg(reinterpret_cast<const float4*>(mean + c));
    const float x[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double qs = 0.0;
      for (int g = 0; g < group; ++g) qs += static_cast<double>(__bfloat162float(q[g * D + c + e]));
      s = fma(qs, static_cast<double>(x[e]), s);
    }
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  return s;
}

// Exact scores of the n blocks near[0..n) (null: 0..n), to out.
template <int D>
__device__ void score_all_exact(const __nv_bfloat16* q, int group, const float* means, const int32_t* near, int n,
                                double* out) {
  for (int i0 = 0; i0 < n; i0 += kTokThreads / 8) {
    const int i = i0 + threadIdx.x / 8, at = i < n ? i : n - 1;
    const double s = score_exact<D>(q, group, means + static_cast<int64_t>(near != nullptr ? near[at] : at) * D);
    if ((threadIdx.x & 7) == 0 && i < n) out[i] = s;
  }
}

// Positions among the `n` exact scores, one a thread: is this thread's one of the `take` best?
__device__ __forceinline__ bool best_exact(const double* exact, int n, int take) {
  const unsigned long long key = static_cast<int>(threadIdx.x) < n ? score_key(exact[threadIdx.x]) : 0ull;
  int above = 0;
  for (int i = 0; i < n; ++i) above += score_key(exact[i]) + (i < static_cast<int>(threadIdx.x) ? 1u : 0u) > key;
  return static_cast<int>(threadIdx.x) < n && above < take;
}

// Two counts over the CTA: lower threads' flags a and b go to before_a, before_b; totals to *all_a, *all_b.
__device__ __forceinline__ void count2(RankShared* st, bool a, bool b, int* before_a, int* before_b, int* all_a,
                                       int* all_b) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned ba = __ballot_sync(0xFFFFFFFFu, a), bb = __ballot_sync(0xFFFFFFFFu, b), low = (1u << lane) - 1u;
  if (lane == 0) {
    st->tot[0][w] = __popc(ba);
    st->tot[1][w] = __popc(bb);
  }
  __syncthreads();
  *before_a = __popc(ba & low);
  *before_b = __popc(bb & low);
  *all_a = *all_b = 0;
#pragma unroll
  for (int x = 0; x < kTokThreads / 32; ++x) {
    if (x < w) {
      *before_a += st->tot[0][x];
      *before_b += st->tot[1][x];
    }
    *all_a += st->tot[0][x];
    *all_b += st->tot[1][x];
  }
  __syncthreads();
}

__device__ __forceinline__ float max_over_cta(RankShared* st, float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, off);
    v = (isnan(v) || v > o) ? v : o;  // NaN stays
  }
  if ((threadIdx.x & 31) == 0) st->most[threadIdx.x >> 5] = v;
  __syncthreads();
  v = st->most[0];
#pragma unroll
  for (int x = 1; x < kTokThreads / 32; ++x) v = (isnan(v) || v > st->most[x]) ? v : st->most[x];
  __syncthreads();
  return v;
}

// Class of a score against the cut: 2 in, 1 between, 0 out.
__device__ __forceinline__ int score_class(float s, float cut, float margin) {
  if (!isfinite(margin)) return 1;
  return s - cut > margin ? 2 : s - cut >= -margin ? 1 : 0;
}

// Ranks up to kFew candidates, one a thread (of equal ones the lower is better: its key counts as one
// more). The chosen positions go, ascending, to fix->chosen. One CTA, all threads.
template <int D>
__device__ __forceinline__ void rank_few(TokFixed* fix, const __nv_bfloat16* q, int group, const float* means, int n,
                                         int take) {
  const int tid = threadIdx.x;
  const bool in = tid < n;
  const float2 v = in ? fix->fast[tid] : make_float2(0.f, 0.f);
  const uint32_t key = in ? score_key32(v.x) : 0u;
  fix->key[tid] = key;
  const float margin = score_margin(max_over_cta(&fix->rank, v.y));
  int above = 0;
#pragma unroll 8
  for (int i = 0; i < n; ++i) above += fix->key[i] + (i < tid ? 1u : 0u) > key;
  if (in && above == take - 1) fix->rank.cut = v.x;
  __syncthreads();
  const int cls = in ? score_class(v.x, fix->rank.cut, margin) : 0;
  int before_sure, before_near, sure, near;
  count2(&fix->rank, cls == 2, cls == 1, &before_sure, &before_near, &sure, &near);
  bool mine = cls != 0;
  if (sure + near != take) {
    if (cls == 1) fix->near[before_near] = tid;
    __syncthreads();
    score_all_exact<D>(q, group, means, fix->near, near, fix->exact);
    __syncthreads();
    if (best_exact(fix->exact, near, take - sure))
      fix->chosen[tid] = 1;
    else
      fix->chosen[tid] = 0;
    __syncthreads();
    mine = cls == 2 || (cls == 1 && fix->chosen[before_near] != 0);
    __syncthreads();
  }
  int before, none, all;
  count2(&fix->rank, mine, false, &before, &none, &all, &none);
  if (mine) fix->chosen[before] = tid;
}

// The same for many candidates, whose fp32 scores one CTA holds; writes base + position to out. With more
// than kFew blocks between, all are scored exactly (over the fp32 scores) and ranked by their fp64 keys.
template <int D>
__device__ void rank_many(float2* scores, TokFixed* fix, RankState* st, const __nv_bfloat16* q, int group,
                          const float* means, int n, int take, int base, int32_t* out) {
  const int tid = threadIdx.x;
  float most = 0.f;
  for (int i = tid; i < n; i += kTokThreads) most = (isnan(most) || most > scores[i].y) ? most : scores[i].y;
  const float margin = score_margin(max_over_cta(&fix->rank, most));
  bool all_exact = !isfinite(margin);
  if (!all_exact) {
    const uint32_t cut_key = static_cast<uint32_t>(
        kth_key(n, take, 24, st, [&](int i) { return static_cast<unsigned long long>(score_key32(scores[i].x)); }).key);
    const float cut = __uint_as_float((cut_key >> 31) ? cut_key & 0x7FFFFFFFu : ~cut_key);
    int sure = 0, near = 0;
    for (int i0 = 0; i0 < n; i0 += kTokThreads) {
      const int i = i0 + tid;
      const int cls = i < n ? score_class(scores[i].x, cut, margin) : 0;
      int before_sure, before_near, more_sure, more_near;
      count2(&fix->rank, cls == 2, cls == 1, &before_sure, &before_near, &more_sure, &more_near);
      if (cls == 1 && near + before_near < kFew) fix->near[near + before_near] = i;
      sure += more_sure;
      near += more_near;
    }
    all_exact = near > kFew;
    if (!all_exact) {
      __syncthreads();
      fix->chosen[tid] = 1;
      if (sure + near != take) {
        score_all_exact<D>(q, group, means, fix->near, near, fix->exact);
        __syncthreads();
        fix->chosen[tid] = best_exact(fix->exact, near, take - sure);
      }
      __syncthreads();
      int placed = 0, seen = 0;
      for (int i0 = 0; i0 < n; i0 += kTokThreads) {
        const int i = i0 + tid;
        const int cls = i < n ? score_class(scores[i].x, cut, margin) : 0;
        int before, before_near, none, more, more_near;
        count2(&fix->rank, false, cls == 1, &none, &before_near, &none, &more_near);
        const bool mine = cls == 2 || (cls == 1 && fix->chosen[seen + before_near] != 0);
        count2(&fix->rank, mine, false, &before, &none, &more, &none);
        if (mine) out[placed + before] = base + i;
        placed += more;
        seen += more_near;
      }
      return;
    }
  }
  double* exact = reinterpret_cast<double*>(scores);
  __syncthreads();
  score_all_exact<D>(q, group, means, nullptr, n, exact);
  __syncthreads();
  const KthKey k = kth_key(n, take, 56, st, [&](int i) { return score_key(exact[i]); });
  int placed = 0, seen = 0;
  for (int i0 = 0; i0 < n; i0 += kTokThreads) {
    const int i = i0 + tid;
    const unsigned long long key = i < n ? score_key(exact[i]) : 0ull;
    const bool same = i < n && key == k.key;
    int before, before_same, none, more, more_same;
    count2(&fix->rank, same, false, &before_same, &none, &more_same, &none);
    const bool mine = i < n && (key > k.key || (same && seen + before_same < k.equal));
    count2(&fix->rank, mine, false, &before, &none, &more, &none);
    if (mine) out[placed + before] = base + i;
    placed += more;
    seen += more_same;
  }
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
  TokFixed* fix = reinterpret_cast<TokFixed*>(smem + p.fixed_at);
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

  if (ATT && tid == 128) {  // the thread that loads
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
  const bool all = SEL && nb <= p.keep, few = SEL && !all && n_cand <= kFew;
  // The i-th entry of this CTA: with SEL the recent blocks come first, then the first ones, then the
  // chosen ones.
  auto entry = [&](int i) {
    const int pos = rank + i * size;
    if (!SEL || all) return pos;
    return pos < p.n_recent ? p.keep - p.n_recent + pos : pos - p.n_recent;
  };
  auto load_tile = [&](uint32_t it, int j) {  // K (even it) or V of block j into its stage
    const uint32_t st = it % C::kStages;
    mbar_arrive_expect_tx(&full[st], C::kTileBytes);
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c)
      tma_load_3d(smem_u32(smem) + st * C::kTileBytes + c * C::kChunkBytes, (it & 1u) == 0 ? &tm_k : &tm_v, &full[st],
                  c * 64, j * 128, static_cast<int>(row));
  };
  // Tiles that are loaded before the choice is made: of every block where all are kept, else of the
  // forced ones, as far as the ring goes.
  int early = 0;
  if (SEL && ATT && p.score_at != 0) {
    const int known = all ? nb : p.n_recent + p.n_sink;
    early = known > rank ? 2 * ((known - rank + size - 1) / size) : 0;
    if (early > C::kStages) early = C::kStages;
    if (tid == 128)
      for (int it = 0; it < early; ++it) {
        const int e = entry(it >> 1);
        load_tile(it, all || e < p.n_sink ? e : nb - p.keep + e);
      }
  }
  bool synced = false;
  if (SEL && !all && take > 0) {  // 0 < take < n_cand
    const float* means = p.means + (row * p.nb_cap + p.n_sink) * D;
    if (few) {
      score_fast<D>(q, p.group, means, n_cand, 0, kTokThreads / 8, fix->fast);
      __syncthreads();
      rank_few<D>(fix, q, p.group, means, n_cand, take);
      __syncthreads();
    } else {
      if (size > 1) cluster.sync();  // the first CTA runs before anyone writes to it
      constexpr int kPer = kTokThreads / 8;  // blocks a CTA scores at a time
      score_fast<D>(q, p.group, means, n_cand, rank * kPer, size * kPer,
                    cluster.map_shared_rank(reinterpret_cast<float2*>(smem + p.score_at), 0));
      if (size > 1)
        cluster.sync();
      else
        __syncthreads();
      if (rank == 0) {
        uint8_t* mine = smem + p.score_at;
        RankState* st = reinterpret_cast<RankState*>(mine + ((static_cast<size_t>(n_cand) * 8 + 15) & ~15ull));
        rank_many<D>(reinterpret_cast<float2*>(mine), fix, st, q, p.group, means, n_cand, take, p.n_sink,
                     list + p.n_sink);
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
    const int e = entry(i);
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
      if (early == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // scores may have lain there
      uint32_t it = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_mine; ++i) {
        const int j = block_at(i, true);
        if (j < 0) continue;
        for (int kv = 0; kv < 2; ++kv, ++it) {
          if (static_cast<int>(it) < early) continue;
          const uint32_t st = it % C::kStages;
          ok = mbar_wait(&empty[st], ((it / C::kStages) & 1u) ^ 1u, abort_flag, p.status);
          if (!ok) break;
          load_tile(it, j);
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
    // Gives a stage back. The proxy fence holds the arrival until this warp's ldmatrix reads are done:
    // the copy that follows writes through the async proxy, and without the fence it overtook them.
    auto release = [&](uint32_t st) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    };
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
      release(st);
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
      release(st);
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
    const float base = m == -INFINITY ? 0.f : m;  // no token, or scores that are NaN: l tells them apart
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float f = ex2_approx(pm[w * 16 + r] - base);
      v = fmaf(f, po[(w * 16 + r) * kPad + c], v);
      l = fmaf(f, pl[w * 16 + r], l);
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
    const float base = m == -INFINITY ? 0.f : m;
    for (int x = 0; x < size; ++x) {
      const float f = ex2_approx(cluster.map_shared_rank(cm, x)[r] - base);
      v = fmaf(f, cluster.map_shared_rank(co, x)[i], v);
      l = fmaf(f, cluster.map_shared_rank(cl, x)[r], l);
    }
    // a sequence with no kept token: o = 0, lse = -inf
    p.o[row * p.group * D + i] = __float2bfloat16_rn(l == 0.f ? 0.f : v / l);
    if (c == 0 && p.lse != nullptr)
      p.lse[row * p.group + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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

constexpr uint32_t kScoreBeside = 10000;  // scores up to here get their own room: two CTAs an SM still fit

// Shared memory: the ring, the scores of many candidates (behind the ring, or in its place), TokFixed.
void tok_layout(int d, int64_t nb, bool many, bool att, uint32_t* score_at, uint32_t* fixed_at) {
  const uint32_t ring = att ? (d == 128 ? TokConfig<128>::kRingBytes : TokConfig<64>::kRingBytes) : 0;
  const uint32_t score = many ? static_cast<uint32_t>(nb * 8 + 16 + sizeof(RankState)) : 0;
  const bool beside = score <= kScoreBeside;
  *score_at = beside ? ring : 0;
  *fixed_at = ((beside ? ring + score : ring > score ? ring : score) + 127u) & ~127u;
}

template <int D>
int tok_set_attrs() {
  uint32_t score_at, fixed_at;
  tok_layout(D, kTokMaxBlocks, true, true, &score_at, &fixed_at);
  const uint32_t most = fixed_at + 1024 + sizeof(TokFixed);
  for (auto kernel : {token_kernel<D, true, true>, token_kernel<D, true, false>, token_kernel<D, false, true>})
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return SPARSTAR_ERR_CUDA;
  return SPARSTAR_OK;
}

// CTAs of a cluster: enough to give every SM about four CTAs (two at a time: the last ones then leave
// little idle; 48 sequences x 8 key heads, 32 blocks of 64 KB: 124 us of attention with clusters of two,
// 130 us with one, 129 us with four), at most one per two kept blocks.
int tok_cluster(int n_seq, int heads_k, int keep, int sms) {
  int c = 1;
  while (c < 8 && static_cast<int64_t>(n_seq) * heads_k * c < 4 * sms && 4 * c <= keep) c *= 2;
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
  tok_layout(head_dim, p.nb_cap, sel && p.nb_cap - n_sink - n_recent > kFew && p.nb_cap > keep, att, &p.score_at,
             &p.fixed_at);
  // Without the attention, CTAs that would all rank the same few candidates are not worth a cluster.
  const bool few = p.nb_cap - n_sink - n_recent <= kFew;
  const unsigned c = !att && few ? 1u : static_cast<unsigned>(tok_cluster(n_seq, heads_k, keep, dev->sms));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, static_cast<unsigned>(heads_k), static_cast<unsigned>(n_seq));
  cfg.blockDim = dim3(kTokThreads);
  cfg.dynamicSmemBytes = p.fixed_at + 1024 + sizeof(TokFixed);
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
