// RMS norm of the queries and keys of each head with the position rotation, and its gradient.
//
// Forward, per token n and head h, on x = the head's d projected values:
//   r = 1 / sqrt(mean(x^2) + eps),  u = w * r * x,  y = R(theta_n) u,
// R turning each coordinate pair (a, b) by the token's angle: (a c - b s, b c + a s). Pairs are
// (i, i + d/2), or (2i, 2i + 1) when interleaved. V has no norm and no rotation; it is carried
// along because the same pass changes the layout from token-major [N, heads, d] (a slice of a
// fused projection) to the head-major [heads, rows, d] that selection and attention read, or
// to a row of each sequence's cache.
// Backward, from dy: g_u = R(-theta_n) dy (R is orthogonal),
//   dw = sum over tokens and heads of g_u * r * x,
//   dx = r * (w g_u - xh * mean(w g_u * xh)),  xh = r x  (r is recomputed: x is read anyway).
// All arithmetic is fp32; each output is rounded once, when it is stored.
//
// Bound: memory. Each value is read once and written once, nothing is staged: d/8 neighbouring
// lanes hold one head vector (8 values each, so that both members of every pair are in one
// lane: no exchange but the sum of squares), and an item is one token x up to H heads of
// one kind (1, 2 or 4 by the call's size), loaded together before any is used (H x 16 bytes in flight
// per lane in bf16, H x 32 in fp32), which also reads the token's angles once per item.
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "host.h"
#include "ptx.cuh"

namespace sparstar {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrMaxParts = 1024;  // partial dw rows at most (one per CTA of the gradient)

struct NrView {
  void* data;
  int64_t token, head, seq;  // strides in elements
};

struct NrParams {
  NrView x[3], y[3];       // q, k, v: token-major values x; head-major results y (gradient: dy)
  NrView dx[3];            // gradient: token-major dx
  const float* w[2];       // norm weights of q and k, or null (ones)
  const float *cos, *sin;  // [N, d/2], or null (no rotation)
  const int32_t* kv_rows;  // [N] or null: row of each token's k and v
  int64_t kv_offset, kv_capacity;
  int64_t n_tokens;
  int chunks[3];           // head chunks of q, k, v
  int heads[3];
  float eps;
  unsigned* status;
  float* dw_part;          // gradient: [CTAs of q and k][d]
  int ctas[3];             // gradient: CTAs of q, k, v
};

// 8 values of a head vector per lane. Lane l holds 4l.. and d/2 + 4l.. (pairs i, i + d/2), or
// with adjacent pairs 8l..8l+7; either way the lane's four angles are 4l..4l+3.
template <int D, bool IL>
struct Lane8 {
  __device__ static int first(int l) { return IL ? 8 * l : 4 * l; }
  __device__ static int second(int l) { return IL ? 8 * l + 4 : D / 2 + 4 * l; }
};

template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint2 a, b;
  __device__ void load(const __nv_bfloat16* p, int i0, int i1) {
    a = __ldcs(reinterpret_cast<const uint2*>(p + i0));
    b = __ldcs(reinterpret_cast<const uint2*>(p + i1));
  }
  __device__ void zero() { a = b = make_uint2(0u, 0u); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ void load(const float* p, int i0, int i1) {
    a = __ldcs(reinterpret_cast<const float4*>(p + i0));
    b = __ldcs(reinterpret_cast<const float4*>(p + i1));
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, int i0, int i1, const float (&y)[8]) {
  *reinterpret_cast<uint2*>(p + i0) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  *reinterpret_cast<uint2*>(p + i1) = make_uint2(pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
}
__device__ __forceinline__ void store8(float* p, int i0, int i1, const float (&y)[8]) {
  *reinterpret_cast<float4*>(p + i0) = make_float4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<float4*>(p + i1) = make_float4(y[4], y[5], y[6], y[7]);
}

// Turns the lane's four pairs by (c, s).
template <bool IL>
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = IL ? 2 * i : i, ib = IL ? 2 * i + 1 : i + 4;
    const float a = x[ia], b = x[ib];
    x[ia] = a * c[i] - b * s[i];
    x[ib] = b * c[i] + a * s[i];
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  return v;
}

// One item of a group of lanes: a token and a run of heads of one kind (0 q, 1 k, 2 v).
struct NrItem {
  int64_t n;
  int kind, h0, nh;
  bool live;
};

template <int H>
__device__ __forceinline__ NrItem nr_item(const NrParams& p, int64_t tile, int chunk, int groups, int g) {
  NrItem it;
  it.n = tile * groups + g;
  it.live = it.n < p.n_tokens;
  it.kind = 0;
  if (chunk >= p.chunks[0]) {
    chunk -= p.chunks[0];
    it.kind = 1;
    if (chunk >= p.chunks[1]) {
      chunk -= p.chunks[1];
      it.kind = 2;
    }
  }
  it.h0 = chunk * H;
  it.nh = min(H, p.heads[it.kind] - it.h0);
  return it;
}

__device__ __forceinline__ NrView pick(const NrView (&v)[3], int kind) {
  return kind == 0 ? v[0] : kind == 1 ? v[1] : v[2];
}

template <int D, bool IL>
__device__ __forceinline__ void load_angles(const NrParams& p, int64_t n, int l, float (&c)[4], float (&s)[4]) {
  if (p.cos != nullptr) {
    const float4 cc = __ldg(reinterpret_cast<const float4*>(p.cos + n * (D / 2) + 4 * l));
    const float4 ss = __ldg(reinterpret_cast<const float4*>(p.sin + n * (D / 2) + 4 * l));
    c[0] = cc.x, c[1] = cc.y, c[2] = cc.z, c[3] = cc.w;
    s[0] = ss.x, s[1] = ss.y, s[2] = ss.z, s[3] = ss.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
  }
}

template <int D, bool IL>
__device__ __forceinline__ void load_weight(const float* w, int l, float (&out)[8]) {
  if (w != nullptr) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + Lane8<D, IL>::first(l)));
    const float4 b = __ldg(reinterpret_cast<const float4*>(w + Lane8<D, IL>::second(l)));
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.f;
  }
}

// grid: (token tiles x head chunks), chunks fastest, so that the CTAs of a token tile run
// together and share its angles in L2.
template <int D, typename T, bool IL, int H>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NrParams p) {
  constexpr int G = D / 8, kGroups = kNrThreads / G;
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  const int n_chunks = p.chunks[0] + p.chunks[1] + p.chunks[2];
  const int64_t tile = blockIdx.x / n_chunks;
  const NrItem it = nr_item<H>(p, tile, static_cast<int>(blockIdx.x - tile * n_chunks), kGroups, g);
  const int i0 = Lane8<D, IL>::first(l), i1 = Lane8<D, IL>::second(l);
  const NrView xv = pick(p.x, it.kind), yv = pick(p.y, it.kind);
  const T* src = static_cast<const T*>(xv.data) + it.n * xv.token + it.h0 * xv.head;
  Raw8<T> raw[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (it.live && h < it.nh)
      raw[h].load(src + h * xv.head, i0, i1);
    else
      raw[h].zero();
  }
  // destination row: the token itself for q, its place in the K/V rows for k and v
  int64_t row = it.n;
  bool put = it.live;
  if (it.kind != 0) {
    if (p.kv_rows != nullptr) {
      row = it.live ? __ldg(p.kv_rows + it.n) : -1;
      if (row >= p.kv_capacity) {
        if (l == 0) atomicOr(p.status, kStatusBounds);
        row = -1;
      }
      put = row >= 0;
    } else {
      row = p.kv_offset + it.n;
    }
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(yv.data) + it.n * yv.seq + row * yv.token + it.h0 * yv.head;
  if (it.kind == 2) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float x[8];
      raw[h].get(x);
      if (put && h < it.nh) store8(dst + h * yv.head, i0, i1, x);
    }
    return;
  }
  float c[4], s[4], w[8];
  load_angles<D, IL>(p, it.live ? it.n : 0, l, c, s);
  load_weight<D, IL>(it.kind == 0 ? p.w[0] : p.w[1], l, w);
#pragma unroll
  for (int h = 0; h < H; ++h) {
    float x[8];
    raw[h].get(x);
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
    const float r = rsqrtf(group_sum<G>(ss) * (1.f / D) + p.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * r * w[e];
    turn<IL>(x, c, s);
    if (put && h < it.nh) store8(dst + h * yv.head, i0, i1, x);
  }
}

// Persistent: every CTA serves one kind (shares of the CTAs go by bytes, see nr_bwd_grid) and walks
// its items with a fixed stride, keeping the sums of dw of its lanes in registers, so dw costs no
// traffic until the CTA's one partial row; the rows are added in order by norm_rope_dw_kernel (no
// atomics: the same inputs give the same bits).
// Three CTAs an SM with four heads an item (80 registers): 18,432 tokens x 32 heads of q, k and v in
// 207 us, 5.87 TB/s; with two heads an item 260 us, with four CTAs and two heads 224 us, and with the
// kinds mixed in every CTA (two sums of dw, 128 registers, two CTAs) 256 us.
constexpr int kNrBwdCtas = 3;
template <int D, typename T, bool IL, int H>
__global__ void __launch_bounds__(kNrThreads, kNrBwdCtas) norm_rope_bwd_kernel(const NrParams p) {
  constexpr int G = D / 8, kGroups = kNrThreads / G;
  __shared__ float part[kGroups][D];
  griddep_launch_dependents();
  const int l = threadIdx.x % G, g = threadIdx.x / G;
  const int i0 = Lane8<D, IL>::first(l), i1 = Lane8<D, IL>::second(l);
  int kind = 0, first = blockIdx.x;
  while (kind < 2 && first >= p.ctas[kind]) first -= p.ctas[kind++];
  const NrView xv = pick(p.x, kind), yv = pick(p.y, kind), dv = pick(p.dx, kind);
  const int chunks = kind == 0 ? p.chunks[0] : p.chunks[1];  // v has k's heads
  const int heads = kind == 0 ? p.heads[0] : p.heads[1];
  const int step = kind == 0 ? p.ctas[0] : kind == 1 ? p.ctas[1] : p.ctas[2];
  const int n_items = static_cast<int>((p.n_tokens + kGroups - 1) / kGroups) * chunks;
  const int64_t row0 = kind == 0 ? 0 : p.kv_offset;
  float dw[8], w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = 0.f;
  load_weight<D, IL>(kind == 0 ? p.w[0] : p.w[1], l, w);
  for (int t = first; t < n_items; t += step) {
    const int tile = t / chunks, h0 = (t - tile * chunks) * H;
    const int64_t n = static_cast<int64_t>(tile) * kGroups + g;
    const int nh = n < p.n_tokens ? min(H, heads - h0) : 0;
    const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(yv.data) + (row0 + n) * yv.token + h0 * yv.head;
    T* dst = static_cast<T*>(dv.data) + n * dv.token + h0 * dv.head;
    Raw8<__nv_bfloat16> rdy[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h < nh)
        rdy[h].load(dy + h * yv.head, i0, i1);
      else
        rdy[h].zero();
    }
    if (kind == 2) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float d[8];
        rdy[h].get(d);
        if (h < nh) store8(dst + h * dv.head, i0, i1, d);
      }
      continue;
    }
    const T* src = static_cast<const T*>(xv.data) + n * xv.token + h0 * xv.head;
    Raw8<T> rx[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h < nh)
        rx[h].load(src + h * xv.head, i0, i1);
      else
        rx[h].zero();
    }
    float c[4], s[4];
    load_angles<D, IL>(p, nh > 0 ? n : 0, l, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = -s[i];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float x[8], d[8];
      rx[h].get(x);
      rdy[h].get(d);
      turn<IL>(d, c, s);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
      // a place without a token or head holds zeros: with eps 0 its root would be infinite, and dw NaN
      const float mean = group_sum<G>(ss) * (1.f / D);
      const float r = h < nh ? rsqrtf(mean + p.eps) : 0.f;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= r;
        dw[e] = fmaf(d[e], x[e], dw[e]);
        d[e] *= w[e];
        dot = fmaf(d[e], x[e], dot);
      }
      const float m = group_sum<G>(dot) * (1.f / D);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = r * (d[e] - x[e] * m);
      if (h < nh) store8(dst + h * dv.head, i0, i1, d);
    }
  }
  if (kind == 2) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    part[g][i0 + e] = dw[e];
    part[g][i1 + e] = dw[4 + e];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) a += part[i][threadIdx.x];
    p.dw_part[static_cast<int64_t>(blockIdx.x) * D + threadIdx.x] = a;  // q's rows, then k's
  }
}

// dw[d] of one kind, 32 columns a CTA: 32 warps each add every 32nd partial row of their columns,
// then the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* __restrict__ part, int rows_q, int rows_k,
                                                            float* dwq, float* dwk) {
  __shared__ float sum[32][33];
  griddep_wait();
  const int kind = blockIdx.x & 1, c0 = (blockIdx.x >> 1) * 32;
  float* dw = kind == 0 ? dwq : dwk;
  if (dw == nullptr) return;
  const int rows = kind == 0 ? rows_q : rows_k;
  part += static_cast<int64_t>(kind == 0 ? 0 : rows_q) * D;
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5;
  float a = 0.f;
  for (int r0 = w; r0 < rows; r0 += 8 * 32) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = r0 + 32 * u;
      v[u] = r < rows ? part[static_cast<int64_t>(r) * D + c0 + c] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) a += v[u];
  }
  sum[w][c] = a;
  __syncthreads();
  if (w == 0) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a += sum[i][c];
    dw[c0 + c] = a;
  }
}

bool strides_ok(const sparstar_view& v, int elem, bool has_token, bool has_head) {
  const int64_t q = 16 / elem;
  return aligned16(v.data) && v.data != nullptr && (!has_token || (v.token_stride > 0 && v.token_stride % q == 0)) &&
         (!has_head || (v.head_stride > 0 && v.head_stride % q == 0)) && v.seq_stride >= 0 && v.seq_stride % q == 0;
}

NrView view(const sparstar_view& v) { return NrView{v.data, v.token_stride, v.head_stride, v.seq_stride}; }

// Checks and parameters that both directions share. x: token-major values, y: head-major.
int nr_setup(const sparstar_view (&x)[3], const sparstar_view (&y)[3], int x_dtype, int64_t n_tokens, int heads_q,
             int heads_k, int head_dim, const float* wq, const float* wk, const float* cos, const float* sin,
             float eps, int64_t kv_offset, NrParams* p) {
  if (heads_q < 1 || heads_k < 0 || n_tokens < 0 || !(eps >= 0.f) || std::isinf(eps)) return SPARSTAR_ERR_ARG;
  if (x_dtype != SPARSTAR_BF16 && x_dtype != SPARSTAR_FP32) return SPARSTAR_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return SPARSTAR_ERR_UNSUPPORTED;
  if (heads_q > 65535 || heads_k > 65535 || n_tokens > INT32_MAX) return SPARSTAR_ERR_UNSUPPORTED;
  if ((cos == nullptr) != (sin == nullptr) || !aligned16(cos) || !aligned16(sin) || !aligned16(wq) || !aligned16(wk))
    return SPARSTAR_ERR_ARG;
  if (kv_offset < 0) return SPARSTAR_ERR_ARG;
  const bool has_v = heads_k > 0 && x[2].data != nullptr;
  if (n_tokens > 0 && has_v != (heads_k > 0 && y[2].data != nullptr)) return SPARSTAR_ERR_ARG;
  const int e = x_dtype == SPARSTAR_BF16 ? 2 : 4;
  *p = NrParams{};
  for (int kind = 0; kind < 3; ++kind) {
    const int h = kind == 0 ? heads_q : kind == 1 ? heads_k : (has_v ? heads_k : 0);
    p->heads[kind] = h;
    if (x[kind].seq_stride != 0 || (kind == 0 && y[kind].seq_stride != 0)) return SPARSTAR_ERR_ARG;
    if (h > 0 && n_tokens > 0 &&
        (!strides_ok(x[kind], e, n_tokens > 1, h > 1) || !strides_ok(y[kind], 2, n_tokens > 1 || kind > 0, h > 1)))
      return SPARSTAR_ERR_ARG;
    p->x[kind] = view(x[kind]);
    p->y[kind] = view(y[kind]);
  }
  p->w[0] = wq;
  p->w[1] = wk;
  p->cos = cos;
  p->sin = sin;
  p->eps = eps;
  p->n_tokens = n_tokens;
  return SPARSTAR_OK;
}

void nr_chunks(NrParams* p, int per) {
  for (int kind = 0; kind < 3; ++kind) p->chunks[kind] = (p->heads[kind] + per - 1) / per;
}

int64_t nr_items(const NrParams& p, int head_dim) {
  const int64_t groups = kNrThreads / (head_dim / 8);
  return (p.n_tokens + groups - 1) / groups * (p.chunks[0] + p.chunks[1] + p.chunks[2]);
}

// CTAs of the gradient: as many as run at once, shared out to q, k and v by the bytes that each
// moves (dy, x and dx; v has no x), at most one per item and one per kind that has heads.
void nr_bwd_grid(NrParams* p, int head_dim, int x_bytes, int per_sm, int sms) {
  const int64_t groups = kNrThreads / (head_dim / 8), tiles = (p->n_tokens + groups - 1) / groups;
  const int64_t most = static_cast<int64_t>(per_sm) * sms < kNrMaxParts ? per_sm * sms : kNrMaxParts;
  const int64_t bytes[3] = {p->heads[0] * (2 + 2 * x_bytes), p->heads[1] * (2 + 2 * x_bytes),
                            p->heads[2] * (2 + x_bytes)};
  const int64_t all = bytes[0] + bytes[1] + bytes[2];
  for (int kind = 0; kind < 3; ++kind) {
    const int64_t items = tiles * p->chunks[kind];
    int64_t c = most * bytes[kind] / all;
    if (c < 1) c = 1;
    p->ctas[kind] = static_cast<int>(p->heads[kind] == 0 ? 0 : c < items ? c : items);
  }
}

// Calls f<D, T, IL>() for the runtime head_dim, type and pairing.
template <typename F>
void nr_dispatch(int head_dim, int x_dtype, bool il, F&& f) {
  auto by_pair = [&](auto d, auto t) {
    if (il)
      f(d, t, std::integral_constant<bool, true>{});
    else
      f(d, t, std::integral_constant<bool, false>{});
  };
  auto by_type = [&](auto d) {
    if (x_dtype == SPARSTAR_BF16)
      by_pair(d, __nv_bfloat16{});
    else
      by_pair(d, float{});
  };
  if (head_dim == 128)
    by_type(std::integral_constant<int, 128>{});
  else
    by_type(std::integral_constant<int, 64>{});
}

}  // namespace
}  // namespace sparstar

using namespace sparstar;

extern "C" {

int sparstar_qk_norm_rope(sparstar_view q, sparstar_view k, sparstar_view v, int x_dtype, int64_t n_tokens, int heads_q,
                          int heads_k, int head_dim, const float* wq, const float* wk, const float* cos,
                          const float* sin, float eps, int interleaved, sparstar_view q_out, sparstar_view k_out,
                          sparstar_view v_out, const int32_t* kv_rows, int64_t kv_offset, int64_t kv_capacity,
                          void* stream) {
  NrParams p;
  int rc = nr_setup({q, k, v}, {q_out, k_out, v_out}, x_dtype, n_tokens, heads_q, heads_k, head_dim, wq, wk, cos, sin,
                    eps, kv_offset, &p);
  if (rc != SPARSTAR_OK) return rc;
  if (heads_k > 0 && (kv_capacity < 0 || (kv_rows == nullptr && kv_offset > kv_capacity - n_tokens)))
    return SPARSTAR_ERR_ARG;
  if (kv_rows == nullptr && (k_out.seq_stride != 0 || v_out.seq_stride != 0)) return SPARSTAR_ERR_ARG;
  if (n_tokens == 0) return SPARSTAR_OK;
  if ((reinterpret_cast<uintptr_t>(kv_rows) & 3u) != 0) return SPARSTAR_ERR_ARG;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != SPARSTAR_OK) return rc;
  if (dev->major != 10) return SPARSTAR_ERR_UNSUPPORTED;
  p.kv_rows = kv_rows;
  p.kv_offset = kv_offset;
  p.kv_capacity = kv_capacity;
  p.status = dev->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Four heads per item keep 64 bytes in flight per lane; with few tokens one head per item
  // spreads the call over more SMs instead (48 heads of 128 in bf16, four against one: 16 tokens 2.24
  // and 1.96 us, 256 tokens 2.90 and 2.83 us, 512 tokens 3.49 and 4.20 us; fp32 crosses there too).
  nr_chunks(&p, 4);
  const bool wide = nr_items(p, head_dim) >= 2 * dev->sms;
  if (!wide) nr_chunks(&p, 1);
  const int64_t items = nr_items(p, head_dim);
  if (items > INT32_MAX) return SPARSTAR_ERR_UNSUPPORTED;
  nr_dispatch(head_dim, x_dtype, interleaved != 0, [&](auto d, auto t, auto il) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    constexpr bool IL = decltype(il)::value;
    const unsigned grid = static_cast<unsigned>(items);
    if (wide)
      norm_rope_kernel<D, T, IL, 4><<<grid, kNrThreads, 0, st>>>(p);
    else
      norm_rope_kernel<D, T, IL, 1><<<grid, kNrThreads, 0, st>>>(p);
  });
  return launch_status();
}

int sparstar_qk_norm_rope_bwd_workspace_size(int head_dim, size_t* bytes) {
  if (bytes == nullptr) return SPARSTAR_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return SPARSTAR_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(kNrMaxParts) * head_dim * sizeof(float);
  return SPARSTAR_OK;
}

int sparstar_qk_norm_rope_bwd(sparstar_view dq, sparstar_view dk, sparstar_view dv, sparstar_view q, sparstar_view k,
                              int x_dtype, int64_t n_tokens, int heads_q, int heads_k, int head_dim, const float* wq,
                              const float* wk, const float* cos, const float* sin, float eps, int interleaved,
                              int64_t kv_offset, sparstar_view dq_in, sparstar_view dk_in, sparstar_view dv_in,
                              float* dwq, float* dwk, void* workspace, size_t workspace_bytes, void* stream) {
  NrParams p;
  int rc = nr_setup({dq_in, dk_in, dv_in}, {dq, dk, dv}, x_dtype, n_tokens, heads_q, heads_k, head_dim, wq, wk, cos,
                    sin, eps, kv_offset, &p);
  if (rc != SPARSTAR_OK) return rc;
  if (dk.seq_stride != 0 || dv.seq_stride != 0 || q.seq_stride != 0 || k.seq_stride != 0) return SPARSTAR_ERR_ARG;
  const int e = x_dtype == SPARSTAR_BF16 ? 2 : 4;
  if (n_tokens > 0 && (!strides_ok(q, e, n_tokens > 1, heads_q > 1) ||
                       (heads_k > 0 && !strides_ok(k, e, n_tokens > 1, heads_k > 1))))
    return SPARSTAR_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(dwq) & 3u) != 0 || (reinterpret_cast<uintptr_t>(dwk) & 3u) != 0)
    return SPARSTAR_ERR_ARG;
  size_t need = 0;
  if ((rc = sparstar_qk_norm_rope_bwd_workspace_size(head_dim, &need)) != SPARSTAR_OK) return rc;
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace)) return SPARSTAR_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != SPARSTAR_OK) return rc;
  if (dev->major != 10) return SPARSTAR_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i) p.dx[i] = p.x[i];
  p.x[0] = view(q);
  p.x[1] = view(k);
  p.kv_offset = kv_offset;
  p.status = dev->status;
  p.dw_part = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Four heads an item in bf16; two where fp32 values would not fit the registers, or where few
  // items leave SMs without one (1,000 tokens x 6 heads fp32: 5.3 us against 6.4 us with four).
  nr_chunks(&p, 4);
  const bool four = x_dtype == SPARSTAR_BF16 && nr_items(p, head_dim) >= kNrBwdCtas * dev->sms;
  if (!four) nr_chunks(&p, 2);
  if (nr_items(p, head_dim) > INT32_MAX) return SPARSTAR_ERR_UNSUPPORTED;
  nr_bwd_grid(&p, head_dim, e, kNrBwdCtas, dev->sms);
  const int grid = p.ctas[0] + p.ctas[1] + p.ctas[2];  // 0 tokens: none, and dw is a sum of nothing
  nr_dispatch(head_dim, x_dtype, interleaved != 0, [&](auto d, auto t, auto il) {
    using T = decltype(t);
    constexpr int D = decltype(d)::value;
    constexpr bool IL = decltype(il)::value;
    if (grid > 0 && four) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value)
        norm_rope_bwd_kernel<D, T, IL, 4><<<grid, kNrThreads, 0, st>>>(p);
    } else if (grid > 0) {
      norm_rope_bwd_kernel<D, T, IL, 2><<<grid, kNrThreads, 0, st>>>(p);
    }
    if (dwq != nullptr || dwk != nullptr)
      launch_after(norm_rope_dw_kernel<D>, dim3(D / 32 * 2), dim3(1024), 0, st, p.dw_part, p.ctas[0], p.ctas[1], dwq,
                   dwk);
  });
  return launch_status();
}

}  // extern "C"
