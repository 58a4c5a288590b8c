// Host side of sparstar_attn_bwd: argument checks, workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_bwd_sm100.cuh"
#include "host.h"

namespace sparstar {
namespace {

std::mutex g_attr_mutex;
bool g_attrs_set[kMaxDevices];

template <int D, int B>
int set_attrs() {
  using C = BwdConfig<D, B>;
  auto* kernel = attn_bwd_kernel<D, B>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess)
    return SPARSTAR_ERR_CUDA;
  // setmaxnreg draws on the block's launch allocation: a build with fewer registers would wait
  // there for good, so it is refused before any launch
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess) return SPARSTAR_ERR_CUDA;
  return a.numRegs * C::kThreads < C::kRegsNeeded ? SPARSTAR_ERR_UNSUPPORTED : SPARSTAR_OK;
}

int set_kernel_attrs(const DeviceInfo* dev) {
  std::lock_guard<std::mutex> lock(g_attr_mutex);
  if (g_attrs_set[dev->index]) return SPARSTAR_OK;
  int rc;
  if ((rc = set_attrs<128, 128>()) != SPARSTAR_OK || (rc = set_attrs<64, 128>()) != SPARSTAR_OK ||
      (rc = set_attrs<128, 64>()) != SPARSTAR_OK || (rc = set_attrs<64, 64>()) != SPARSTAR_OK)
    return rc;
  for (auto kernel : {bwd_prep_kernel<128>, bwd_prep_kernel<64>})
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaskMaxBlocks * 4) != cudaSuccess)
      return SPARSTAR_ERR_CUDA;
  g_attrs_set[dev->index] = true;
  return SPARSTAR_OK;
}

// Entries of a part of a list: an SM's share of all entries, so that no list holds a CTA longer than the
// others work, but enough tiles to be worth the sums that a part stores (16 at least; with 8, 12 or 24 the
// 8 heads of 4,096 queries take the same 74 to 76 us). A list of n > part entries makes
// ceil(n / part) < 2 n / part parts: with entries / 148 <= part, below 296 in all. 148: a B200's SMs, a
// constant because a workspace's size is asked for without a device.
int64_t bwd_part_entries(int heads, int64_t nqb, int32_t kmax) {
  const int64_t share = (static_cast<int64_t>(heads) * nqb * kmax + 147) / 148;
  return share < 16 ? 16 : share;
}

// Parts at most: none where no list (of nqb entries, or more only with blocks listed twice) can be that long.
int bwd_parts(int heads, int64_t nqb, int32_t kmax) {
  const int64_t part = bwd_part_entries(heads, nqb, kmax), all = static_cast<int64_t>(heads) * nqb * kmax;
  const int64_t most = nqb * kmax <= part ? 0 : 2 * all / part;
  return static_cast<int>(most < kBwdMaxParts ? most : kBwdMaxParts);
}

struct BwdWorkspace {
  size_t next, done, parts, sums, lse2, delta, words, place, twice, col_at, col_row, total;
};

BwdWorkspace bwd_layout(int heads, int64_t nqb, int64_t nkb, int block, int32_t kmax, int head_dim) {
  const size_t h = static_cast<size_t>(heads);
  const size_t rows = align256(h * nqb * block * 4);
  BwdWorkspace w;
  w.next = 0;
  w.done = 256;
  w.parts = w.done + align256(kBwdMaxParts * 8 * 4);
  w.sums = w.parts + align256(kBwdMaxParts * sizeof(BwdPart));
  w.lse2 = w.sums + static_cast<size_t>(bwd_parts(heads, nqb, kmax)) * 2 * block * head_dim * 4;
  w.delta = w.lse2 + rows;
  const size_t chunks = static_cast<size_t>((nqb + kMaskRows - 1) / kMaskRows);
  w.words = w.delta + rows;
  w.place = w.words + align256(h * chunks * nkb * 4);
  w.twice = w.place + align256(h * chunks * nkb * 4);
  w.col_at = w.twice + align256(h * chunks * 4);
  w.col_row = w.col_at + align256(h * (nkb + 1) * 4);
  w.total = w.col_row + align256(h * nqb * kmax * 4);
  return w;
}

// Sizes that the lists and the launch geometry hold.
int bwd_sizes(int heads, int64_t n_q, int64_t n_kv, int head_dim, int block, int32_t kmax) {
  if (heads < 1 || n_q < 0 || n_kv < 1 || kmax < 1) return SPARSTAR_ERR_ARG;
  if (head_dim != 64 && head_dim != 128) return SPARSTAR_ERR_UNSUPPORTED;
  if (block != 64 && block != 128) return SPARSTAR_ERR_UNSUPPORTED;
  if (n_q > INT32_MAX || n_kv > INT32_MAX || heads > 65535) return SPARSTAR_ERR_UNSUPPORTED;
  const int64_t nqb = ceil_blocks(n_q, block), nkb = ceil_blocks(n_kv, block);
  if (nkb > kMaskMaxBlocks || heads * nqb > INT32_MAX / 2 || heads * nkb > INT32_MAX / 2 || nqb * kmax > INT32_MAX)
    return SPARSTAR_ERR_UNSUPPORTED;
  return SPARSTAR_OK;
}

template <int D, int B>
void launch_bwd(const BwdMaps& maps, const BwdParams& p, int sms, cudaStream_t st) {
  using C = BwdConfig<D, B>;
  const int items = p.n_dkv + p.n_dq;
  launch_after(attn_bwd_kernel<D, B>, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(C::kThreads),
               C::kSmemBytes, st, maps, p);
}

}  // namespace
}  // namespace sparstar

using namespace sparstar;

extern "C" {

int sparstar_attn_bwd_workspace_size(int heads, int64_t n_q, int64_t n_kv, int head_dim, int block, int32_t kmax,
                                     size_t* bytes) {
  if (bytes == nullptr) return SPARSTAR_ERR_ARG;
  const int rc = bwd_sizes(heads, n_q, n_kv, head_dim, block, kmax);
  if (rc != SPARSTAR_OK) return rc;
  *bytes = bwd_layout(heads, ceil_blocks(n_q, block), ceil_blocks(n_kv, block), block, kmax, head_dim).total;
  return SPARSTAR_OK;
}

int sparstar_attn_bwd(const void* d_o, const void* q, const void* k, const void* v, const void* o, const float* lse,
                      int heads, int64_t n_q, int64_t n_kv, int head_dim, int block, const int32_t* idx,
                      const int32_t* cnt, int32_t kmax, float sm_scale, void* dq, void* dk, void* dv, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = bwd_sizes(heads, n_q, n_kv, head_dim, block, kmax);
  if (rc != SPARSTAR_OK) return rc;
  if (!(sm_scale == sm_scale) || std::isinf(sm_scale)) return SPARSTAR_ERR_ARG;
  if (dk == nullptr || dv == nullptr || !aligned16(dk) || !aligned16(dv)) return SPARSTAR_ERR_ARG;
  if (n_q > 0) {
    for (const void* ptr : {d_o, q, k, v, o, static_cast<const void*>(dq)})
      if (ptr == nullptr || !aligned16(ptr)) return SPARSTAR_ERR_ARG;
    if (lse == nullptr || idx == nullptr || cnt == nullptr || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(idx) & 3u) != 0 || (reinterpret_cast<uintptr_t>(cnt) & 3u) != 0)
      return SPARSTAR_ERR_ARG;
  }
  const int64_t nqb = ceil_blocks(n_q, block), nkb = ceil_blocks(n_kv, block);
  const BwdWorkspace ws = bwd_layout(heads, nqb, nkb, block, kmax, head_dim);
  if (n_q > 0 && (workspace == nullptr || workspace_bytes < ws.total ||
                  (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
    return SPARSTAR_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  if ((rc = device_info(&dev)) != SPARSTAR_OK) return rc;
  if (dev->major != 10) return SPARSTAR_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n_q == 0) {  // no query attends to anything: the gradients of k and v are zero
    const size_t bytes = static_cast<size_t>(heads) * n_kv * head_dim * 2;
    return cudaMemsetAsync(dk, 0, bytes, st) == cudaSuccess && cudaMemsetAsync(dv, 0, bytes, st) == cudaSuccess
               ? SPARSTAR_OK
               : SPARSTAR_ERR_CUDA;
  }
  if ((rc = set_kernel_attrs(dev)) != SPARSTAR_OK) return rc;
  BwdMaps maps;
  const void* base[4] = {q, d_o, k, v};
  for (int i = 0; i < 4; ++i) {
    const int64_t rows = i < 2 ? n_q : n_kv;
    if ((rc = make_map(&maps.walk[i], base[i], rows, heads, head_dim, static_cast<unsigned>(block))) != SPARSTAR_OK ||
        (rc = make_map(&maps.held[i], base[i], rows, heads, head_dim)) != SPARSTAR_OK)
      return rc;
  }
  uint8_t* w = static_cast<uint8_t*>(workspace);
  BwdPrep r = {};
  r.o = static_cast<const __nv_bfloat16*>(o);
  r.d_o = static_cast<const __nv_bfloat16*>(d_o);
  r.lse = lse;
  r.idx = idx;
  r.cnt = cnt;
  r.neg_lse2 = reinterpret_cast<float*>(w + ws.lse2);
  r.neg_delta = reinterpret_cast<float*>(w + ws.delta);
  r.words = reinterpret_cast<uint32_t*>(w + ws.words);
  r.place = reinterpret_cast<int32_t*>(w + ws.place);
  r.twice = reinterpret_cast<int32_t*>(w + ws.twice);
  r.col_at = reinterpret_cast<int32_t*>(w + ws.col_at);
  r.col_row = reinterpret_cast<int32_t*>(w + ws.col_row);
  r.parts = reinterpret_cast<BwdPart*>(w + ws.parts);
  r.part_done = reinterpret_cast<int*>(w + ws.done);
  const int64_t part = bwd_part_entries(heads, nqb, kmax);
  r.part_ent = static_cast<int>(part < INT32_MAX ? part : INT32_MAX);
  r.next = reinterpret_cast<int*>(w + ws.next);
  r.status = dev->status;
  r.n_q = n_q;
  r.n_pad = nqb * block;
  r.heads = heads;
  r.nqb = static_cast<int>(nqb);
  r.nkb = static_cast<int>(nkb);
  r.kmax = kmax;
  r.n_chunks = static_cast<int>((nqb + kMaskRows - 1) / kMaskRows);
  BwdParams p = {};
  p.idx = idx;
  p.cnt = cnt;
  p.col_row = r.col_row;
  p.col_at = r.col_at;
  p.neg_lse2 = r.neg_lse2;
  p.neg_delta = r.neg_delta;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.status = dev->status;
  p.next = r.next;
  p.parts = r.parts;
  p.part_done = r.part_done;
  p.part_sum = reinterpret_cast<float*>(w + ws.sums);
  p.part_ent = r.part_ent;
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.nqb = r.nqb;
  p.nkb = r.nkb;
  p.kmax = kmax;
  p.n_dkv = static_cast<int>(heads * nkb);
  p.n_dq = static_cast<int>(heads * nqb);
  p.scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
  p.scale_log2 = p.scale * 1.4426950408889634f;

  const int rows_per_cta = 256 / (head_dim / 8);
  const int64_t row_tiles = (r.n_pad + rows_per_cta - 1) / rows_per_cta * heads;
  const int64_t row_ctas = row_tiles < 16 * dev->sms ? row_tiles : 16 * dev->sms;
  const unsigned prep_grid = static_cast<unsigned>(static_cast<int64_t>(r.n_chunks) * heads + row_ctas);
  const size_t word_bytes = static_cast<size_t>(nkb) * 4;
  if (head_dim == 128)
    bwd_prep_kernel<128><<<prep_grid, 256, word_bytes, st>>>(r);
  else
    bwd_prep_kernel<64><<<prep_grid, 256, word_bytes, st>>>(r);
  launch_after(bwd_lists_kernel, dim3(static_cast<unsigned>(heads)), dim3(1024), 0, st, r);
  if (head_dim == 128) {
    if (block == 128)
      launch_bwd<128, 128>(maps, p, dev->sms, st);
    else
      launch_bwd<128, 64>(maps, p, dev->sms, st);
  } else {
    if (block == 128)
      launch_bwd<64, 128>(maps, p, dev->sms, st);
    else
      launch_bwd<64, 64>(maps, p, dev->sms, st);
  }
  return launch_status();
}

}  // extern "C"
