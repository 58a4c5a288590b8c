// Host-side helpers shared by the library's translation units: device record, tensor maps,
// argument checks, launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <utility>

#include "sparstar.h"

namespace sparstar {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  int index = 0;
  int major = 0, minor = 0, sms = 0;
  unsigned* status = nullptr;  // the device's status word
  bool attrs_set = false;
};

// Record of the current device (filled on its first use). Defined in sparstar.cu.
int device_info(DeviceInfo** out);

// Tensor map of a contiguous bf16 [heads][rows][d] array; box = 64 elements x box_rows rows x
// 1 head, 128-byte swizzle, rows out of range read as zero. Defined in sparstar.cu.
int make_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int d, unsigned box_rows = 128);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_blocks(int64_t n, int64_t block = SPARSTAR_BLOCK) { return (n + block - 1) / block; }
inline size_t align256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
inline int launch_status() { return cudaGetLastError() == cudaSuccess ? SPARSTAR_OK : SPARSTAR_ERR_CUDA; }

// Launch with programmatic stream serialization: the kernel may be scheduled while the
// previous kernel of the stream drains; it calls griddep_wait() before reading that
// kernel's output.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace sparstar
