// Host-side helpers shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/wkv.h"

namespace wkv {

// Records a CUDA runtime error for wkv_last_cuda_error (defined in
// wkv_api.cu); true for cudaSuccess.
bool cuda_ok(cudaError_t e);

// Status of the <<<>>> launch just made.
inline wkv_status launch_result() { return cuda_ok(cudaGetLastError()) ? WKV_OK : WKV_ERR_CUDA; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Launches a kernel that begins with follow_on() (wkv_pair.cuh): its CTAs may
// take their places while the kernel before it on the stream still runs, and
// wait there until that one has ended. Hides the launch between two kernels of
// the library.
template <typename... P, typename... A>
wkv_status launch_follow_on(void (*fn)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cuda_ok(cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...)) ? WKV_OK : WKV_ERR_CUDA;
}

constexpr uint64_t kDefaultTimeoutNs = 1000000000ull;  // 1 s, the limit of every device-side wait

}  // namespace wkv
