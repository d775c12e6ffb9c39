// Element types of the stateless operators: a value of S2_F32 / S2_BF16 / S2_F16 as fp32 and back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "../../include/s2frame.h"
#include "ptx.cuh"

namespace s2 {

inline std::atomic<int> wait_tries{kWaitTries};  // of the device waits of calls launched from here on

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

inline int dtype_bytes(int dtype) { return dtype == S2_F32 ? 4 : dtype == S2_BF16 || dtype == S2_F16 ? 2 : 0; }

// f(T{}) with T the C++ type of `dtype` (checked by the caller with dtype_bytes)
template <typename F>
inline auto with_dtype(int dtype, F f) {
  if (dtype == S2_F32) return f(float{});
  if (dtype == S2_BF16) return f(__nv_bfloat16{});
  return f(__half{});
}

// Lets a kernel be launched with up to kMost bytes of dynamic shared memory on the current device.  The limit is set
// once for a device (setting it again would cost every launch about a microsecond).
template <auto kKernel, int kMost>
inline bool allow_smem() {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

}  // namespace s2
