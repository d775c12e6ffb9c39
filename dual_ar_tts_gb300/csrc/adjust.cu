// Logits rows adjusted before a draw: penalties for repeated tokens, a bias and a grammar mask.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

constexpr int kSlice = 2048;  // entries of a row that one CTA takes

struct AdjustArgs {
  int n, sem_begin, im_end;
  const void* logits;
  const int32_t* history;
  const int32_t* hist_len;
  int hist_cols;
  const float* penalties;
  const float* bias;
  long long bias_stride;
  const uint32_t* mask;
  long long mask_stride;
  float* out;
};

// One CTA per (slice, row).  The occurrences of the slice's tokens are counted in shared memory from
// the row's whole history (whole-number adds: the order does not matter), then the slice is streamed.
template <typename T>
__global__ void __launch_bounds__(256) k_adjust(const AdjustArgs a) {
  __shared__ int count[kSlice];
  const size_t r = blockIdx.y;
  const int e0 = blockIdx.x * kSlice, e1 = min(a.n, e0 + kSlice);
  const bool seen = a.history != nullptr && a.penalties != nullptr;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (seen) {
    for (int i = threadIdx.x; i < kSlice; i += blockDim.x) count[i] = 0;
    rep = a.penalties[3 * r];
    freq = a.penalties[3 * r + 1];
    pres = a.penalties[3 * r + 2];
    __syncthreads();
    const int len = min(max(a.hist_len ? a.hist_len[r] : a.hist_cols, 0), a.hist_cols);
    for (int i = threadIdx.x; i < len; i += blockDim.x) {
      const long long id = a.history[r * a.hist_cols + i];
      long long e = id;
      if (a.sem_begin >= 0) e = id == a.im_end ? a.n - 1 : (id - a.sem_begin < a.n - 1 ? id - a.sem_begin : -1);
      if (e >= e0 && e < e1) atomicAdd(count + (e - e0), 1);
    }
    __syncthreads();
  }
  const T* x = static_cast<const T*>(a.logits) + r * a.n;
  for (int e = e0 + threadIdx.x; e < e1; e += blockDim.x) {
    float v = to_f(x[e]);
    const int c = seen ? count[e - e0] : 0;
    if (c > 0) v = (v > 0.f ? __fdiv_rn(v, rep) : v * rep) - freq * static_cast<float>(c) - pres;
    if (a.bias) v += a.bias[r * a.bias_stride + e];
    if (a.mask && !(a.mask[r * a.mask_stride + e / 32] >> (e % 32) & 1u)) v = -INFINITY;
    a.out[r * a.n + e] = v;
  }
}

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_adjust_logits(int rows, int n, int sem_begin, int im_end, const void* logits, int dtype,
                                const int32_t* history, const int32_t* hist_len, int hist_cols,
                                const float* penalties, const float* bias, long long bias_stride,
                                const uint32_t* mask, long long mask_stride, float* out, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (rows < 1 || n < 1 || !logits || !esz || !out || rows > 65535) return S2_EINVAL;
  if (sem_begin >= 0 && n < 2) return S2_EINVAL;
  if ((history != nullptr) != (penalties != nullptr) || (history && hist_cols < 1)) return S2_EINVAL;
  if ((bias && bias_stride != 0 && bias_stride < n) || (mask && mask_stride != 0 && mask_stride < n / 32 + (n % 32 != 0)))
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(logits) % esz != 0) return S2_EINVAL;
  for (const void* p : {static_cast<const void*>(history), static_cast<const void*>(hist_len),
                        static_cast<const void*>(penalties), static_cast<const void*>(bias),
                        static_cast<const void*>(mask), static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return S2_EINVAL;
  const AdjustArgs a{n, sem_begin, im_end, logits, history, hist_len, hist_cols, penalties, bias, bias_stride,
                     mask, mask_stride, out};
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    k_adjust<T><<<dim3(n / kSlice + (n % kSlice != 0), rows), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
