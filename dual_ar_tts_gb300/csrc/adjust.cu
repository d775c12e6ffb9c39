// Logits rows adjusted before a draw: penalties for repeated tokens, a bias and a grammar mask.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

constexpr int kSlice = 2048;    // entries of a row that one block takes
constexpr int kAdjustThreads = 256;
constexpr int kPer = kSlice / kAdjustThreads;

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

// One block per (slice, row).  The occurrences of the slice's tokens are counted in shared memory from the row's
// whole history (whole-number adds: the order does not matter) while the slice's logits, bias and mask are on their
// way; entry e0 + 256 i + t is thread t's, so rows of any alignment are read and written in whole lines.  Bound by
// those bytes; the history is read again by every slice, from L2 (four bytes a token against 20 KB and more).
template <typename T>
__global__ void __launch_bounds__(kAdjustThreads) k_adjust(const AdjustArgs a) {
  __shared__ int count[kSlice];
  const size_t r = blockIdx.y;
  const int e0 = blockIdx.x * kSlice, n = min(a.n - e0, kSlice);
  const bool seen = a.history != nullptr;
  const T* x = static_cast<const T*>(a.logits) + r * a.n + e0;
  const float* bias = a.bias ? a.bias + r * a.bias_stride + e0 : nullptr;
  const uint32_t* mask = a.mask ? a.mask + r * a.mask_stride : nullptr;
  T v[kPer];
  float b[kPer];
  uint32_t m[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kAdjustThreads + threadIdx.x;
    v[i] = e < n ? x[e] : from_f<T>(0.f);
    b[i] = bias && e < n ? __ldg(bias + e) : 0.f;
    m[i] = mask && e < n ? __ldg(mask + (e0 + e) / 32) : ~0u;
  }
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (seen) {
    rep = __ldg(a.penalties + 3 * r), freq = __ldg(a.penalties + 3 * r + 1), pres = __ldg(a.penalties + 3 * r + 2);
    const int len = min(max(a.hist_len ? __ldg(a.hist_len + r) : a.hist_cols, 0), a.hist_cols);
#pragma unroll
    for (int i = 0; i < kPer; ++i) count[i * kAdjustThreads + threadIdx.x] = 0;
    __syncthreads();
    const int32_t* h = a.history + r * a.hist_cols;
#pragma unroll 8
    for (int i = threadIdx.x; i < len; i += kAdjustThreads) {
      const int id = __ldg(h + i);
      // in 64 bits: any 32-bit id may be there
      long long e = id;
      if (a.sem_begin >= 0)
        e = id == a.im_end ? a.n - 1 : (static_cast<long long>(id) - a.sem_begin < a.n - 1 ? static_cast<long long>(id) - a.sem_begin : -1);
      if (e >= e0 && e < e0 + n) atomicAdd(count + (e - e0), 1);
    }
    __syncthreads();
  }
  float* out = a.out + r * a.n + e0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * kAdjustThreads + threadIdx.x;
    if (e >= n) break;
    float l = to_f(v[i]);
    const int c = seen ? count[e] : 0;
    if (c > 0) l = (l > 0.f ? __fdiv_rn(l, rep) : l * rep) - freq * static_cast<float>(c) - pres;
    if (bias) l += b[i];
    if (!(m[i] >> ((e0 + e) % 32) & 1u)) l = -INFINITY;
    out[e] = l;
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
    k_adjust<T><<<dim3(n / kSlice + (n % kSlice != 0), rows), kAdjustThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
