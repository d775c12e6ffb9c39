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
constexpr int kPer = kSlice / kAdjustThreads;  // entries of a thread
static_assert(kPer == 8, "16-byte reads and writes");

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

template <int kBytes>
struct Words;
template <>
struct Words<16> {
  using type = uint4;
};
template <>
struct Words<32> {
  struct alignas(16) type {
    uint4 a, b;
  };
};

// One block per (slice, row).  The occurrences of the slice's tokens are counted in shared memory from the row's
// whole history (whole-number adds: the order does not matter) while the slice's logits, bias and mask are on their
// way.  A thread's kPer entries are consecutive and read 16 bytes at a time where rows are aligned to that (kWide);
// else they are 256 apart, so that rows of any alignment are read and written in whole lines.  Bound by those bytes;
// the history is read again by every slice, from L2 (four bytes a token against 20 KB and more).  32 bf16 rows of
// 155776, each with its bias, mask and 2048 tokens: 15.7 us, 3.2 TB/s; 14.2 with part of that in L2, where slices of 1024
// entries took 15.4, of 4096 14.5, of 8192 19.8.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kAdjustThreads) k_adjust(const AdjustArgs a) {
  __shared__ __align__(16) int count[kSlice];
  const size_t r = blockIdx.y;
  const int e0 = blockIdx.x * kSlice, n = min(a.n - e0, kSlice);
  const bool seen = a.history != nullptr;
  const T* x = static_cast<const T*>(a.logits) + r * a.n + e0;
  const float* bias = a.bias ? a.bias + r * a.bias_stride + e0 : nullptr;
  const uint32_t* mask = a.mask ? a.mask + r * a.mask_stride + e0 / 32 : nullptr;
  auto entry = [](int i) { return kWide ? threadIdx.x * kPer + i : i * kAdjustThreads + threadIdx.x; };
  const bool in = entry(0) < n;  // wide rows are whole groups of kPer
  T v[kPer];
  float b[kPer] = {};
  uint32_t m = 0;  // this thread's mask bits
  if constexpr (kWide) {
    using W = typename Words<sizeof(T) * kPer>::type;
    using F = Words<sizeof(float) * kPer>::type;
    if (in) {
      *reinterpret_cast<W*>(v) = *reinterpret_cast<const W*>(x + entry(0));
      if (bias) *reinterpret_cast<F*>(b) = *reinterpret_cast<const F*>(bias + entry(0));
      if (mask) m = __ldg(mask + entry(0) / 32) >> (entry(0) % 32);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = entry(i);
      v[i] = e < n ? x[e] : from_f<T>(0.f);
      if (bias && e < n) b[i] = __ldg(bias + e);
      if (mask && e < n) m |= (__ldg(mask + e / 32) >> (e % 32) & 1u) << i;
    }
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
      if (a.sem_begin >= 0) {
        e -= a.sem_begin;
        if (e >= a.n - 1) e = -1;
        if (id == a.im_end) e = a.n - 1;
      }
      if (e >= e0 && e < e0 + n) atomicAdd(count + (e - e0), 1);
    }
    __syncthreads();
  }
  float* out = a.out + r * a.n + e0;
  float y[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float l = to_f(v[i]);
    const int c = seen ? count[entry(i)] : 0;
    if (c > 0) l = (l > 0.f ? __fdiv_rn(l, rep) : l * rep) - freq * static_cast<float>(c) - pres;
    if (bias) l += b[i];
    if (mask && !(m >> i & 1u)) l = -INFINITY;
    y[i] = l;
    if (!kWide && entry(i) < n) out[entry(i)] = l;
  }
  if (kWide && in) {
    float4* o = reinterpret_cast<float4*>(out + entry(0));
    o[0] = make_float4(y[0], y[1], y[2], y[3]);
    o[1] = make_float4(y[4], y[5], y[6], y[7]);
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
  const bool wide = n % kPer == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(out) % 16 == 0 && reinterpret_cast<uintptr_t>(bias) % 16 == 0 &&
                    bias_stride % 4 == 0;
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const dim3 grid(n / kSlice + (n % kSlice != 0), rows);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (wide)
      k_adjust<T, true><<<grid, kAdjustThreads, 0, st>>>(a);
    else
      k_adjust<T, false><<<grid, kAdjustThreads, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
