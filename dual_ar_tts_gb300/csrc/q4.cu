// 4-bit weights with group scales: the quantiser and the products with activation rows.
//   w[r][k] = scale[r][k / G] * (code[r][k] - 8),   y[n][r] = sum_k x[n][k] * w[r][k]
// Codes are stored in blocks of 128 columns (64 bytes): 32-bit word 4c + j of a block holds the codes
// of columns 32j + 8c .. 32j + 8c + 7 (lowest nibble first), so the 16 bytes at offset 16c are the
// c-th eight columns of each of the block's four 32-column parts.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

constexpr int kBlock = 128;  // columns of a code block

// One warp per block of 128 columns; lane l holds columns 4l .. 4l + 3.  A group's scale is its entry
// of the largest magnitude (the first of equals) divided by -8, rounded to bf16, so that entry takes
// code 0 and the range -8..7 is used whole; the codes are taken against the rounded scale.
template <typename T>
__global__ void __launch_bounds__(256) k_quant_q4(const T* __restrict__ w, long long rows, int cols, int blocks,
                                                  int group, uint8_t* __restrict__ codes,
                                                  __nv_bfloat16* __restrict__ scales) {
  const int lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if (item >= rows * blocks) return;
  const long long r = item / blocks;
  const int b = static_cast<int>(item % blocks);
  float v[4];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = b * kBlock + 4 * lane + i;
    v[i] = k < cols ? to_f(w[r * cols + k]) : 0.f;
    finite = finite && isfinite(v[i]);
  }
  float m = v[0];
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (fabsf(v[i]) > fabsf(m)) m = v[i];
  const int lanes = group / 4;  // 8, 16 or 32
  for (int o = 1; o < lanes; o <<= 1) {
    const float other = __shfl_xor_sync(0xffffffffu, m, o);
    const bool other_first = (lane & o) != 0;
    if (fabsf(other) > fabsf(m) || (fabsf(other) == fabsf(m) && other_first)) m = other;
    finite = __shfl_xor_sync(0xffffffffu, static_cast<int>(finite), o) && finite;
  }
  __nv_bfloat16 sb = __float2bfloat16_rn(m / -8.f);
  if (__bfloat162float(sb) == 0.f) sb = __float2bfloat16_rn(0.f);  // never -0
  if (!finite) sb = __float2bfloat16_rn(NAN);
  const float s = __bfloat162float(sb);
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int c = 8;
    if (finite && s != 0.f) c = static_cast<int>(fminf(fmaxf(rintf(v[i] / s) + 8.f, 0.f), 15.f));
    packed |= static_cast<uint32_t>(c) << (4 * i);
  }
  const int j = lane / 8, c = lane % 8 / 2;
  uint8_t* dst = codes + (r * blocks + b) * (kBlock / 2) + (4 * c + j) * 4 + lane % 2 * 2;
  *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(packed);
  if (lane % lanes == 0) scales[(r * blocks + b) * (kBlock / group) + lane / lanes] = sb;
}

// One warp per weight row, eight activation rows at a time.
template <typename T>
__global__ void __launch_bounds__(256) k_q4_rows(const T* __restrict__ x, long long x_stride, int n,
                                                 const uint8_t* __restrict__ codes,
                                                 const __nv_bfloat16* __restrict__ scales, int m, int k, int group,
                                                 T* __restrict__ y) {
  const int lane = threadIdx.x % 32;
  const int r = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (r >= m) return;
  const int n0 = blockIdx.y * 8, nn = min(8, n - n0);
  const int blocks = (k + kBlock - 1) / kBlock;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(r) * blocks * (kBlock / 2));
  const __nv_bfloat16* sr = scales + static_cast<size_t>(r) * blocks * (kBlock / group);
  float acc[8] = {};
  for (int wi = lane; wi < blocks * 16; wi += 32) {
    const int col = wi / 16 * kBlock + wi % 4 * 32 + wi % 16 / 4 * 8;
    if (col >= k) continue;
    const uint32_t w = words[wi];
    const float s = to_f(sr[col / group]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = s * static_cast<float>(static_cast<int>(w >> (4 * i) & 15) - 8);
    for (int a = 0; a < nn; ++a) {
      const T* xr = x + (n0 + a) * x_stride + col;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[a] += f[i] * to_f(xr[i]);
    }
  }
  for (int a = 0; a < nn; ++a) {
    const float t = warp_sum(acc[a]);
    if (lane == 0) y[static_cast<size_t>(n0 + a) * m + r] = from_f<T>(t);
  }
}

bool bad_group(int group) { return group != 32 && group != 64 && group != 128; }

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_quantize_q4(const void* w, int dtype, long long rows, int cols, int group, uint8_t* codes,
                              void* scales, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (!w || !codes || !scales || !esz || rows < 1 || cols < 1 || bad_group(group) || cols % group != 0)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(w) % esz != 0 || reinterpret_cast<uintptr_t>(codes) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(scales) % 2 != 0)
    return S2_EINVAL;
  const int blocks = cols / kBlock + (cols % kBlock != 0);
  if (rows > 0x7fffffffll * 8 / blocks) return S2_EINVAL;
  const long long grid = (rows * blocks + 7) / 8;
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    k_quant_q4<T><<<static_cast<unsigned>(grid), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(w), rows, cols, blocks, group, codes, static_cast<__nv_bfloat16*>(scales));
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

extern "C" int s2_q4_matmul(int n, const void* x, int dtype, long long x_stride, const uint8_t* codes,
                            const void* scales, int m, int k, int group, void* y, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (!x || !codes || !scales || !y || !esz || n < 1 || m < 1 || k < 1 || bad_group(group) || k % group != 0 ||
      x_stride < k)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % 16 != 0 || x_stride * esz % 16 != 0 ||
      reinterpret_cast<uintptr_t>(codes) % 16 != 0 || reinterpret_cast<uintptr_t>(scales) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(y) % esz != 0)
    return S2_EINVAL;
  if ((n + 7) / 8 > 65535) return S2_EINVAL;
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    k_q4_rows<T><<<dim3((m + 7) / 8, (n + 7) / 8), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const T*>(x), x_stride, n, codes, static_cast<const __nv_bfloat16*>(scales), m, k, group,
        static_cast<T*>(y));
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
