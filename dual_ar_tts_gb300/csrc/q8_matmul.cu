// Products of 8-bit integers with a scale for each activation row and each weight row:
//   y[n][r] = xs[n] ws[r] sum_k xc[n][k] wc[r][k]
// The sum is the exact integer.  sm_103a's tensor cores have next to no rate for 8-bit integers (mma.sync on s8 and dp4a
// both measured 256 products a clock and SM; fp16 has 1024 on mma.sync and 4096 on tcgen05), so codes are expanded to fp16,
// which holds them exactly; a product has 14 bits, and fp32 holds the sum of 1024 of them exactly (2^24).  Every 1024
// columns (a chunk) the sums go over to 32-bit integers.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"
#include "tc05.cuh"

namespace s2 {
namespace {

constexpr int kStep = 128;    // columns of a step
constexpr int kChunk = 8;     // steps of a chunk

struct Q8Args {
  const int8_t* x;
  const float* xs;
  const int8_t* w;
  const float* ws;
  void* y;
  int n, m, k;
};

// Four codes as two pairs of fp16.  A code's byte with its sign bit turned is code + 128, as the low byte of fp16's
// 1024 + that: one subtraction gives the code.
__device__ __forceinline__ void expand(uint32_t w, uint32_t& a, uint32_t& b) {
  const uint32_t u = w ^ 0x80808080u, base = 0x64806480u;  // 1152 twice
  const uint32_t p = __byte_perm(u, 0x64646464u, 0x5140), q = __byte_perm(u, 0x64646464u, 0x5342);
  const __half2 z = *reinterpret_cast<const __half2*>(&base);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&p), z), s = __hsub2(*reinterpret_cast<const __half2*>(&q), z);
  a = *reinterpret_cast<const uint32_t*>(&r);
  b = *reinterpret_cast<const uint32_t*>(&s);
}

// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void* gmem, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster_int(uint32_t addr, uint32_t rank) {
  int v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(addr), "r"(rank));
  return v;
}

template <typename T>
__device__ __forceinline__ T scaled(int sum, float xs, float ws) {
  return from_f<T>(__int2float_rn(sum) * xs * ws);
}

// ---- up to 32 activation rows (columns of the product): mma.sync.m16n8k16.
//
// A warp takes 16 weight rows, a block 128, its columns in steps of 128; the blocks of a cluster split W's columns and
// add up through distributed shared memory.  Weights come through a warp's own ring of cp.async, kAhead steps deep.  The
// activations of a chunk are expanded once a block, laid out as the lanes' B operands.  K is permuted alike in both
// operands: lane c of a row's four holds 16 consecutive columns of 64, and a word of them is its part of one product.
constexpr int kFewWarps = 8, kFewRows = 16 * kFewWarps, kFewAhead = 4;
constexpr int kFewRing = kFewWarps * kFewAhead * 16 * kStep;
constexpr int kJoinRow = kFewRows + 4;
template <int NT>
constexpr int kFewBytes = kFewRing + kChunk * 2 * NT * 1024;

template <typename T, int NT>
__global__ void __launch_bounds__(32 * kFewWarps) k_q8_few(const Q8Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int ranks = gridDim.y, rank = blockIdx.y, n0 = blockIdx.z * NT * 8, nn = min(NT * 8, a.n - n0);
  const int steps = (a.k + kStep - 1) / kStep;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * rank / ranks);
  const int count = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / ranks) - s0;
  const int row0 = blockIdx.x * kFewRows + warp * 16;
  uint8_t* ring = smem + warp * kFewAhead * 16 * kStep;
  uint8_t* xb = smem + kFewRing;

  // copies: eight lanes a row of 128 bytes; odd rows have their halves swapped, so that a quarter of a warp reads
  // 16-byte pieces of two rows without a conflict
  const uint32_t to = smem_u32(ring) + lane / 8 * kStep + (((lane % 8) ^ (lane / 8 % 2 * 4)) * 16);
  const int at = s0 * kStep + lane % 8 * 16;
  const int8_t* from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) from[i] = a.w + static_cast<size_t>(min(row0 + lane / 8 + 4 * i, a.m - 1)) * a.k;
  auto issue = [&](int j) {
    if (j < count) {
      const int col = at + j * kStep;
      const bool live = col < a.k;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cp_async16_or_zero(to + j % kFewAhead * 16 * kStep + i * 4 * kStep, from[i] + (live ? col : 0), live);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kFewAhead - 1; ++i) issue(i);

  int sum[NT][4] = {};
  for (int j0 = 0; j0 < count; j0 += kChunk) {
    const int here = min(kChunk, count - j0);
    __syncthreads();  // the chunk before is used up
#pragma unroll 4
    for (int i = warp; i < here * 2 * NT; i += kFewWarps) {  // (64 columns, tile)
      const int half = i / NT, col = i % NT * 8 + g, k = (s0 + j0) * kStep + half * 64 + c * 16;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (col < nn && k < a.k)
        v = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(n0 + col) * a.k + k));
      uint4 p, q;
      expand(v.x, p.x, p.y);
      expand(v.y, p.z, p.w);
      expand(v.z, q.x, q.y);
      expand(v.w, q.z, q.w);
      uint4* dst = reinterpret_cast<uint4*>(xb + i * 1024) + lane;
      dst[0] = p;
      dst[32] = q;
    }
    __syncthreads();
    float z[NT][4] = {};
    for (int j = j0; j < j0 + here; ++j) {
      issue(j + kFewAhead - 1);
      cp_async_wait_group<kFewAhead - 1>();
      __syncwarp();
      const uint32_t w = smem_u32(ring) + j % kFewAhead * 16 * kStep + g * kStep;
      const uint32_t x = smem_u32(xb) + (j - j0) * 2 * NT * 1024 + lane * 16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t o = ((c + 4 * half) ^ (g % 2 * 4)) * 16;
        const uint4 u = lds128(w + o), v = lds128(w + 8 * kStep + o);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t p[4], q[4];
          expand(uu[2 * i], p[0], p[1]);
          expand(uu[2 * i + 1], p[2], p[3]);
          expand(vv[2 * i], q[0], q[1]);
          expand(vv[2 * i + 1], q[2], q[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 b = lds128(x + (half * NT + t) * 1024 + i * 512);
            mma_f16_16816(z[t], p[0], q[0], p[1], q[1], b.x, b.y);
            mma_f16_16816(z[t], p[2], q[2], p[3], q[3], b.z, b.w);
          }
        }
      }
      __syncwarp();  // the ring's place may be filled again
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[t][i] += __float2int_rn(z[t][i]);
  }
  cp_async_wait_all();
  __syncthreads();
  int* out = reinterpret_cast<int*>(smem);  // [column][row]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[(8 * t + 2 * c + i % 2) * kJoinRow + warp * 16 + g + i / 2 * 8] = sum[t][i];
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  const int first = kFewRows * rank / ranks, mine = kFewRows * (rank + 1) / ranks - first;
  for (int i = threadIdx.x; i < mine * nn; i += 32 * kFewWarps) {
    const int r = first + i % mine, col = i / mine, row = blockIdx.x * kFewRows + r;
    int v = 0;
    if (ranks > 1) {
      int u[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) u[q] = q < ranks ? ld_cluster_int(smem_u32(out + col * kJoinRow + r), q) : 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += u[q];
    } else {
      v = out[col * kJoinRow + r];
    }
    if (row < a.m)
      static_cast<T*>(a.y)[static_cast<size_t>(n0 + col) * a.m + row] = scaled<T>(v, __ldg(a.xs + n0 + col), __ldg(a.ws + row));
  }
  if (ranks > 1) cluster_sync();  // no block leaves while its sums are read
}

int launch_clusters(void (*kernel)(Q8Args), dim3 grid, int threads, int smem, int ranks, const Q8Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = ranks;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? S2_OK : S2_ECUDA;
}

template <typename T, int NT>
int launch_few(const Q8Args& a, cudaStream_t st) {
  const int rows = (a.m + kFewRows - 1) / kFewRows, cols = (a.n + NT * 8 - 1) / (NT * 8), steps = (a.k + kStep - 1) / kStep;
  // two blocks an SM (one, where it holds no more), of two steps at least
  const long long groups = static_cast<long long>(rows) * cols;
  const int ranks = std::max(1, std::min({8, static_cast<int>((NT == 4 ? 152 : 304) / groups), steps / 2}));
  if (!allow_smem<k_q8_few<T, NT>, kFewBytes<NT>>()) return S2_ECUDA;
  return launch_clusters(k_q8_few<T, NT>, dim3(rows, ranks, cols), 32 * kFewWarps, kFewBytes<NT>, ranks, a, st);
}

constexpr int kRowsMost = (1 << 21) - 32, kOutMost = 1 << 28, kColsMost = (1 << 17) - 16;  // activation and weight rows; columns

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_q8_matmul(int n, const int8_t* x_codes, const float* x_scales, const int8_t* codes, const float* scales,
                            int m, int k, void* y, int dtype, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (!x_codes || !x_scales || !codes || !scales || !y || !esz || n < 1 || m < 1 || k < 16 || k % 16 != 0 ||
      n > kRowsMost || m > kOutMost || k > kColsMost)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(x_codes) % 16 != 0 || reinterpret_cast<uintptr_t>(codes) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(x_scales) % 4 != 0 || reinterpret_cast<uintptr_t>(scales) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(y) % esz != 0)
    return S2_EINVAL;
  const Q8Args a{x_codes, x_scales, codes, scales, y, n, m, k};
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return n <= 8 ? launch_few<T, 1>(a, st) : n <= 16 ? launch_few<T, 2>(a, st) : launch_few<T, 4>(a, st);
  });
}
