// 4-bit weights with group scales: the quantiser and the products with activation rows.
//   w[r][k] = scale[r][k / G] * (code[r][k] - 8),   y[n][r] = sum_k x[n][k] * w[r][k]
// Codes are stored in blocks of 128 columns (64 bytes): 32-bit word 4c + j of a block holds the codes
// of columns 32j + 8c .. 32j + 8c + 7 (lowest nibble first), so the 16 bytes at offset 16c are the
// c-th eight columns of each of the block's four 32-column parts.
#include <cuda_runtime.h>

#include <algorithm>
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

// ---------------------------------------------------------------- products
//
// y = x W^T on mma.sync.m16n8k16 (bf16 operands, fp32 sums): 16 weight rows are the A operand, expanded
// from their codes in registers (0x4300 | code is 128 + code in bf16, less 136 exactly), 8 activation
// columns the B operand.  tcgen05 would want the expanded weights in tensor or shared memory first; a
// decode step has 1 to 32 columns, and what bounds it is the reading of the codes.  A 32-bit word of codes
// feeds the k positions of two instructions in the order (0,4)(1,5) | (2,6)(3,7) of its nibbles; the
// activations are staged in that order.
//
// Activations enter in full: an fp16 value is two bf16 terms and an fp32 value three (truncations of what
// is left), each a column of its own, added at the end.  Codes are whole numbers, so products are exact;
// a group's scale multiplies its fp32 sum.
//
// A block takes 128 rows (a warp 16) and a range of the columns of W; the blocks of a cluster split W's
// columns and add their sums through distributed shared memory in rank order.

constexpr int kRows = 128;        // weight rows of a block
constexpr int kChunk = 8;         // code blocks of activations in shared memory at a time
constexpr int kAhead = 4;         // code blocks of weights that a warp has in flight (a chunk is whole turns of them)

template <typename T>
struct Terms;
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int n = 1;
};
template <>
struct Terms<__half> {
  static constexpr int n = 2;
};
template <>
struct Terms<float> {
  static constexpr int n = 3;
};

// the next bf16 term of v (its leading 8 bits; what is not finite whole), which is taken off v
__device__ __forceinline__ uint32_t next_term(float& v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7f800000u) == 0x7f800000u) {
    v = 0.f;
    return (u & 0x7fffffu) ? 0x7fffu : u >> 16;
  }
  v -= __uint_as_float(u & 0xffff0000u);
  return u >> 16;
}

// eight consecutive activations
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f(h[i]);
}

__device__ __forceinline__ void mma_bf16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// nibbles i and i + 4 of w as bf16 code - 8
__device__ __forceinline__ uint32_t expand_q4(uint32_t w, int i) {
  const uint32_t u = (w >> (4 * i) & 0x000f000fu) | 0x43004300u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), __float2bfloat162_rn(136.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(addr), "r"(rank));
  return v;
}

struct MatmulArgs {
  const void* x;
  long long x_stride;
  int n, m, k;
  const uint8_t* codes;
  const __nv_bfloat16* scales;
  void* y;
};

// a warp's part of one code block: 16 bytes of rows g and g + 8 each, and the rows' scales
template <int G>
struct WeightBlock {
  uint4 w[2];
  uint32_t s[2][G == 32 ? 2 : 1];
};

template <typename T, int NT, int G>
__global__ void __launch_bounds__(256) k_q4_matmul(const MatmulArgs a) {
  constexpr int TN = Terms<T>::n;
  constexpr int kCols = 8 * NT / TN;  // activation rows of a pass
  constexpr int kOut = 8 * NT + 1;    // floats of a weight row in the joining buffer
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* xs = reinterpret_cast<uint4*>(smem);  // [code block][32-column part][8-column tile][lane]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int blocks = (a.k + kBlock - 1) / kBlock;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * rank / ranks);
  const int b1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / ranks);
  const int n0 = blockIdx.z * kCols, nn = min(kCols, a.n - n0);
  const int row0 = blockIdx.x * kRows + warp * 16;
  const int ra = min(row0 + g, a.m - 1), rb = min(row0 + g + 8, a.m - 1);
  const uint4* wa = reinterpret_cast<const uint4*>(a.codes) + static_cast<size_t>(ra) * blocks * 4 + c;
  const uint4* wb = reinterpret_cast<const uint4*>(a.codes) + static_cast<size_t>(rb) * blocks * 4 + c;
  constexpr int SB = kBlock / G;  // scales of a block
  const __nv_bfloat16* sa = a.scales + static_cast<size_t>(ra) * blocks * SB;
  const __nv_bfloat16* sb = a.scales + static_cast<size_t>(rb) * blocks * SB;

  auto fetch = [&](WeightBlock<G>& f, int b) {
    if (b >= b1) return;
    f.w[0] = __ldcs(wa + static_cast<size_t>(b) * 4);
    f.w[1] = __ldcs(wb + static_cast<size_t>(b) * 4);
    const __nv_bfloat16* p[2] = {sa + b * SB, sb + b * SB};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (G == 32) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p[r]));
        f.s[r][0] = v.x, f.s[r][1] = v.y;
      } else if constexpr (G == 64) {
        f.s[r][0] = __ldg(reinterpret_cast<const uint32_t*>(p[r]));
      } else {
        f.s[r][0] = __ldg(reinterpret_cast<const uint16_t*>(p[r]));
      }
    }
  };
  auto scale = [](const WeightBlock<G>& f, int r, int part) {  // of 32-column part 0..3
    const int i = part * 32 / G;
    return i % 2 ? bf16hi(f.s[r][i / 2]) : bf16lo(f.s[r][i / 2]);
  };

  WeightBlock<G> ring[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(ring[i], b0 + i);

  float y[NT][4] = {};
  for (int base = b0; base < b1; base += kChunk) {
    const int nb = min(kChunk, b1 - base);
    if (base > b0) __syncthreads();
    // stage the activations: one item is eight columns of W of one row
    const T* x = static_cast<const T*>(a.x);
    for (int i = threadIdx.x; i < nb * 16 * kCols; i += blockDim.x) {
      const int col = i / (nb * 16), part = i % (nb * 16);  // part: 4 * (block, 32-column part) + lane c
      const int k = (base + part / 16) * kBlock + part % 16 * 8;
      float v[8] = {};
      if (col < nn && k < a.k) load8(x + (n0 + col) * a.x_stride + k, v);
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = next_term(v[e]);
        const int j = col * TN + t;
        xs[((part / 4) * NT + j / 8) * 32 + j % 8 * 4 + part % 4] =
            make_uint4(h[0] | h[4] << 16, h[1] | h[5] << 16, h[2] | h[6] << 16, h[3] | h[7] << 16);
      }
    }
    if constexpr (8 * NT % TN != 0) {  // columns that no term fills
      for (int i = threadIdx.x; i < nb * 16; i += blockDim.x)
        for (int j = kCols * TN; j < 8 * NT; ++j)
          xs[((i / 4) * NT + j / 8) * 32 + j % 8 * 4 + i % 4] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int q = 0; q < nb; q += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (q + u >= nb) break;
        const WeightBlock<G> f = ring[u];
        fetch(ring[u], base + q + u + kAhead);
        const uint32_t wv[2][4] = {{f.w[0].x, f.w[0].y, f.w[0].z, f.w[0].w}, {f.w[1].x, f.w[1].y, f.w[1].z, f.w[1].w}};
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          const uint32_t A0[4] = {expand_q4(wv[0][part], 0), expand_q4(wv[1][part], 0), expand_q4(wv[0][part], 1),
                                  expand_q4(wv[1][part], 1)};
          const uint32_t A1[4] = {expand_q4(wv[0][part], 2), expand_q4(wv[1][part], 2), expand_q4(wv[0][part], 3),
                                  expand_q4(wv[1][part], 3)};
          const float s0 = scale(f, 0, part), s1 = scale(f, 1, part);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 b = xs[(((q + u) * 4 + part) * NT + t) * 32 + lane];
            float d[4];
            mma_bf16_zero(d, A0, b.x, b.y);
            mma_bf16_16816(d, A1[0], A1[1], A1[2], A1[3], b.z, b.w);
            y[t][0] += s0 * d[0];
            y[t][1] += s0 * d[1];
            y[t][2] += s1 * d[2];
            y[t][3] += s1 * d[3];
          }
        }
      }
    }
  }
  // join: this block's sums, then every block of the cluster adds up a share of the rows
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[(warp * 16 + g + i / 2 * 8) * kOut + 8 * t + 2 * c + i % 2] = y[t][i];
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  const int share = kRows / ranks;
  for (int i = threadIdx.x; i < share * nn; i += blockDim.x) {
    const int r = rank * share + i % share, col = i / share, row = blockIdx.x * kRows + r;
    if (row >= a.m) continue;
    float v = 0.f;
    const uint32_t at = smem_u32(out + r * kOut + col * TN);
    for (int k = 0; k < ranks; ++k)
#pragma unroll
      for (int t = TN - 1; t >= 0; --t) v += ranks > 1 ? ld_cluster(at + 4 * t, k) : out[r * kOut + col * TN + t];
    static_cast<T*>(a.y)[static_cast<size_t>(n0 + col) * a.m + row] = from_f<T>(v);
  }
  if (ranks > 1) cluster_sync();  // no block leaves while its sums are read
}

template <typename T, int NT, int G>
int launch_matmul(const MatmulArgs& a, cudaStream_t st) {
  constexpr int kCols = 8 * NT / Terms<T>::n;
  constexpr int kXs = kChunk * 4 * NT * 32 * 16, kJoin = kRows * (8 * NT + 1) * 4;
  const int blocks = (a.k + kBlock - 1) / kBlock;
  const int grid = (a.m + kRows - 1) / kRows, passes = (a.n + kCols - 1) / kCols;
  if (passes > 65535) return S2_EINVAL;
  int ranks = 1;
  while (ranks < 8 && static_cast<long long>(grid) * passes * ranks < 152 * 3 && blocks >= 4 * ranks) ranks *= 2;
  const int smem = std::max(std::min(blocks, kChunk) * (kXs / kChunk), kJoin);
  static_assert(kXs <= 200 * 1024 && kJoin <= 200 * 1024, "shared memory");
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_q4_matmul<T, NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, std::max(kXs, kJoin)) !=
          cudaSuccess)
    return S2_ECUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, ranks, passes);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = ranks;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_q4_matmul<T, NT, G>, a) == cudaSuccess ? S2_OK : S2_ECUDA;
}

template <typename T, int G>
int launch_columns(const MatmulArgs& a, cudaStream_t st) {
  const int cols = a.n * Terms<T>::n;  // a pass of the fewest 8-column tiles that hold them, 4 at most
  if (cols <= 8) return launch_matmul<T, 1, G>(a, st);
  if (cols <= 16) return launch_matmul<T, 2, G>(a, st);
  return launch_matmul<T, 4, G>(a, st);
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
      x_stride < k || n > 0x3fffffff || m > 0x3fffffff || k > 0x3fffffff)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % 16 != 0 || x_stride * esz % 16 != 0 ||
      reinterpret_cast<uintptr_t>(codes) % 16 != 0 || reinterpret_cast<uintptr_t>(scales) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(y) % esz != 0)
    return S2_EINVAL;
  const MatmulArgs a{x, x_stride, n, m, k, codes, static_cast<const __nv_bfloat16*>(scales), y};
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return group == 32 ? launch_columns<T, 32>(a, st)
                       : group == 64 ? launch_columns<T, 64>(a, st) : launch_columns<T, 128>(a, st);
  });
}
