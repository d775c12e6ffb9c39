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
  int tries;  // of a wait
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

// ---- more activation rows: tcgen05, its A operand the weights, B the activations.
//
// A block takes 128 weight rows and N activation rows.  Twice four warps expand steps in turn: a thread a weight row to fp16
// in tensor memory, and a share of the activations into the swizzled tiles that the tensor core reads.  A ninth warp issues
// the products.  Sums of a chunk are exact; two places in tensor memory take chunks in turn, and the expanding warps add
// the one that is done to their integers while the other is filled.  The blocks of a cluster split W's columns.
template <int N>
struct Tc {
  static constexpr int kStages = N == 128 ? 3 : 4;                  // expanded steps: 64 tensor memory columns and B each
  static constexpr int kAhead = 3;                                  // steps of a warp's weights
  static constexpr int kBBytes = N * 256, kWarpRow = 32 * kStep;
  static constexpr int kRing = kStages * kBBytes, kBars = kRing + 8 * kAhead * kWarpRow, kBytes = kBars + 128 + 1024;
  static constexpr uint32_t kCols = 512, kA = 2 * N;                // tensor memory: two places for sums, then A
  static_assert(kA + 64 * kStages <= kCols && N * 128 * 4 <= kBars, "room");
};

constexpr int kTcThreads = 288;
template <typename T, int N>
__global__ void __launch_bounds__(kTcThreads, 1) k_q8_tc(const Q8Args a) {
  using M = Tc<N>;
  extern __shared__ __align__(16) uint8_t smraw[];
  __shared__ int failed;
  uint8_t* sm = smraw + (-smem_u32(smraw) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + M::kBars);  // [j % kStages]: step j is expanded
  uint64_t* empty = full + M::kStages;                          // and used up
  uint64_t *done = empty + M::kStages, *taken = done + 2;       // [chunk % 2]: its products; its sums read
  uint64_t* drained = taken + 2;                                // nothing under way
  uint32_t* tbase = reinterpret_cast<uint32_t*>(drained + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int steps = (a.k + kStep - 1) / kStep;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * rank / ranks);
  const int count = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / ranks) - s0;
  const int chunks = (count + kChunk - 1) / kChunk;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < M::kStages; ++i) {
      mbar_init(full + i, 4);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(done + i, 1);
      mbar_init(taken + i, 8);
    }
    mbar_init(drained, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tbase, M::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tbase, 0);

  bool ok = true;
  const int n0 = blockIdx.z * N, nn = min(N, a.n - n0), wg = warp / 4;
  int sum[N / 2] = {};  // of this thread's row, half of the columns
  if (warp == 8) {
    // ---------------------------------------------------------------- issuing the products
    if (elect_one()) {
      for (int j = 0; j < count; ++j) {
        const int s = j % M::kStages, chunk = j / kChunk;
        ok = mbar_wait_short(full + s, j / M::kStages & 1, a.tries) &&
             (j % kChunk || chunk < 2 || mbar_wait_short(taken + chunk % 2, (chunk / 2 - 1) & 1, a.tries));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = tm + M::kA + s * 64, td = tm + chunk % 2 * N;
        const uint64_t b = desc_sw128(smem_u32(sm + s * M::kBBytes));
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          tc_mma_tmem_a(td, ta + k * 8, b + ((k / 4 * (N * 128) + k % 4 * 32) >> 4), idesc_f16(128, N), j % kChunk > 0 || k > 0);
        tc_commit(empty + s);
        if (j == count - 1 || j % kChunk == kChunk - 1) tc_commit(done + chunk % 2);
      }
      tc_commit(drained);  // no end before that of the products, whoever gave up
      mbar_wait_short(drained, 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- expanding
    const int mine = (count - wg + 1) / 2;  // the steps 2 t + wg
    const int in = warp % 4 * 32, row0 = blockIdx.x * 128 + in, tid = threadIdx.x % 128;
    // weights: eight lanes a row of 128 bytes, its 16-byte pieces swizzled by the row
    const uint32_t ring = smem_u32(sm + M::kRing + warp * M::kAhead * M::kWarpRow);
    const int8_t* from[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) from[i] = a.w + static_cast<size_t>(min(row0 + i * 4 + lane / 8, a.m - 1)) * a.k;
    auto issue = [&](int t) {
      if (t < mine) {
        const uint32_t dst = ring + t % M::kAhead * M::kWarpRow;
        const int col = (s0 + 2 * t + wg) * kStep + lane % 8 * 16;
        const bool live = col < a.k;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + lane / 8;
          cp_async16_or_zero(dst + r * kStep + ((lane % 8) ^ (r & 7)) * 16, from[i] + (live ? col : 0), live);
        }
      }
      cp_async_commit();
    };
    // activations: four lanes 64 bytes of a row
    constexpr int kLoads = N / 16;
    uint4 held[kLoads];
    auto load = [&](int t) {
      const int col = (s0 + 2 * t + wg) * kStep + tid % 4 * 16;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i / 2 * 32 + tid / 4, at = col + i % 2 * 64;
        held[i] = make_uint4(0, 0, 0, 0);
        if (t < mine && r < nn && at < a.k)
          held[i] = __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(n0 + r) * a.k + at));
      }
    };
    // adds a chunk's sums, which makes room for the chunk after the next
    auto take = [&](int chunk) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_short(done + chunk % 2, chunk / 2 & 1, a.tries));
      if (!ok) return;
      tc_fence_after();
      const uint32_t at = tm + (static_cast<uint32_t>(in) << 16) + chunk % 2 * N + wg * (N / 2);
#pragma unroll
      for (int i = 0; i < N / 32; ++i) {
        float v[16];
        tmem_ld16(at + i * 16, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[i * 16 + e] += __float2int_rn(v[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(taken + chunk % 2);
    };
#pragma unroll
    for (int i = 0; i < M::kAhead - 1; ++i) issue(i);
    load(0);
    const uint32_t tlane = tm + M::kA + (static_cast<uint32_t>(in) << 16);
    int next = 0;  // chunk to take
    for (int t = 0; t < mine; ++t) {
      const int j = 2 * t + wg, s = j % M::kStages;
      issue(t + M::kAhead - 1);
      cp_async_wait_group<M::kAhead - 1>();
      __syncwarp();
      const uint32_t at = ring + t % M::kAhead * M::kWarpRow + lane * kStep;
      uint4 w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = lds128(at + ((c ^ (lane & 7)) * 16));
      __syncwarp();  // the ring's place may be filled again
      if (j >= M::kStages) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait_short(empty + s, (j / M::kStages - 1) & 1, a.tries));
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = w[half * 4 + c];
          expand(x.x, r[c * 8], r[c * 8 + 1]);
          expand(x.y, r[c * 8 + 2], r[c * 8 + 3]);
          expand(x.z, r[c * 8 + 4], r[c * 8 + 5]);
          expand(x.w, r[c * 8 + 6], r[c * 8 + 7]);
        }
        tmem_st32(tlane + s * 64 + half * 32, r);
      }
      uint8_t* b = sm + s * M::kBBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i / 2 * 32 + tid / 4, c = tid % 4 * 2;
        uint4 p, q;
        expand(held[i].x, p.x, p.y);
        expand(held[i].y, p.z, p.w);
        expand(held[i].z, q.x, q.y);
        expand(held[i].w, q.z, q.w);
        uint8_t* dst = b + i % 2 * (N * 128) + r * 128;
        *reinterpret_cast<uint4*>(dst + ((c ^ (r & 7)) * 16)) = p;
        *reinterpret_cast<uint4*>(dst + (((c + 1) ^ (r & 7)) * 16)) = q;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + s);
      load(t + 1);
      // by now the chunk before is done, since the stage that this step took was its
      if (j % kChunk >= M::kStages && j / kChunk > next) {
        take(next++);
        if (!ok) break;
      }
    }
    cp_async_wait_all();
    while (ok && next < chunks) take(next++);
    if (!ok && lane == 0) failed = 1;
  }
  // two threads a row, each half of the columns; a wait that gave up leaves no numbers
  const int r = threadIdx.x % 128, row = blockIdx.x * 128 + r;
  T* y = static_cast<T*>(a.y) + static_cast<size_t>(n0) * a.m + row;
  __syncthreads();
  if (ranks == 1) {
    if (warp < 8 && row < a.m) {
      const float ws = failed ? __uint_as_float(0x7fc00000u) : __ldg(a.ws + row);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const int col = wg * (N / 2) + i;
        if (col < nn) y[static_cast<size_t>(col) * a.m] = scaled<T>(sum[i], __ldg(a.xs + n0 + col), ws);
      }
    }
  } else {
    int* out = reinterpret_cast<int*>(sm);  // [column][row], where the operands were
    if (warp < 8) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) out[(wg * (N / 2) + i) * 128 + r] = sum[i];
    }
    cluster_sync();
    if (warp < 8) {
      int bad = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < ranks) bad |= ld_cluster_int(smem_u32(&failed), q);
      const float ws = bad ? __uint_as_float(0x7fc00000u) : __ldg(a.ws + min(row, a.m - 1));
      for (int col = wg * ranks + rank; col < nn; col += 2 * ranks) {
        int v[8], total = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < ranks ? ld_cluster_int(smem_u32(out + col * 128 + r), q) : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) total += v[q];
        if (row < a.m) y[static_cast<size_t>(col) * a.m] = scaled<T>(total, __ldg(a.xs + n0 + col), ws);
      }
    }
    cluster_sync();  // no block leaves while its sums are read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tm, M::kCols);
  }
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

template <typename T, int N>
int launch_tc(const Q8Args& a, cudaStream_t st) {
  const int rows = (a.m + 127) / 128, cols = (a.n + N - 1) / N, steps = (a.k + kStep - 1) / kStep;
  const long long groups = static_cast<long long>(rows) * cols;
  const int ranks = std::max(1, std::min({8, static_cast<int>(152 / groups), steps / 4}));
  if (!allow_smem<k_q8_tc<T, N>, Tc<N>::kBytes>()) return S2_ECUDA;
  return launch_clusters(k_q8_tc<T, N>, dim3(rows, ranks, cols), kTcThreads, Tc<N>::kBytes, ranks, a, st);
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
  const Q8Args a{x_codes, x_scales, codes, scales, y, n, m, k, wait_tries.load(std::memory_order_relaxed)};
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (n <= 32) return n <= 8 ? launch_few<T, 1>(a, st) : n <= 16 ? launch_few<T, 2>(a, st) : launch_few<T, 4>(a, st);
    return n <= 64 ? launch_tc<T, 64>(a, st) : launch_tc<T, 128>(a, st);
  });
}
