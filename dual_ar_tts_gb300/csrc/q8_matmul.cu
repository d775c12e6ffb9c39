// Products of 8-bit integers with a scale for each activation row and each weight row:
//   y[n][r] = xs[n] ws[r] sum_k xc[n][k] wc[r][k]
// The sum is the exact integer.  sm_103a's tensor cores have next to no rate for 8-bit integers (mma.sync on s8 and dp4a
// both measured 256 products a clock and SM; fp16 has 1024 on mma.sync and 4096 on tcgen05), so codes are expanded to fp16,
// which holds them exactly; a product has 14 bits, and fp32 holds the sum of 1024 of them exactly (2^24).  Every 1024
// columns (a chunk) the sums go over to 32-bit integers.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "convert.cuh"
#include "ptx.cuh"
#include "q8.cuh"
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

// (.aligned: a warp arrives as one.  What comes before may have been done by some of its lanes alone, and a warp that is still
// apart would count more than once, so that the other block could leave early.)
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster_int(uint32_t addr, uint32_t rank) {
  int v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(addr), "r"(rank));
  return v;
}

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr, uint32_t rank) {
  int4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
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
// It is bound by latency: of 11.7 us for one row of 19456 x 2560 (4.3 TB/s; 8.3 us with the weights in L2), 4 are there at any
// size: the launch, the first copies, the join.  7 rows of 6144 x 2560 6.8 us, 16 of 19456 x 2560 14.4.  (Results stored behind the
// last meeting of the cluster instead of before: 11.7, 6.4 .. 6.9 us, no gain.)
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
  pdl_trigger();
  pdl_wait();
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
        v = __ldcg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(n0 + col) * a.k + k));
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
      static_cast<T*>(a.y)[static_cast<size_t>(n0 + col) * a.m + row] = scaled<T>(v, __ldcg(a.xs + n0 + col), __ldcg(a.ws + row));
  }
  if (ranks > 1) cluster_sync();  // no block leaves while its sums are read
}

// ---- more activation rows: tcgen05, its A operand the weights, B the activations.
//
// A tile is 128 weight rows a block times N activation rows.  Twice four warps take steps of 128 columns in turn: a thread
// expands a weight row to fp16 in tensor memory.  Four warps expand every step's activations into the swizzled tiles that the
// tensor core reads.  One warp issues the products, in two halves of the columns.  The first eight warps also own the sums, a
// thread half a row's: when a chunk's products are done they are added to integers, and the next chunk starts in their place;
// the halves end one after the other, and the operands of the next steps lie ready meanwhile.
// kPair: the blocks of a pair work on one tile of 256 weight rows (cta_group::2), each holds half of the activations, which
// halves what a block reads and stores of them.  Blocks take tiles in turn (there is no end of a pipeline between them), or
// the blocks of a cluster split W's columns of one tile.
// Bound by the hand-overs of a step with few rows (some 800 clocks a step, the slowest of copying, expanding either operand and
// issuing; the weights in L2 or not), and with many by the tensor core beside the expansion (2048 rows of 19456 x 2560 132 us,
// 1.55 PFLOP/s, 0.81 of what the library's bf16 products reach; 32 rows of 2560 x 9728 11.0 us, 512 rows of 19456 x 2560 38).
// Waits know a phase's parity only, so none may be two phases behind: a stage's `empty` comes in the order of its steps, since
// products are done in order, and who fills it has waited for the step before; copies land in any order, see kW.
template <int N, bool kPair>
struct Tc {
  static constexpr int kRows = kPair ? N / 2 : N;                   // of activations in a block
  static constexpr int kStages = kRows == 128 ? 3 : 4;              // expanded steps: 64 tensor memory columns and B each
  // Steps of codes.  A place of the weights' is always the same four warps': copies may land out of order, and a warp that had
  // not waited for a place's former step could take that step's phase, still open, for its own (waits know a phase's parity).
  static constexpr int kW = kRows == 128 ? 4 : 6, kX = kRows == 128 ? 3 : 4;
  static_assert(kW % 2 == 0, "a place's steps are of one parity");
  static constexpr int kBBytes = kRows * 256, kWBytes = 128 * kStep, kXBytes = kRows * kStep;
  static constexpr int kWRing = kStages * kBBytes, kXRing = kWRing + kW * kWBytes;
  // Parts of the columns, each with its products and its sums.  A pair's are two (all at once: 138 us for 2048 rows of
  // 19456 x 2560, 134 so); a block's one (in two: 11.4 us for 32 rows of 2560 x 9728, 10.9 so).
  static constexpr int kParts = kPair ? 2 : 1, kPart = N / kParts;
  static constexpr int kOut = kXRing + kX * kXBytes, kOutWarp = 2048;  // results on their way, of a warp
  static constexpr int kBars = kOut + 8 * kOutWarp, kBytes = kBars + 512 + 1024;
  static constexpr uint32_t kCols = 512, kA = 256;                  // tensor memory: sums, then A
  static_assert(N <= 256 && kA + 64 * kStages <= kCols && N * 128 * 4 <= kBars && kBytes <= 232000, "room");
};

struct Maps {
  CUtensorMap w, x;  // codes as [rows][k]: boxes of 128 columns, swizzled
  CUtensorMap y;     // results, where `bulk`: boxes of 32 weight rows
  bool bulk;
};

// Box at (column, row) of a tensor map into shared memory.
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                   smem_u32(dst)),
               "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
               : "memory");
}

// Arrival at the same barrier of the pair's first block.  What it tells of lies in the arriving block's own shared and tensor
// memory, and is complete: fence.proxy.async and tcgen05.wait::st come first.  So the release is the block's; one at cluster
// scope cost 1200 clocks each, and 2048 rows of 19456 x 2560 193 us.
__device__ __forceinline__ void mbar_arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// Whether a phase is done, without waiting.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// 32 columns of tensor memory; their values are there after tmem_loaded().
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));  // not used before
}
// A step's products with one part of the columns: eight of 16 columns of K.  b: the low word of the part's descriptor, whose
// address is the only thing that moves (bits 0 - 13, in 16 bytes); kFar: from K's first 64 columns to the second.
template <bool kPair, int kFar>
__device__ __forceinline__ void mma_part(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc, bool add) {
#define S2_MMA(group)                                                                                         \
  asm volatile(                                                                                               \
      "{\n\t.reg .pred p, q;\n\t.reg .b64 d0, d1, d2, d3, d4, d5, d6, d7;\n\t"                                \
      "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, %4, %4;\n\t"                                                  \
      "mov.b64 d0, {%5, %3};\n\tmov.b64 d1, {%6, %3};\n\tmov.b64 d2, {%7, %3};\n\tmov.b64 d3, {%8, %3};\n\t" \
      "mov.b64 d4, {%9, %3};\n\tmov.b64 d5, {%10, %3};\n\tmov.b64 d6, {%11, %3};\n\tmov.b64 d7, {%12, %3};\n\t" \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%1], d0, %2, p;\n\t"                                 \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%13], d1, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%14], d2, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%15], d3, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%16], d4, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%17], d5, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%18], d6, %2, q;\n\t"                                \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], [%19], d7, %2, q;\n\t}"                               \
      ::"r"(d), "r"(a), "r"(idesc), "r"(b_high), "r"(static_cast<uint32_t>(add)), "r"(b), "r"(b + 2), "r"(b + 4), "r"(b + 6), \
      "r"(b + kFar), "r"(b + kFar + 2), "r"(b + kFar + 4), "r"(b + kFar + 6), "r"(a + 8), "r"(a + 16), "r"(a + 24),           \
      "r"(a + 32), "r"(a + 40), "r"(a + 48), "r"(a + 56)                                                      \
      : "memory")
  if constexpr (kPair)
    S2_MMA("2");
  else
    S2_MMA("1");
#undef S2_MMA
}
// An arrival at `bar` (in both blocks of a pair) when the products issued so far are done.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (!kPair)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// The same at this block's alone.
template <bool kPair>
__device__ __forceinline__ void commit_here(uint64_t* bar) {
  if constexpr (!kPair)
    tc_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tmem_get(uint32_t* dst, uint32_t cols) {
  if constexpr (!kPair) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
  if constexpr (!kPair)
    tmem_dealloc(at, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}
template <int kRegs>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// sum += v, a whole number of up to 2^24.  The machine's conversion passes one lane in eight a clock; by arithmetic it takes
// six instructions.  Where the next part's products wait, half of them go each way.
__device__ __forceinline__ void add_whole(int& sum, float v, bool arithmetic) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, it rounds to a whole number, which the sum's low bits then hold
  constexpr uint32_t kBits = 0x4b400000;
  if (arithmetic) {
    const float t = __fmaf_rn(v, 0x1p-12f, kMagic), low = __fmaf_rn(t - kMagic, -4096.f, v) + kMagic;  // v = 4096 t + low
    sum = static_cast<int>(static_cast<uint32_t>(sum) + __float_as_uint(t) * 4096u + __float_as_uint(low) - (kBits * 4096u + kBits));
  } else {
    sum += __float2int_rn(v);
  }
}

// Threads: eight warps for weights, four for activations, four of which one issues.  A pair's sums take 128 registers a thread:
// of the launch's 512 x 128 registers the first eight warps' threads take 208, the next four's 72, the last four's 24.
constexpr int kTcThreads = 512;
template <typename T, int N, bool kPair>
__global__ void __launch_bounds__(kTcThreads, 1) k_q8_tc(const Q8Args a, const __grid_constant__ Maps maps) {
  using M = Tc<N, kPair>;
  constexpr int S = M::kStages, kHalf = N / 2, P = M::kParts, kPart = M::kPart;  // columns of four warps, of a part
  extern __shared__ __align__(16) uint8_t smraw[];
  __shared__ int failed;
  uint8_t* sm = smraw + (-smem_u32(smraw) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + M::kBars);  // [step % S]: expanded
  uint64_t* empty = full + S;                                   // and used up
  uint64_t *done = empty + S, *taken = done + P;                // [part]: a chunk's products; its sums read
  uint64_t* drained = taken + P;                                // nothing under way
  uint64_t *w_here = drained + 1, *w_free = w_here + M::kW;     // [step % kW]: codes of weights
  uint64_t *x_here = w_free + M::kW, *x_free = x_here + M::kX;  // [step % kX]: codes of activations
  uint32_t* tbase = reinterpret_cast<uint32_t*>(x_free + M::kX);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int steps = (a.k + kStep - 1) / kStep;
  const int ranks = kPair ? 1 : gridDim.y, rank = kPair ? 0 : blockIdx.y, side = kPair ? blockIdx.x % 2 : 0;
  const int s0 = static_cast<int>(static_cast<long long>(steps) * rank / ranks);
  const int count = static_cast<int>(static_cast<long long>(steps) * (rank + 1) / ranks) - s0;
  const int chunks = (count + kChunk - 1) / kChunk;  // of a tile
  // tiles: weight rows first, so that blocks at work together share activations
  constexpr int kTile = kPair ? 256 : 128;
  const int row_tiles = (a.m + kTile - 1) / kTile, tiles = row_tiles * ((a.n + N - 1) / N);
  const int first = kPair ? blockIdx.x / 2 : blockIdx.x, apart = kPair ? gridDim.x / 2 : gridDim.x;
  const int mine = first < tiles ? (tiles - first + apart - 1) / apart : 0;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, kPair ? 16 : 8);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < P; ++i) {
      mbar_init(done + i, 1);
      mbar_init(taken + i, (kPair ? 8 : 4) * 2 / P);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < M::kW; ++i) {
      mbar_init(w_here + i, 1);
      mbar_init(w_free + i, 4);
    }
    for (int i = 0; i < M::kX; ++i) {
      mbar_init(x_here + i, 1);
      mbar_init(x_free + i, 4);
    }
    fence_barrier_init();
  }
  if (warp == 13 && lane == 0) {
    prefetch_tmap(&maps.w);
    prefetch_tmap(&maps.x);
  }
  // All of an SM's tensor memory is taken when the kernel in front has ended, and the next is let on when it is: two kernels that
  // wait for each other's memory and end would never do either.
  pdl_wait();
  if (warp == 12) tmem_get<kPair>(tbase, M::kCols);
  tc_fence_before();
  if constexpr (kPair)
    cluster_sync();  // the barriers that the other block arrives at
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tbase, 0);
  pdl_trigger();
  auto arrive = [&](uint64_t* bar) {
    if constexpr (kPair)
      mbar_arrive_first(bar);
    else
      mbar_arrive(bar);
  };

  bool ok = true;
  if (warp >= 12) {
    // ---------------------------------------------------------------- issuing the products
    if constexpr (N >= 128) fewer_registers<24>();
    if (warp == 12 && side == 0) {
      if (elect_one()) {
        int chunk = 0, j = 0, s = 0;  // chunks so far; the step's place in its tile, its stage
        bool here = false;            // whether the step is known to be expanded
        for (int g = 0, all = mine * count; g < all; ++g) {
          const bool starts = j % kChunk == 0, ends = j % kChunk == kChunk - 1 || j == count - 1;
          ok = here || mbar_wait_short(full + s, g / S & 1, a.tries);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = tm + M::kA + s * 64;
          const uint64_t b = desc_sw128(smem_u32(sm + s * M::kBBytes));
          const int next = s + 1 == S ? 0 : s + 1;
#pragma unroll
          for (int p = 0; p < P; ++p) {
            if (starts && chunk > 0) {
              ok = mbar_wait_short(taken + p, (chunk - 1) & 1, a.tries);
              if (!ok) break;
              tc_fence_after();
            }
            // the next step is looked for while products are left to do
            if (p == P - 1) here = g + 1 < all && mbar_done(full + next, (g + 1) / S & 1);
            mma_part<kPair, M::kRows * 8>(tm + p * kPart, ta, static_cast<uint32_t>(b) + p * (M::kRows / P) * 8,
                                          static_cast<uint32_t>(b >> 32), idesc_f16(kTile, kPart), !starts);
            if (p == P - 1) commit<kPair>(empty + s);
            if (ends) commit<kPair>(done + p);
          }
          if (!ok) break;
          if (ends) ++chunk;
          if (++j == count) j = 0;
          s = next;
        }
        commit_here<kPair>(drained);  // no end before that of the products, whoever gave up
        mbar_wait_short(drained, 0);
      }
      __syncwarp();
    } else if (warp == 13 || warp == 14) {
      // -------------------------------------------------------------- copying codes
      if (elect_one()) {
        const bool w = warp == 13;
        const int ring = w ? M::kW : M::kX;
        uint64_t *here = w ? w_here : x_here, *freed = w ? w_free : x_free;
        uint8_t* to = sm + (w ? M::kWRing : M::kXRing);
        int g = 0;
        for (int i = 0; i < mine && ok; ++i) {
          const int t = first + i * apart, row = t % row_tiles * kTile + side * 128, n0 = t / row_tiles * N;
          for (int j = 0; j < count; ++j, ++g) {
            const int s = g % ring, col = (s0 + j) * kStep;
            if (g >= ring) ok = mbar_wait_short(freed + s, (g / ring - 1) & 1, a.tries);
            if (!ok) break;
            mbar_arrive_expect_tx(here + s, w ? M::kWBytes : M::kXBytes);
            if (w) {
              tma_box(to + s * M::kWBytes, &maps.w, col, row, here + s);
            } else if constexpr (kPair) {
#pragma unroll
              for (int p = 0; p < P; ++p)
                tma_box(to + s * M::kXBytes + p * (M::kXBytes / P), &maps.x, col, n0 + p * kPart + side * (kPart / 2), here + s);
            } else {
              tma_box(to + s * M::kXBytes, &maps.x, col, n0, here + s);
            }
          }
        }
        for (int q = max(g - ring, 0); q < g; ++q) mbar_wait_short(here + q % ring, q / ring & 1);  // no end before that of the copies
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- expanding activations
    if constexpr (N >= 128) fewer_registers<72>();
    // Eight lanes take the low half of a row's 128 codes and the high half of its neighbour's, then the other two: neither
    // reading the swizzled codes nor writing the swizzled tiles, in which the halves are apart, meets a bank twice.
    constexpr int kLoads = M::kRows / 16;
    const int tid = threadIdx.x % 128, all = mine * count, high = tid / 4 % 2, c = tid % 4;
    for (int g = 0; g < all; ++g) {
      const int s = g % S, slot = g % M::kX;
      ok = mbar_wait_short(x_here + slot, g / M::kX & 1, a.tries);
      if (g >= S) ok = ok && mbar_wait_short(empty + s, (g / S - 1) & 1, a.tries);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t from = smem_u32(sm + M::kXRing + slot * M::kXBytes);
      uint8_t* b = sm + s * M::kBBytes + high * (M::kRows * 128);
      uint4 held[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i / 2 * 32 + tid / 8 * 2 + (high ^ (i & 1));
        held[i] = lds128(from + r * kStep + (((high * 4 + c) ^ (r & 7)) * 16));
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i / 2 * 32 + tid / 8 * 2 + (high ^ (i & 1));
        const uint4 v = held[i];
        uint4 p, q;
        expand(v.x, p.x, p.y);
        expand(v.y, p.z, p.w);
        expand(v.z, q.x, q.y);
        expand(v.w, q.z, q.w);
        uint8_t* dst = b + r * 128;
        *reinterpret_cast<uint4*>(dst + (((2 * c) ^ (r & 7)) * 16)) = p;
        *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ (r & 7)) * 16)) = q;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        arrive(full + s);
        mbar_arrive(x_free + slot);
      }
    }
    // the last arrivals of the pair's first block, which the second may not leave before
    for (int g = max(all - S, 0); kPair && ok && g < all; ++g)
      ok = __all_sync(0xffffffffu, mbar_wait_short(empty + g % S, g / S & 1, a.tries));
  } else {
    // ---------------------------------------------------------------- expanding weights, adding up
    if constexpr (N >= 128) more_registers<208>();
    const int wg = warp / 4, in = warp % 4 * 32;
    const int all = mine * count;
    const uint32_t lanes = static_cast<uint32_t>(in) << 16, tlane = tm + M::kA + lanes;
    int sum[kHalf];  // of this thread's row, half of the columns
#pragma unroll
    for (int i = 0; i < kHalf; ++i) sum[i] = 0;
    int chunk = 0, tile = 0, in_tile = 0, last = min(kChunk, count) - 1;  // the chunk to take: its tile, place there, last step
    const int part = wg * P / 2;
    auto take = [&] {
      ok = __all_sync(0xffffffffu, mbar_wait_short(done + part, chunk & 1, a.tries));
      if (!ok) return;
      tc_fence_after();
      constexpr int kPass = std::min(kHalf, 64);
#pragma unroll
      for (int c = 0; c < kHalf; c += kPass) {
        uint32_t v[kPass / 32][32];
#pragma unroll
        for (int i = 0; i < kPass / 32; ++i) tmem_load32(tm + lanes + wg * kHalf + c + i * 32, v[i]);
#pragma unroll
        for (int i = 0; i < kPass / 32; ++i) tmem_loaded(v[i]);
        if (c + kPass == kHalf) {  // the next chunk's products may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(taken + part);
        }
#pragma unroll
        for (int i = 0; i < kPass; ++i) add_whole(sum[c + i], __uint_as_float(v[i / 32][i % 32]), c + kPass < kHalf && i % 2);
      }
      ++chunk;
    };
    // A tile's results, two threads a row; a quarter of a thread's columns after each of the next tile's first steps, by TMA, so
    // that the tensor core does not wait for them (all at once and by plain stores: 5000 to 7000 clocks).
    int left = 0, written = 0;  // quarters to write, and their tile
    float ws = 0.f, xs[4] = {};  // its scales: the thread's row's, and every 32nd (kQ-th) of the columns'
    constexpr int kQ = kHalf / 4, kC = std::min(kQ, static_cast<int>(M::kOutWarp / 32 / sizeof(T)));  // columns of a quarter, of a box
    T* const out = reinterpret_cast<T*>(sm + M::kOut + warp * M::kOutWarp);
    auto row_of = [&](int t) { return t % row_tiles * kTile + side * 128 + in; };
    auto column_of = [&](int t) { return t / row_tiles * N + wg * kHalf; };
    auto load_scales = [&] {
      const int t = first + tile * apart;
      ws = __ldcg(a.ws + min(row_of(t) + lane, a.m - 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) xs[i] = __ldcg(a.xs + min(column_of(t) + i * kQ + lane % kQ, a.n - 1));
    };
    auto write = [&](auto quarter) {
      constexpr int q = decltype(quarter)::value;
      const int t = first + written * apart, row = row_of(t), n0 = column_of(t) + q * kQ;
      if (maps.bulk) {
#pragma unroll
        for (int c = 0; c < kQ; c += kC) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the box before is read
          __syncwarp();
#pragma unroll
          for (int i = c; i < c + kC; ++i) {
            out[(i - c) * 32 + lane] = scaled<T>(sum[q * kQ + i], __shfl_sync(0xffffffffu, xs[q], i), ws);
            sum[q * kQ + i] = 0;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row < a.m && n0 + c < a.n)
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
                "cp.async.bulk.commit_group;" ::"l"(&maps.y),
                "r"(row), "r"(n0 + c), "r"(smem_u32(out))
                : "memory");
          __syncwarp();
        }
      } else {
        T* y = static_cast<T*>(a.y) + static_cast<size_t>(n0) * a.m + row + lane;
        const int live = row + lane < a.m ? a.n - n0 : 0;
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const T v = scaled<T>(sum[q * kQ + i], __shfl_sync(0xffffffffu, xs[q], i), ws);
          if (i < live) *y = v;
          y += a.m;
          sum[q * kQ + i] = 0;
        }
      }
    };
    auto write_some = [&] {
      if (left == 4) write(std::integral_constant<int, 0>{});
      if (left == 3) write(std::integral_constant<int, 1>{});
      if (left == 2) write(std::integral_constant<int, 2>{});
      if (left == 1) write(std::integral_constant<int, 3>{});
      --left;
    };
    for (int g = wg; ok && (tile < mine || left > 0); g += 2) {
      const int s = g % S, slot = g % M::kW;
      // A chunk is taken when it is done.  One whose last step has to leave its stage before this one can come is waited for, and
      // behind the last step those that are left.
      bool due;
      do {
        due = tile < mine &&
              (last <= g - S || g >= all || (last < g && __all_sync(0xffffffffu, mbar_done(done + part, chunk & 1))));
        if (left > 0) {
          write_some();
        } else if (due) {
          if (in_tile == chunks - 1) load_scales();
          take();
          if (ok && ++in_tile == chunks) {
            if (ranks == 1) left = 4, written = tile;
            in_tile = 0, ++tile;
          }
          last = tile * count + min((in_tile + 1) * kChunk, count) - 1;
        }
      } while (ok && due);
      if (!ok || g >= all) continue;
      ok = mbar_wait_short(w_here + slot, g / M::kW & 1, a.tries);
      if (g >= S) ok = ok && mbar_wait_short(empty + s, (g / S - 1) & 1, a.tries);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = smem_u32(sm + M::kWRing + slot * M::kWBytes) + (in + lane) * kStep;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 x = lds128(at + (((half * 4 + c) ^ (lane & 7)) * 16));
          expand(x.x, r[c * 8], r[c * 8 + 1]);
          expand(x.y, r[c * 8 + 2], r[c * 8 + 3]);
          expand(x.z, r[c * 8 + 4], r[c * 8 + 5]);
          expand(x.w, r[c * 8 + 6], r[c * 8 + 7]);
        }
        tmem_st32(tlane + s * 64 + half * 32, r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        arrive(full + s);
        mbar_arrive(w_free + slot);
      }
    }
    if (!ok) {
      if (lane == 0) failed = 1;
      // a wait that gave up leaves no numbers
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // none of its results come later
      __syncwarp();
      if (left > 0) tile = written;
      for (; ranks == 1 && tile < mine; ++tile) {
        const int t = first + tile * apart, n0 = column_of(t), row = row_of(t) + lane;
#pragma unroll 1
        for (int i = n0; row < a.m && i < min(n0 + kHalf, a.n); ++i)
          static_cast<T*>(a.y)[static_cast<size_t>(i) * a.m + row] = from_f<T>(__uint_as_float(0x7fc00000u));
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    if (ranks > 1) {
      named_bar(1, 256);  // every operand is used up
      int* out = reinterpret_cast<int*>(sm);  // [column][row], where the operands were
#pragma unroll
      for (int i = 0; i < kHalf; ++i) out[(wg * kHalf + i) * 128 + in + lane] = sum[i];
    }
  }
  if constexpr (!kPair) {
    if (ranks > 1) {
      cluster_sync();
      if (warp < 8) {  // the others have few registers left; four rows of a column a thread
        const int r = lane * 4, row = first % row_tiles * 128 + r, n0 = first / row_tiles * N, nn = min(N, a.n - n0);
        const int* out = reinterpret_cast<const int*>(sm);
        int bad = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < ranks) bad |= ld_cluster_int(smem_u32(&failed), q);
        float ws[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) ws[e] = bad ? __uint_as_float(0x7fc00000u) : __ldcg(a.ws + min(row + e, a.m - 1));
#pragma unroll 2
        for (int col = warp * ranks + rank; col < nn; col += 8 * ranks) {
          int4 v[8];
          int total[4] = {};
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = q < ranks ? ld_cluster_int4(smem_u32(out + col * 128 + r), q) : make_int4(0, 0, 0, 0);
          const float xs = __ldcg(a.xs + n0 + col);
#pragma unroll
          for (int q = 0; q < 8; ++q) total[0] += v[q].x, total[1] += v[q].y, total[2] += v[q].z, total[3] += v[q].w;
          T* y = static_cast<T*>(a.y) + static_cast<size_t>(n0 + col) * a.m + row;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (row + e < a.m) y[e] = scaled<T>(total[e], xs, ws[e]);
        }
      }
      cluster_sync();  // no block leaves while its sums are read
    }
  }
  tc_fence_before();
  if constexpr (kPair)
    cluster_sync();  // no block leaves while its operands are read, or its barriers arrived at
  else
    __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_free<kPair>(tm, M::kCols);
  }
}

// Blocks that split W's columns for each of `groups` tiles: the most, up to eight and `most`, whose clusters the device
// holds at a time.  (It takes whole clusters in whole groups of its SMs, so many sizes leave SMs over: 20 clusters of seven
// blocks of k_q8_tc took two rounds, 22 us for 64 rows of 2560 x 9728 against 15 with six, which are 11.5 now.)  What it holds is asked once.
template <auto kKernel>
int split(long long groups, int most, int threads, int smem) {
  static std::atomic<int> held[64][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  for (int ranks = std::min(8, most); ranks > 1; --ranks) {
    int n = dev < 64 ? held[dev][ranks].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(1, ranks);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 1;
      at[0].val.clusterDim.y = ranks;
      at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();  // not a failure of the call's
        n = -1;
      }
      if (dev < 64) held[dev][ranks].store(n, std::memory_order_relaxed);
    }
    if (groups <= n) return ranks;
  }
  return 1;
}

template <typename T, int NT>
int launch_few(const Q8Args& a, cudaStream_t st) {
  const int rows = (a.m + kFewRows - 1) / kFewRows, cols = (a.n + NT * 8 - 1) / (NT * 8), steps = (a.k + kStep - 1) / kStep;
  if (!allow_smem<k_q8_few<T, NT>, kFewBytes<NT>>()) return S2_ECUDA;
  const int ranks = split<k_q8_few<T, NT>>(static_cast<long long>(rows) * cols, steps / 2, 32 * kFewWarps, kFewBytes<NT>);
  return launch_ahead(k_q8_few<T, NT>, dim3(rows, ranks, cols), dim3(1, ranks), 32 * kFewWarps, kFewBytes<NT>, st, a);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p)
               : nullptr;
  }();
  return encode;
}
// Boxes of `box` rows by 128 columns of codes [rows][k], swizzled in 128 bytes; zeros outside.
bool code_map(CUtensorMap* map, const int8_t* codes, long long rows, int k, int box) {
  const auto encode = encoder();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)}, stride[1] = {static_cast<cuuint64_t>(k)};
  const cuuint32_t boxes[2] = {kStep, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(codes), dims, stride, boxes, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Boxes of 32 weight rows by `box` activation rows of results [n][m], where their rows start on 16 bytes.
template <typename T>
bool result_map(CUtensorMap* map, void* y, int n, int m, int box) {
  const long long stride = static_cast<long long>(m) * sizeof(T);
  const auto encode = encoder();
  if (reinterpret_cast<uintptr_t>(y) % 16 != 0 || stride % 16 != 0 || !encode) return false;
  const CUtensorMapDataType type = std::is_same<T, float>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(m), static_cast<cuuint64_t>(n)}, strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t boxes[2] = {32, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return encode(map, type, 2, y, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch of k_q8_tc: what it splits, and what it takes, in ns.
struct Plan {
  int blocks, ranks;
  double time;
};
// A block has 5.5 to 7.5 us of launch, filling and draining, and a time a step; blocks at work together are a round (152 SMs, 76 pairs).
// A join costs by its columns.  Measured, us, at (rows) for one column tile of 64 and 128 and a pair's 256, weights not in L2:
// 19456 x 2560 (64) 14.8, 17.4, 21.7; (128) 25.3, 17.9, 21.8; (256) 45.7, 30.5, 22.5; (1024) -, 108, 69; 6144 x 2560 (64) 10.9,
// 14.4, 20.0; (128) 13.6, 17.8, 20.0; (256) 23.8, 16.8, 20.3; (512) -, 29.6, 21.2; 2560 x 9728 (64) 11.6, 15.0, 54.6; (128) 16.9, 16.4,
// 54.7; (512) -, 45.9, 55.0; (2048) -, 129, 107.  The constants were fitted before launches came to begin ahead of the kernel
// in front: times are off by up to 5 us, or a seventh, but the fastest is the shortest at each of these.
template <typename T, int N, bool kPair>
Plan plan_tc(const Q8Args& a) {
  using M = Tc<N, kPair>;
  constexpr int kTile = kPair ? 256 : 128, kAtOnce = kPair ? 76 : 152;
  constexpr double kFixed = kPair ? 7500 : N == 128 ? 6000 : 5500, kPerStep = kPair ? 720 : N == 128 ? 600 : 500;
  constexpr double kPerColumn = N == 128 ? 45 : 20;
  const int steps = (a.k + kStep - 1) / kStep;
  const long long tiles = static_cast<long long>((a.m + kTile - 1) / kTile) * ((a.n + N - 1) / N);
  Plan p{};
  p.ranks = kPair ? 1 : split<k_q8_tc<T, N, kPair>>(tiles, steps / 4, kTcThreads, M::kBytes);
  p.blocks = static_cast<int>(p.ranks > 1 ? tiles : std::min<long long>(tiles, kAtOnce));
  const long long rounds = p.ranks > 1 ? 1 : (tiles + kAtOnce - 1) / kAtOnce;
  p.time = kFixed + rounds * kPerStep * ((steps + p.ranks - 1) / p.ranks) + (p.ranks > 1 ? 1500 + kPerColumn * std::min(N, a.n) : 0);
  return p;
}

template <typename T, int N, bool kPair>
int launch_tc(const Q8Args& a, const Plan& plan, cudaStream_t st) {
  using M = Tc<N, kPair>;
  Maps maps;
  if (!code_map(&maps.w, a.w, a.m, a.k, 128) || !code_map(&maps.x, a.x, a.n, a.k, kPair ? M::kPart / 2 : N)) return S2_ECUDA;
  maps.bulk = result_map<T>(&maps.y, a.y, a.n, a.m, std::min(N / 8, static_cast<int>(M::kOutWarp / 32 / sizeof(T))));
  return launch_ahead(k_q8_tc<T, N, kPair>, dim3(plan.blocks * (kPair ? 2 : 1), plan.ranks),
                         kPair ? dim3(2) : dim3(1, plan.ranks), kTcThreads, M::kBytes, st, a, maps);
}

template <typename T>
int launch_matmul(const Q8Args& a, cudaStream_t st) {
  // mma.sync up to 16 rows, and up to 64 of a matrix of less than 4 Mi weights (1024 x 1024 5.7 us against 6.1 at 32 rows,
  // 5.8 against 6.7 at 64; 2560 x 4096 9.8 against 7.9 at 32).
  if (a.n <= 16) return a.n <= 8 ? launch_few<T, 1>(a, st) : launch_few<T, 2>(a, st);
  if (a.n <= 64 && static_cast<long long>(a.m) * a.k < 4ll << 20) return launch_few<T, 4>(a, st);
  if (!allow_smem<k_q8_tc<T, 64, false>, Tc<64, false>::kBytes>() || !allow_smem<k_q8_tc<T, 128, false>, Tc<128, false>::kBytes>() ||
      !allow_smem<k_q8_tc<T, 256, true>, Tc<256, true>::kBytes>())
    return S2_ECUDA;
  const Plan one = plan_tc<T, 64, false>(a), two = plan_tc<T, 128, false>(a), pair = plan_tc<T, 256, true>(a);
  if (one.time <= two.time && one.time <= pair.time) return launch_tc<T, 64, false>(a, one, st);
  return two.time <= pair.time ? launch_tc<T, 128, false>(a, two, st) : launch_tc<T, 256, true>(a, pair, st);
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
    return launch_matmul<T>(a, reinterpret_cast<cudaStream_t>(stream));
  });
}
