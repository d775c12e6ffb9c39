// 4-bit weights with group scales: the quantiser and the products with activation rows.
//   w[r][k] = scale[r][k / G] * (code[r][k] - 8),   y[n][r] = sum_k x[n][k] * w[r][k]
// Codes are stored in blocks of 128 columns (64 bytes): 32-bit word 4c + j of a block holds the codes
// of columns 32j + 8c .. 32j + 8c + 7 (lowest nibble first), so the 16 bytes at offset 16c are the
// c-th eight columns of each of the block's four 32-column parts.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"
#include "tc05.cuh"

namespace s2 {
namespace {

constexpr int kBlock = 128;  // columns of a code block

// One warp per block of 128 columns; lane l holds columns 4l .. 4l + 3 (19456 x 2560: 118 us, bound by its divisions;
// weights are quantised once).  A group's scale is its entry
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
// y = x W^T.  Up to 16 or 32 columns (activation rows; an fp32 row is two) on mma.sync.m16n8k16 (fp16 operands, fp32 sums):
// 16 weight rows are the A operand, expanded from their codes in registers, 8 columns the B operand.  tcgen05 wants
// the expanded weights in tensor memory first; with more columns that pays (k_q4_tc, below).
//
// A code is expanded to the whole number code - 8.  (Masked alone it would be the fp16 subnormal code * 2^-24, and the
// sum would have to start with -8 * sum x.  That is four instructions a word less, 10.5 us against 11.3 for one row
// of 19456 x 2560, but the tensor cores line products up by their operands' exponents and cut off what is below a
// sum's last bit, and the rest cancels: fp32 products were 1e-6 to 2e-6 off, where they now are 1e-7.)  A 32-bit word of codes feeds the k positions of two instructions in the
// order (0,4)(1,5) | (2,6)(3,7) of its nibbles; activations are staged in that order.  A group's scale multiplies its
// fp32 sum.
//
// Activations are scaled by a power of two so that the largest of a row (of a staged chunk of it) lies in
// 2^13 .. 2^14.  fp16 and bf16 values are then exact in fp16, but for elements 2^-27 below the largest and less,
// which keep 2^-38 of it; an fp32 value is two fp16 terms (22 bits), each a column of its own, added at the end.
//
// A warp copies its codes ahead of their use (cp.async, its own ring).  Few activations are staged by each
// block itself (k_q4_few); more of them once, by a kernel in front (k_q4_planes, then k_q4_many or k_q4_tc).

constexpr int kWarps = 8;

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;

// eight consecutive activations as loaded
template <typename T>
struct Eight {
  uint4 raw[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float operator[](int i) const {
    const uint32_t w = (&raw[0].x)[sizeof(T) == 4 ? i : i / 2];
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<uint16_t>(i % 2 ? w >> 16 : w)));
    else return i % 2 ? bf16hi(w) : bf16lo(w);
  }
};

// The power of two that takes a largest magnitude (its bits) to 2^13 .. 2^14, by its exponent; what is not
// finite, and zero, stays as it is.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  const int e = static_cast<int>(top >> 23);
  return top == 0 || e == 255 ? 0 : min(13 + 127 - e, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int kSize>
__device__ __forceinline__ void cp_async_small(void* smem, const void* gmem, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(smem)), "l"(gmem), "n"(kSize), "r"(bytes)
               : "memory");
}

struct MatmulArgs {
  const void* x;
  long long x_stride;
  int n, m, k;
  const uint8_t* codes;
  const __nv_bfloat16* scales;
  void* y;
  int tiles;  // R
  int tries;  // of a wait
};

// One 8-element item of an activation row, scaled by `up`: the B operand's 16 bytes of each term, as the pairs
// (0,4) (1,5) (2,6) (3,7).
template <typename T>
struct Staged {
  uint4 b[kTerms<T>];
  __device__ __forceinline__ Staged(const Eight<T>& v, float up) {
    float rest[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rest[e] = v[e] * up;
#pragma unroll
    for (int t = 0; t < kTerms<T>; ++t) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 two = __floats2half2_rn(rest[e], rest[e + 4]);
        const float2 r = __half22float2(two);
        h[e] = *reinterpret_cast<const uint32_t*>(&two);
        rest[e] -= r.x;
        rest[e + 4] -= r.y;
      }
      b[t] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
};

// The eight codes of a word as fp16 code - 8, in the order 0 4 1 5 2 6 3 7.  0x6400 | code is 1024 + code in fp16 and
// 0x6400 | code << 4 is 1024 + 16 code: code - 8 comes out of one exact subtraction or FMA.
__device__ __forceinline__ void expand(uint32_t w, __half2 (&v)[4]) {
  const uint32_t m = 0x64006400u, w8 = w >> 8;
  const __half2 z = __float2half2_rn(1032.f), z16 = __float2half2_rn(-72.f), sixteenth = __float2half2_rn(0.0625f);
  auto h2 = [](uint32_t u) { return *reinterpret_cast<__half2*>(&u); };
  v[0] = __hsub2(h2((w & 0x000f000fu) | m), z);
  v[1] = __hfma2(h2((w & 0x00f000f0u) | m), sixteenth, z16);
  v[2] = __hsub2(h2((w8 & 0x000f000fu) | m), z);
  v[3] = __hfma2(h2((w8 & 0x00f000f0u) | m), sixteenth, z16);
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

template <typename T>
__device__ __forceinline__ uint32_t largest(const Eight<T>& v) {  // bits of the magnitude; NaN counts as the largest
  uint32_t t = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) t = max(t, __float_as_uint(v[e]) & 0x7fffffffu);
  return t;
}

constexpr int kRing = 1024 + 128;  // a code block of 16 rows and its scales

// A warp's codes: entry j of its sequence is block first + j * step of its 16 rows, kAhead in flight.
template <int G, int kAhead>
struct Codes {
  static constexpr int SB = kBlock / G;  // scales of a block
  uint8_t* ring;
  const uint8_t *wa, *wb;
  const __nv_bfloat16* scales;
  size_t sat, send;
  uint32_t par0, par1;  // parities of the rows' first scales (G = 128)
  int issued = 0, count, step;

  __device__ __forceinline__ Codes(uint8_t* r, const MatmulArgs& a, int row0, int blocks, int first, int n, int st)
      : ring(r), scales(a.scales), count(n), step(st) {
    const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const int ra = min(row0 + g, a.m - 1), rb = min(row0 + g + 8, a.m - 1);
    wa = a.codes + (static_cast<size_t>(ra) * blocks + first) * 64 + c * 16;
    wb = a.codes + (static_cast<size_t>(rb) * blocks + first) * 64 + c * 16;
    sat = (static_cast<size_t>(c ? rb : ra) * blocks + first) * SB;  // lanes c = 0, 1 copy the scales
    send = static_cast<size_t>(a.m) * blocks;
    par0 = static_cast<uint32_t>(ra) * blocks + first;
    par1 = static_cast<uint32_t>(rb) * blocks + first;
  }
  __device__ __forceinline__ void issue() {  // does not commit
    if (issued < count) {
      const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
      uint8_t* dst = ring + issued % kAhead * kRing;
      cp_async16(dst + lane * 16, wa);
      cp_async16(dst + 512 + lane * 16, wb);
      wa += step * 64;
      wb += step * 64;
      if (c < 2) {
        uint8_t* to = dst + 1024 + (g + 8 * c) * 8;
        if constexpr (G == 128)  // two bytes wanted: the aligned four around them, less what lies past the last scale
          cp_async_small<4>(to, scales + (sat & ~size_t{1}), (sat | 1) < send ? 4 : 2);
        else
          cp_async_small<2 * SB>(to, scales + sat, 2 * SB);
        sat += step * SB;
      }
    }
    ++issued;
  }
};

// One code block (entry j of a ring) times the staged activations: z += W x.  xq: this lane's B operands, part p of
// tile t at xq[p * part_stride + t * 32].
template <int NT, int G>
__device__ __forceinline__ void multiply(uint32_t at, uint32_t par0, uint32_t par1, const uint4* xq, int part_stride,
                                         float (&z)[NT][4]) {
  const int lane = threadIdx.x % 32, g = lane / 4;
  const uint4 w0 = lds128(at + lane * 16), w1 = lds128(at + 512 + lane * 16);
  float s0[4], s1[4];
  const uint32_t sa = at + 1024 + g * 8;
  const uint32_t u = lds32(sa), v = lds32(sa + 64);
  if constexpr (G == 32) {
    const uint32_t u1 = lds32(sa + 4), v1 = lds32(sa + 68);
    s0[0] = bf16lo(u), s0[1] = bf16hi(u), s0[2] = bf16lo(u1), s0[3] = bf16hi(u1);
    s1[0] = bf16lo(v), s1[1] = bf16hi(v), s1[2] = bf16lo(v1), s1[3] = bf16hi(v1);
  } else if constexpr (G == 64) {
    s0[1] = bf16lo(u), s0[3] = bf16hi(u);
    s1[1] = bf16lo(v), s1[3] = bf16hi(v);
  } else {
    s0[3] = par0 & 1 ? bf16hi(u) : bf16lo(u);
    s1[3] = par1 & 1 ? bf16hi(v) : bf16lo(v);
  }
  const uint32_t wv[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
  float d[NT][4];
#pragma unroll
  for (int part = 0; part < 4; ++part) {
    __half2 p[4], q[4];
    expand(wv[0][part], p);
    expand(wv[1][part], q);
    const bool first = part * 32 % G == 0, last = (part + 1) * 32 % G == 0;  // of a group
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 x = xq[part * part_stride + t * 32];
      if (first)
        mma_f16_16816_first(d[t], h2_bits(p[0]), h2_bits(q[0]), h2_bits(p[1]), h2_bits(q[1]), x.x, x.y);
      else
        mma_f16_16816(d[t], h2_bits(p[0]), h2_bits(q[0]), h2_bits(p[1]), h2_bits(q[1]), x.x, x.y);
      mma_f16_16816(d[t], h2_bits(p[2]), h2_bits(q[2]), h2_bits(p[3]), h2_bits(q[3]), x.z, x.w);
      if (last) {
        z[t][0] += s0[part] * d[t][0];
        z[t][1] += s0[part] * d[t][1];
        z[t][2] += s1[part] * d[t][2];
        z[t][3] += s1[part] * d[t][3];
      }
    }
  }
}

// z * 2^e, the power itself perhaps out of fp32's range (e from -252 to 252)
__device__ __forceinline__ float by_pow2(float z, int e) { return z * pow2(e / 2) * pow2(e - e / 2); }
// a row's sum with its scaling taken back
__device__ __forceinline__ float unscale(float z, uint32_t top) { return by_pow2(z, -scale_exponent(top)); }

// ---- few activations: one tile of columns, staged whole by every block.  A block is 8 warps: R tiles of 16 rows
// times 8 / R parts of W's columns (blocks of 128, taken in turn), whose sums are added in order at the end.
// 19456 x 2560, one fp32 row, weights not in L2: 11.0 us, 2.6 TB/s of codes and scales; the launch and the staging are
// 3 of them.
constexpr int kFewAhead = 8;
template <typename T>
constexpr int kFewItems = sizeof(T) == 4 ? 4 : 8;  // loads of 8 activations that a thread has in flight

template <typename T, int G>
__global__ void __launch_bounds__(32 * kWarps, 2) k_q4_few(const MatmulArgs a) {
  constexpr int TN = kTerms<T>, kItems = kFewItems<T>, kOut = 9;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t top[8];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int parts = kWarps / a.tiles, tile = warp % a.tiles, part_k = warp / a.tiles;
  const int blocks = (a.k + kBlock - 1) / kBlock, nn = a.n, live = nn * TN;
  uint4* xs = reinterpret_cast<uint4*>(smem + kWarps * kFewAhead * kRing);  // [block, part][live column][lane c]
  const int row0 = (blockIdx.x * a.tiles + tile) * 16;

  Codes<G, kFewAhead> codes(smem + warp * kFewAhead * kRing, a, row0, blocks, part_k,
                            (blocks - part_k + parts - 1) / parts, parts);
#pragma unroll
  for (int i = 0; i < kFewAhead - 1; ++i) {
    codes.issue();
    cp_async_commit();
  }
  Eight<T> held[kItems];
  const int items = blocks * 16 * nn;
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int i = threadIdx.x + u * 32 * kWarps, pc = i / 4, row = pc % nn, p = pc / nn;
    const int k = p * 32 + i % 4 * 8;
    if (i < items && k < a.k)
      held[u].load(static_cast<const T*>(a.x) + row * a.x_stride + k);
    else
      held[u].zero();
  }
  if (threadIdx.x < 8) top[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (u * 32 * kWarps >= items) break;
    uint32_t t = largest(held[u]);
    if (nn == 1) {
      t = __reduce_max_sync(0xffffffffu, t);
      if (lane == 0) atomicMax(top, t);
    } else {
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
      if (c == 0) atomicMax(top + (threadIdx.x + u * 32 * kWarps) / 4 % nn, t);
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    if (u * 32 * kWarps >= items) break;
    const int i = threadIdx.x + u * 32 * kWarps, pc = i / 4, row = pc % nn, p = pc / nn;
    const Staged<T> st(held[u], pow2(scale_exponent(top[row])));
    if (i < items)
#pragma unroll
      for (int t = 0; t < TN; ++t) xs[(p * live + row * TN + t) * 4 + c] = st.b[t];
  }
  __syncthreads();

  float z[1][4] = {};
  const uint4* xl = xs + (g < live ? lane : 0);  // the other columns' sums are not used
  int j = 0;
  for (int b = part_k; b < blocks; b += parts, ++j) {
    codes.issue();
    cp_async_commit();
    cp_async_wait_group<kFewAhead - 1>();
    __syncwarp();
    multiply<1, G>(smem_u32(codes.ring + j % kFewAhead * kRing), codes.par0 + j * parts, codes.par1 + j * parts,
                   xl + b * 16 * live, 4 * live, z);
    __syncwarp();
  }
  cp_async_wait_all();
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem);
  const int rows = a.tiles * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[(part_k * rows + tile * 16 + g + i / 2 * 8) * kOut + 2 * c + i % 2] = z[0][i];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * nn; i += 32 * kWarps) {
    const int r = i % rows, col = i / rows, row = blockIdx.x * rows + r;
    if (row >= a.m) continue;
    float v = 0.f;
    for (int q = 0; q < parts; ++q)
#pragma unroll
      for (int t = TN - 1; t >= 0; --t) v += out[(q * rows + r) * kOut + col * TN + t];
    static_cast<T*>(a.y)[static_cast<size_t>(col) * a.m + row] = from_f<T>(unscale(v, top[col]));
  }
}

template <typename T>
bool few(int n, int blocks) {
  return static_cast<long long>(n) * kTerms<T> <= 8 &&
         static_cast<long long>(n) * blocks * 16 <= kFewItems<T> * 32 * kWarps;
}

// shared memory: at most kFewItems * 16 (row, block) pairs
template <typename T>
constexpr int kFewMost = kWarps * kFewAhead * kRing + kFewItems<T> * 16 * 256 * kTerms<T>;

template <typename T, int G>
int launch_few(MatmulArgs a, cudaStream_t st) {
  const int all = (a.m + 15) / 16, blocks = (a.k + kBlock - 1) / kBlock;
  a.tiles = kWarps;  // R: the most row tiles in a block that leave two blocks an SM
  while (a.tiles > 1 && (all + a.tiles - 1) / a.tiles < 304) a.tiles /= 2;
  const int smem = kWarps * kFewAhead * kRing + blocks * 256 * a.n * kTerms<T>;
  if (!allow_smem<k_q4_few<T, G>, kFewMost<T>>()) return S2_ECUDA;
  k_q4_few<T, G><<<(all + a.tiles - 1) / a.tiles, 32 * kWarps, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

// ---- more activations: staged once, as planes in the workspace that every block then copies.

// tcgen05 takes over behind 32 columns (19456 x 2560 at 64: 35 us on mma.sync, 21 there), and behind 16 for matrices
// of 32 Mi weights on.  With weights not in L2, groups of 32, at 17 and 32 columns on mma.sync and on tcgen05:
// 19456 x 2560 19.2 and 19.5 us, 17.5 and 18.8; 12288 x 2560 16.0 and 16.8, 16.5 and 17.7; 2560 x 9728 16.1 and 16.8,
// 17.1 and 17.4; 9728 x 2560 14.2 and 14.6, 18.2 and 19.3; 2560 x 2560 7.9 and 9.1, 10.4 and 10.8.
bool on_tcgen05(long long cols, int m, int k) {
  return cols > 32 || (cols > 16 && static_cast<long long>(m) * k >= 32ll << 20);
}

// What the workspace holds: for mma.sync `tiles` tiles of 8 columns; for tcgen05 `tiles` tiles of `width` columns, as
// its B operand (two 128-byte-swizzled tiles of 64 positions a code block).
struct Planes {
  uint4* b;       // [block, part][tile][lane], or [block][tile][half][column][chunk]
  uint32_t* top;  // [row]
  int tiles, width;
  size_t bytes;
};
Planes planes(int n, int k, int terms, bool tc, void* ws) {
  Planes p{};
  const long long cols = static_cast<long long>(n) * terms;
  const size_t blocks = (static_cast<size_t>(k) + kBlock - 1) / kBlock, parts = blocks * 4;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.b = reinterpret_cast<uint4*>(at);
  if (tc) {
    p.width = cols <= 32 ? 32 : cols <= 64 ? 64 : 128;
    p.tiles = static_cast<int>((cols + p.width - 1) / p.width);
    const size_t b = blocks * p.tiles * p.width * 256;
    p.top = reinterpret_cast<uint32_t*>(at + b);
    p.bytes = b + static_cast<size_t>(n) * 4;
    return p;
  }
  p.width = 8;
  p.tiles = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
  p.top = reinterpret_cast<uint32_t*>(at + parts * p.tiles * 512);
  p.bytes = parts * p.tiles * 512 + static_cast<size_t>(p.tiles) * 8 * 4;
  return p;
}

// One block per activation row (for mma.sync also per row of zeros that fills the last tile; columns behind the last
// row of tcgen05's tiles are never looked at).  Rows of up to 4 items a thread are read once.
constexpr int kPlaneThreads = 512;
template <typename T, bool kTc>
__global__ void __launch_bounds__(kPlaneThreads) k_q4_planes(const MatmulArgs a, const Planes p) {
  constexpr int TN = kTerms<T>, kHeld = 4;
  __shared__ uint32_t top;
  pdl_trigger();  // the products may start on their codes
  const int row = blockIdx.x, lane = threadIdx.x % 32;
  const bool live = row < a.n;
  const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(live ? row : 0) * a.x_stride;
  const int items = (a.k + kBlock - 1) / kBlock * 16;
  auto load = [&](int i) {
    Eight<T> v;
    if (live && i < items && i * 8 < a.k)
      v.load(x + i * 8);
    else
      v.zero();
    return v;
  };
  if (threadIdx.x == 0) top = 0;
  Eight<T> held[kHeld];
  uint32_t t = 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) held[u] = load(threadIdx.x + u * kPlaneThreads);
#pragma unroll
  for (int u = 0; u < kHeld; ++u) t = max(t, largest(held[u]));
  for (int i = threadIdx.x + kHeld * kPlaneThreads; i < items; i += kPlaneThreads) t = max(t, largest(load(i)));
  t = __reduce_max_sync(0xffffffffu, t);
  __syncthreads();
  if (lane == 0) atomicMax(&top, t);
  __syncthreads();
  const float up = pow2(scale_exponent(top));
  if (threadIdx.x == 0) p.top[row] = top;
  auto store = [&](const Eight<T>& v, int i) {
    if (i >= items) return;
    const Staged<T> st(v, up);
#pragma unroll
    for (int u = 0; u < TN; ++u) {
      const int col = row * TN + u;
      if constexpr (kTc) {
        const int q = i % 4 * 4 + i / 4 % 4, at = col % p.width;  // q: the word of the code block that holds these columns
        p.b[((static_cast<size_t>(i / 16) * p.tiles + col / p.width) * 2 + q / 8) * p.width * 8 + at * 8 +
            ((q % 8) ^ (at & 7))] = st.b[u];
      } else {
        p.b[(static_cast<size_t>(i / 4) * p.tiles + col / 8) * 32 + col % 8 * 4 + i % 4] = st.b[u];
      }
    }
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (u * kPlaneThreads < items) store(held[u], threadIdx.x + u * kPlaneThreads);
  for (int i0 = kHeld * kPlaneThreads; i0 < items; i0 += kPlaneThreads) store(load(i0 + threadIdx.x), i0 + threadIdx.x);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank));
  return v;
}

__device__ __forceinline__ float ld_cluster1(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(addr), "r"(rank));
  return v;
}

// A block takes 64 rows (a warp 16) and a range of W's columns; the blocks of a cluster split W's columns and add
// their sums through distributed shared memory in rank order.  Every step is one block of 128 columns: its
// activations are copied for all warps, kAhead steps ahead, and one barrier a step passes them on.  16 bf16 rows,
// 19456 x 2560, weights not in L2: 15.8 us; 17 rows, 2560 x 2560: 8.3; 32 rows, 2560 x 9728: 15.1.  At 32 columns a step of 128 takes 0.9 us, bound by mma.sync.
constexpr int kManyWarps = 4, kManyRows = 16 * kManyWarps;
constexpr int kJoinRow = kManyRows + 4;  // floats of a column in the joining buffer: 4-row groups, no bank conflicts
template <int NT>
constexpr int kManyAhead = NT == 1 ? 8 : 4;
template <int NT>
constexpr int kStepBytes = 4 * NT * 512;

template <typename T, int NT, int G>
__global__ void __launch_bounds__(32 * kManyWarps, 16 / kManyWarps) k_q4_many(const MatmulArgs a, const Planes p) {
  constexpr int TN = kTerms<T>, kAhead = kManyAhead<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t top[8 * NT];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int blocks = (a.k + kBlock - 1) / kBlock;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * rank / ranks);
  const int count = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / ranks) - b0;
  uint8_t* xring = smem + kManyWarps * kAhead * kRing;
  Codes<G, kAhead> codes(smem + warp * kAhead * kRing, a, blockIdx.x * kManyRows + warp * 16, blocks, b0, count, 1);
  auto copy_x = [&](int j) {
    if (j >= count) return;
    uint8_t* dst = xring + j % kAhead * kStepBytes<NT>;
    const size_t part = static_cast<size_t>(b0 + j) * 4;
#pragma unroll
    for (int i = threadIdx.x; i < 4 * NT * 32; i += 32 * kManyWarps)
      cp_async16(dst + i * 16, p.b + part * NT * 32 + i);
  };
  // codes do not depend on the kernel in front, which runs after all that came before it
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) codes.issue();
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) {
    copy_x(i);
    cp_async_commit();  // the first group holds the codes of all of them
  }
  if (threadIdx.x < 8 * NT / TN) top[threadIdx.x] = p.top[threadIdx.x];
  float z[NT][4] = {};
  for (int j = 0; j < count; ++j) {
    cp_async_wait_group<kAhead - 2>();
    __syncthreads();  // step j is here, and step j - 1 is used up
    codes.issue();
    copy_x(j + kAhead - 1);
    cp_async_commit();
    const uint8_t* xq = xring + j % kAhead * kStepBytes<NT>;
    multiply<NT, G>(smem_u32(codes.ring + j % kAhead * kRing), codes.par0 + j, codes.par1 + j,
                    reinterpret_cast<const uint4*>(xq) + lane, NT * 32, z);
  }
  cp_async_wait_all();
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[(8 * t + 2 * c + i % 2) * kJoinRow + warp * 16 + g + i / 2 * 8] = z[t][i];
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  // a thread adds up four rows of one column
  const int quads = kManyRows / 4 / ranks;
  for (int i = threadIdx.x; i < quads * a.n; i += 32 * kManyWarps) {
    const int r = (rank * quads + i % quads) * 4, col = i / quads, row = blockIdx.x * kManyRows + r;
    float v[4] = {};
    const float* at = out + col * TN * kJoinRow + r;
    float4 u[8][TN];
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int t = 0; t < TN; ++t) {
        u[q][t] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q < ranks)
          u[q][t] = ranks > 1 ? ld_cluster(smem_u32(at + t * kJoinRow), q)
                              : *reinterpret_cast<const float4*>(at + t * kJoinRow);
      }
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int t = TN - 1; t >= 0; --t) v[0] += u[q][t].x, v[1] += u[q][t].y, v[2] += u[q][t].z, v[3] += u[q][t].w;
    T* y = static_cast<T*>(a.y) + static_cast<size_t>(col) * a.m + row;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (row + e < a.m) y[e] = from_f<T>(unscale(v[e], top[col]));
  }
  if (ranks > 1) cluster_sync();  // no block leaves while its sums are read
}

// a grid of clusters of `ranks` blocks, which may start before the kernel in front ends
int launch_joined(void (*kernel)(MatmulArgs, Planes), dim3 grid, int threads, int smem, int ranks, const MatmulArgs& a,
                  const Planes& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = ranks;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, p) == cudaSuccess ? S2_OK : S2_ECUDA;
}

template <typename T, int NT, int G>
int launch_many(const MatmulArgs& a, const Planes& p, cudaStream_t st) {
  const int blocks = (a.k + kBlock - 1) / kBlock, grid = (a.m + kManyRows - 1) / kManyRows;
  // Up to four blocks an SM in clusters of two, about two in larger ones (608 blocks in clusters of four do not all
  // fit at a time: 9728 x 1024, 32 rows, 13.7 us against 8.5), of two code blocks at least.
  int ranks = 1;
  while (ranks < 8 && static_cast<long long>(grid) * ranks * 2 <= (ranks == 1 ? 608 : 320) && blocks >= 4 * ranks)
    ranks *= 2;
  constexpr int kRings = kManyAhead<NT> * (kManyWarps * kRing + kStepBytes<NT>), kJoin = 8 * NT * kJoinRow * 4;
  constexpr int smem = kRings > kJoin ? kRings : kJoin;
  if (!allow_smem<k_q4_many<T, NT, G>, smem>()) return S2_ECUDA;
  k_q4_planes<T, false><<<p.tiles * 8 / kTerms<T>, kPlaneThreads, 0, st>>>(a, p);
  if (cudaGetLastError() != cudaSuccess) return S2_ECUDA;  // else the products would be of an old workspace
  return launch_joined(k_q4_many<T, NT, G>, dim3(grid, ranks), 32 * kManyWarps, smem, ranks, a, p, st);
}

// ---- many activations: tcgen05, its A operand the weights.  A block takes 128 rows and N columns; twice four warps
// expand code blocks in turn, a thread its row's, to fp16 in tensor memory; a ninth issues the products, a tenth copies
// activations, one bulk copy a code block.  scale * (code - 8) has 8 + 3 significant bits, so it is exact in fp16: each row's scales are
// taken times the power of two that brings the largest of those used here to 2^11 .. 2^12 (scales 2^-28 of it and
// less lose bits).  The blocks of a cluster split W's columns and add their sums in rank order.
// The tensor core cuts every product's sum off at its last bit: a few 1e-8 each, in one direction.  16-bit results do not
// show it (6e-6 over 9728 columns).  Of fp32 rows the sums of two code blocks at a time (chunks) are added up in
// registers: 3e-7 at any k where they were up to 6e-6 off; 1024 rows of 19456 x 2560 take 201 us, 187 without.
// 19456 x 2560, 2048 bf16 rows: 207 us, 990 TFLOP/s; 512 rows 53 us; bound by the activations that every block reads
// again from L2 (9 TB/s).  64 rows 20.5 us.
template <int N>
struct Tc {
  static constexpr int kA = N == 128 ? 2 : 3;                      // expanded code blocks, 64 tensor memory columns each
  static constexpr int kB = N == 32 ? 4 : N == 64 ? 3 : 2;         // code blocks' activations
  static constexpr int kAhead = N == 32 ? 4 : N == 64 ? 3 : 2;     // code blocks of a warp in flight
  static constexpr int kBBytes = N * 256, kRow = 32 * 64 + 32 * 8;  // of a code block: activations; a warp's codes and scales
  static constexpr int kCodes = kB * kBBytes, kBars = kCodes + 8 * kAhead * kRow, kBytes = kBars + 192 + 1024;
  static constexpr uint32_t kCols = 256;
  static_assert(N + 64 * kA <= kCols && (N + 1) * 512 <= kBars, "room");
};

constexpr int kTcThreads = 320;
template <typename T, int N, int G>
__global__ void __launch_bounds__(kTcThreads, 2) k_q4_tc(const MatmulArgs a, const Planes p) {
  using M = Tc<N>;
  constexpr int TN = kTerms<T>, SB = kBlock / G;
  constexpr bool kChunks = TN == 2;
  extern __shared__ __align__(16) uint8_t smraw[];
  __shared__ int ex[N / TN], ew[128];  // powers of two of the activations' and the weights' rows
  uint8_t* sm = smraw + (-smem_u32(smraw) & 1023u);
  uint64_t* arrived = reinterpret_cast<uint64_t*>(sm + M::kBars);  // [j % kB]: activations of code block j
  uint64_t* freed = arrived + M::kB;                               // [j % kB]: used up
  uint64_t *expanded = freed + M::kB, *used = expanded + M::kA;    // [j % kA]: its weights; used up
  uint64_t *done = used + M::kA, *taken = done + 1;                // a chunk's products (or all); its sums read
  uint64_t* drained = taken + 1;                                   // nothing under way
  uint32_t* tbase = reinterpret_cast<uint32_t*>(drained + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const int blocks = (a.k + kBlock - 1) / kBlock;
  const int ranks = gridDim.y, rank = blockIdx.y;
  const int b0 = static_cast<int>(static_cast<long long>(blocks) * rank / ranks);
  const int count = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / ranks) - b0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * M::kB; ++i) mbar_init(arrived + i, 1);
    for (int i = 0; i < M::kA; ++i) {
      mbar_init(expanded + i, 4);
      mbar_init(used + i, 1);
    }
    mbar_init(done, 1);
    mbar_init(taken, 8);
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
  const int n0 = blockIdx.z * (N / TN), nn = min(N / TN, a.n - n0), wg = warp / 4;
  const uint32_t tsum = tm + (static_cast<uint32_t>(warp % 4 * 32) << 16) + wg * 16;
  float acc[kChunks ? N / 4 : 1] = {};  // of this thread's row, half of the columns
  if (warp == 8) {
    // ---------------------------------------------------------------- issuing the products
    if (elect_one()) {
      for (int j = 0; j < count && ok; ++j) {
        ok = mbar_wait_short(arrived + j % M::kB, j / M::kB & 1, a.tries) &&
             mbar_wait_short(expanded + j % M::kA, j / M::kA & 1, a.tries) &&
             (!kChunks || j < 2 || j % 2 || mbar_wait_short(taken, (j / 2 - 1) & 1, a.tries));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = tm + N + j % M::kA * 64;
        const uint64_t b = desc_sw128(smem_u32(sm + j % M::kB * M::kBBytes));
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k)
          tc_mma_tmem_a(tm, ta + k * 8, b + ((k / 4 * (N * 128) + k % 4 * 32) >> 4), idesc_f16(128, N),
                        (kChunks ? j % 2 : j) > 0 || k > 0);
        tc_commit(freed + j % M::kB);
        tc_commit(used + j % M::kA);
        if (j == count - 1 || (kChunks && j % 2)) tc_commit(done);
      }
      tc_commit(drained);  // no end before that of the products, whoever gave up
      mbar_wait_short(drained, 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------------- copying activations
    pdl_wait();
    if (lane == 0) {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(p.b) + (static_cast<size_t>(b0) * p.tiles + blockIdx.z) * M::kBBytes;
      int j = 0;
      for (; j < count; ++j) {
        if (j >= M::kB) ok = mbar_wait_short(freed + j % M::kB, (j / M::kB - 1) & 1, a.tries);
        if (!ok) break;
        mbar_arrive_expect_tx(arrived + j % M::kB, M::kBBytes);
        bulk_g2s_plain(sm + j % M::kB * M::kBBytes, src + static_cast<size_t>(j) * p.tiles * M::kBBytes, M::kBBytes,
                       arrived + j % M::kB);
      }
      for (int i = max(j - M::kB, 0); i < j; ++i)  // no end before that of the copies
        mbar_wait_short(arrived + i % M::kB, i / M::kB & 1);
    }
    __syncwarp();
    for (int i = lane; i < nn; i += 32) ex[i] = scale_exponent(__ldcg(p.top + n0 + i));
  } else {
    // ---------------------------------------------------------------- expanding
    const int mine = (count - wg + 1) / 2;  // the code blocks 2 t + wg
    uint8_t* ring = sm + M::kCodes + warp * M::kAhead * M::kRow;
    const int in = warp % 4 * 32, row0 = blockIdx.x * 128 + in;
    const uint8_t* from[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      from[i] = a.codes + (static_cast<size_t>(min(row0 + i * 8 + lane / 4, a.m - 1)) * blocks + b0 + wg) * 64 + lane % 4 * 16;
    const size_t first = (static_cast<size_t>(min(row0 + lane, a.m - 1)) * blocks + b0 + wg) * SB;
    const size_t send = static_cast<size_t>(a.m) * blocks * SB;
    auto issue = [&](int t) {
      if (t < mine) {
        uint8_t* dst = ring + t % M::kAhead * M::kRow;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4;
          cp_async16(dst + r * 64 + ((lane % 4) ^ (r / 2 & 3)) * 16, from[i] + static_cast<size_t>(t) * 128);
        }
        const size_t at = first + static_cast<size_t>(t) * 2 * SB;
        if constexpr (G == 128)  // two bytes wanted: the aligned four around them, less what lies past the last scale
          cp_async_small<4>(dst + 2048 + lane * 8, a.scales + (at & ~size_t{1}), (at | 1) < send ? 4 : 2);
        else
          cp_async_small<2 * SB>(dst + 2048 + lane * 8, a.scales + at, 2 * SB);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < M::kAhead - 1; ++i) issue(i);
    // the largest finite scale here of each of 16 rows: a code block a lane, the rows under way together
    uint32_t most = 0;
    using Unit = std::conditional_t<SB == 4, uint2, std::conditional_t<SB == 2, uint32_t, uint16_t>>;
#pragma unroll 1
    for (int b = 0; b < count; b += 32) {
      Unit v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] = Unit{};
        if (b + lane < count)
          v[r] = __ldg(reinterpret_cast<const Unit*>(
                           a.scales + (static_cast<size_t>(min(row0 + wg * 16 + r, a.m - 1)) * blocks + b0) * SB) + b + lane);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        uint32_t t = 0;
        auto look = [&](uint32_t bits) { t = max(t, (bits & 0x7fffu) < 0x7f80u ? bits & 0x7fffu : 0u); };
        if constexpr (SB == 4)
          look(v[r].x), look(v[r].x >> 16), look(v[r].y), look(v[r].y >> 16);
        else
          look(v[r]), look(static_cast<uint32_t>(v[r]) >> 16);
        t = __reduce_max_sync(0xffffffffu, t);
        if (lane == r) most = max(most, t);
      }
    }
    if (lane < 16) ew[in + wg * 16 + lane] = most == 0 ? 0 : min(11 + 127 - static_cast<int>(most >> 7), 126);
    named_bar(1, 256);
    const float up = pow2(ew[in + lane]);
    const uint32_t tlane = tm + N + (static_cast<uint32_t>(warp % 4 * 32) << 16);
    // a chunk's sums, which make room for the next chunk's
    auto take = [&](int chunk) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_short(done, chunk & 1, a.tries));
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < N / 32; ++i) {
        float v[16];
        tmem_ld16(tsum + i * 32, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i * 8 + e] += v[2 * e] + v[2 * e + 1];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(taken);
    };
    for (int t = 0; t < mine; ++t) {
      const int j = 2 * t + wg;
      issue(t + M::kAhead - 1);
      cp_async_wait_group<M::kAhead - 1>();
      __syncwarp();
      const uint32_t at = smem_u32(ring + t % M::kAhead * M::kRow);
      uint4 w[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = lds128(at + lane * 64 + ((c ^ (lane / 2 & 3)) * 16));
      __half2 s[4];
      {
        const uint32_t u = lds32(at + 2048 + lane * 8);
        auto h = [&](float f) { return __float2half2_rn(f * up); };
        if constexpr (G == 32) {
          const uint32_t v = lds32(at + 2048 + lane * 8 + 4);
          s[0] = h(bf16lo(u)), s[1] = h(bf16hi(u)), s[2] = h(bf16lo(v)), s[3] = h(bf16hi(v));
        } else if constexpr (G == 64) {
          s[0] = s[1] = h(bf16lo(u)), s[2] = s[3] = h(bf16hi(u));
        } else {
          s[0] = s[1] = s[2] = s[3] = h(first & 1 ? bf16hi(u) : bf16lo(u));
        }
      }
      __syncwarp();  // the ring's place may be filled again
      if (j >= M::kA) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait_short(used + j % M::kA, (j / M::kA - 1) & 1, a.tries));
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 x = w[half * 2 + c];
          const uint32_t word[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __half2 v[4];
            expand(word[i], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) r[c * 16 + i * 4 + e] = h2_bits(__hmul2(s[i], v[e]));
          }
        }
        tmem_st32(tlane + j % M::kA * 64 + half * 32, r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(expanded + j % M::kA);
      if constexpr (kChunks) {
        if (t > 0) take(t - 1);
        if (!ok) break;
      }
    }
    cp_async_wait_all();
    if constexpr (kChunks) {
      for (int i = max(mine - 1, 0); i < (count + 1) / 2 && ok; ++i) take(i);
    } else {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_short(done, 0, a.tries));
      tc_fence_after();
    }
  }
  // two threads a row, each half of the columns; a wait that gave up leaves no numbers
  const int r = threadIdx.x % 128, row = blockIdx.x * 128 + r;
  T* y = static_cast<T*>(a.y) + static_cast<size_t>(n0) * a.m + row;
  constexpr int kAt = 16 / TN;  // columns of x that 16 columns of sums are
  auto sums = [&](auto use) {   // use(first column, kAt sums)
    if constexpr (kChunks) {
#pragma unroll
      for (int i = 0; i < N / 32; ++i)
        if (wg * kAt + i * 2 * kAt < nn) use(wg * kAt + i * 2 * kAt, acc + i * kAt);
    } else {
#pragma unroll 1
      for (int c = wg * 16; c < nn; c += 32) {
        float v[16];
        __syncwarp();
        tmem_ld16(tsum + c - wg * 16, v);
        use(c, v);
      }
    }
  };
  __syncthreads();
  if (ranks == 1) {
    if (warp < 8)
      sums([&](int c, const float* v) {
        if (row >= a.m) return;
#pragma unroll
        for (int i = 0; i < kAt; ++i)
          if (c + i < nn)
            y[static_cast<size_t>(c + i) * a.m] = from_f<T>(ok ? by_pow2(v[i], -ew[r] - ex[c + i]) : NAN);
      });
  } else {
    // sums as [column][row] where the operands were, behind them the weights' powers of two
    float* out = reinterpret_cast<float*>(sm);
    constexpr int kEnd = N / TN * 128;
    if (warp < 8) {
      sums([&](int c, const float* v) {
#pragma unroll
        for (int i = 0; i < kAt; ++i) out[(c + i) * 128 + r] = ok ? v[i] : NAN;
      });
      if (wg == 0) out[kEnd + r] = __int_as_float(ew[r]);
    }
    cluster_sync();
    if (warp < 8) {
      int e[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < ranks) e[q] = __float_as_int(ld_cluster1(smem_u32(out + kEnd + r), q));
      for (int col = wg * ranks + rank; col < nn; col += 2 * ranks) {
        float v[8], sum = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < ranks) v[q] = ld_cluster1(smem_u32(out + col * 128 + r), q);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < ranks) sum += by_pow2(v[q], -e[q] - ex[col]);
        if (row < a.m) y[static_cast<size_t>(col) * a.m] = from_f<T>(sum);
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

template <typename T, int N, int G>
int launch_tc(const MatmulArgs& a, const Planes& p, cudaStream_t st) {
  const int blocks = (a.k + kBlock - 1) / kBlock, grid = (a.m + 127) / 128;
  // Clusters up to what the SMs hold (two blocks each): 256 columns, 2560 x 9728, 34 us against 57 with one block an
  // SM; 19456 x 2560 at 64 columns 23 against 41 with four, which take two rounds.
  int ranks = 1;
  while (ranks < 8 && static_cast<long long>(grid) * p.tiles * ranks * 2 <= 304 && blocks >= 4 * ranks) ranks *= 2;
  constexpr int smem = Tc<N>::kBytes;
  if (!allow_smem<k_q4_tc<T, N, G>, smem>()) return S2_ECUDA;
  k_q4_planes<T, true><<<a.n, kPlaneThreads, 0, st>>>(a, p);
  if (cudaGetLastError() != cudaSuccess) return S2_ECUDA;
  return launch_joined(k_q4_tc<T, N, G>, dim3(grid, ranks, p.tiles), kTcThreads, smem, ranks, a, p, st);
}

template <typename T, int G>
int launch_matmul(const MatmulArgs& a, void* ws, cudaStream_t st) {
  if (few<T>(a.n, (a.k + kBlock - 1) / kBlock)) return launch_few<T, G>(a, st);
  const bool tc = on_tcgen05(static_cast<long long>(a.n) * kTerms<T>, a.m, a.k);
  const Planes p = planes(a.n, a.k, kTerms<T>, tc, ws);
  if (tc)
    return p.width == 32 ? launch_tc<T, 32, G>(a, p, st)
                         : p.width == 64 ? launch_tc<T, 64, G>(a, p, st) : launch_tc<T, 128, G>(a, p, st);
  return p.tiles == 1 ? launch_many<T, 1, G>(a, p, st)
                      : p.tiles == 2 ? launch_many<T, 2, G>(a, p, st) : launch_many<T, 4, G>(a, p, st);
}

constexpr int kRowsMost = 1 << 21, kMatmulMost = 1 << 28;  // activation rows, the other sizes

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

extern "C" size_t s2_q4_matmul_workspace(int n, int k, int dtype) {
  if (n < 1 || k < 1 || n > kRowsMost || k > kMatmulMost || !dtype_bytes(dtype)) return 0;
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (few<T>(n, (k + kBlock - 1) / kBlock)) return size_t{0};
    // whatever the matrix
    const size_t tc = planes(n, k, kTerms<T>, true, nullptr).bytes;
    return on_tcgen05(static_cast<long long>(n) * kTerms<T>, 1, 1) ? tc
                                                                   : std::max(tc, planes(n, k, kTerms<T>, false, nullptr).bytes);
  });
}

extern "C" int s2_q4_matmul(int n, const void* x, int dtype, long long x_stride, const uint8_t* codes,
                            const void* scales, int m, int k, int group, void* y, void* workspace, size_t ws_bytes,
                            CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (!x || !codes || !scales || !y || !esz || n < 1 || m < 1 || k < 1 || bad_group(group) || k % group != 0 ||
      x_stride < k || n > kRowsMost || m > kMatmulMost || k > kMatmulMost)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(x) % 16 != 0 || x_stride * esz % 16 != 0 ||
      reinterpret_cast<uintptr_t>(codes) % 16 != 0 || reinterpret_cast<uintptr_t>(scales) % (group == 32 ? 8 : 4) != 0 ||
      reinterpret_cast<uintptr_t>(y) % esz != 0 || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return S2_EINVAL;
  const size_t need = s2_q4_matmul_workspace(n, k, dtype);
  if (need > 0 && (!workspace || ws_bytes < need)) return S2_EINVAL;
  const MatmulArgs a{x, x_stride, n, m, k, codes, static_cast<const __nv_bfloat16*>(scales), y, 0,
                     wait_tries.load(std::memory_order_relaxed)};
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return group == 32 ? launch_matmul<T, 32>(a, workspace, st)
                       : group == 64 ? launch_matmul<T, 64>(a, workspace, st) : launch_matmul<T, 128>(a, workspace, st);
  });
}
