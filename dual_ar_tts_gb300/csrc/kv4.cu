// Appending to the paged 4-bit cache and reading it back (see kv4.cuh for the layout).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "kv4.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

// exact sum of two fp32 as hi + lo
__device__ __forceinline__ void two_sum(float a, float b, float& hi, float& lo) {
  hi = __fadd_rn(a, b);
  const float t = __fsub_rn(hi, a);
  lo = __fadd_rn(__fsub_rn(a, __fsub_rn(hi, t)), __fsub_rn(b, t));
}

// Sum of squares of a head's elements (8 a lane) to well below one fp32 rounding (hi + lo pairs, products
// split with an FMA): a key is quantised after its norm, and a scale that is off in the last place
// would move codes of elements next to a rounding border.
template <int HD>
__device__ __forceinline__ float sum_squares(const float (&x)[8]) {
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = __fmul_rn(x[i], x[i]);
    lo += __fmaf_rn(x[i], x[i], -p);
    float h, l;
    two_sum(hi, p, h, l);
    hi = h;
    lo += l;
  }
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, lo, o);
    float h, l;
    two_sum(hi, oh, h, l);
    hi = h;
    lo = lo + ol + l;
  }
  return isfinite(hi) ? hi + lo : hi;  // where hi is infinite, lo is none
}

// The same to a few fp32 roundings, for queries.
template <int HD>
__device__ __forceinline__ float sum_squares_fp32(const float (&x)[8]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = __fmaf_rn(x[i], x[i], sum);
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Mean square of a head, for the whole warp.  Where the sum is past fp32's range the mean may not be: it is then taken of
// x / 2^64 (of which what underflows does not count).
template <int HD, bool kKey>
__device__ __forceinline__ float mean_square(const float (&x)[8]) {
  auto mean = [](const float(&v)[8]) { return (kKey ? sum_squares<HD>(v) : sum_squares_fp32<HD>(v)) * (1.f / HD); };
  float m = mean(x);
  if (__any_sync(0xffffffffu, isinf(m))) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * 0x1p-64f;
    const float small = mean(y);
    if (isinf(m)) m = small * 0x1p64f * 0x1p64f;
  }
  return m;
}

struct AppendArgs {
  s2_kv4 c;
  const void* qkv;
  long long stride;
  int n_head;
  const float* rope;
  int n_pos;
  const float* q_norm;
  const float* k_norm;
  float eps;
  void* q_out;
};

// Where a call's row lies: its sequence's position, and that position's page (-1: none, or out of range).
struct Place {
  bool live;  // a row of some sequence
  int pos, page;
};
__device__ __forceinline__ Place place_of(const s2_kv4& c, int row, int n_pos) {
  const int seq = seq_of_row(c.q_start, c.n_seq, row);
  Place p{seq < c.n_seq, -1, -1};
  if (!p.live) return p;
  const int q0 = __ldg(c.q_start + seq), q1 = __ldg(c.q_start + seq + 1), len = __ldg(c.lengths + seq);
  p.pos = len - (q1 - row);
  if (row >= q0 && p.pos >= 0 && p.pos < n_pos && p.pos / kPage < c.table_cols)
    p.page = __ldg(c.table + static_cast<size_t>(seq) * c.table_cols + p.pos / kPage);
  if (p.page >= c.n_pages) p.page = -1;
  return p;
}

// A lane holds 8 consecutive elements: a head is kLanes lanes, four lanes are a quantisation group, and a warp
// works on 32 / kLanes heads at a time.
template <int HD>
constexpr int kLanes = HD / 8;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  uint4 u[sizeof(T) / 2];
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f(e[i]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  uint4 u[sizeof(T) / 2];
  T* e = reinterpret_cast<T*>(u);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f<T>(x[i]);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
}

// maximum and minimum of which a NaN is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// rint(x / s) of the correctly rounded quotient, for quotients of up to 2^8: the product with 1 / s is within
// 2^-14 of it, so a division is needed only where that is next to a border.
struct Quotients {
  float s, inv;
  __device__ __forceinline__ explicit Quotients(float scale) : s(scale), inv(1.f / scale) {}
  __device__ __forceinline__ void round(const float (&x)[8], float (&r)[8]) const {
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = x[i] * inv;
      r[i] = rintf(t);
      near = near || fabsf(t - r[i]) > 0.5f - 0x1p-13f;
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = rintf(__fdiv_rn(x[i], s));
    }
  }
};

// One item: 8 elements of head h (of [q | k | v]) of a row.  Every fp32 operation is rounded by itself, as the
// cache's definition has it.  The heads of a warp may be of different kinds: what has shuffles in it is for all lanes
// where any of them needs it.
template <typename T, int HD>
__device__ __forceinline__ void append_item(const AppendArgs& a, int row, const Place& at, int h, int sub, bool live,
                                            const float4 (&cs)[2], float (&x)[8]) {
  using B = Kv4Block<HD>;
  const bool is_q = h < a.n_head, is_v = h >= a.n_head + a.c.n_kv_head, is_k = !is_q && !is_v;
  const float* w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
  float mean = 0.f;
  if (a.k_norm && __any_sync(0xffffffffu, is_k)) mean = mean_square<HD, true>(x);
  if (a.q_norm && __any_sync(0xffffffffu, is_q)) {
    const float m = mean_square<HD, false>(x);
    if (is_q) mean = m;  // whatever heads share the warp
  }
  if (w) {
    const float r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(mean, a.eps)));
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(w) + sub * 2), w1 = __ldg(reinterpret_cast<const float4*>(w) + sub * 2 + 1);
    const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), ww[i]);
  }
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float t4[4] = {cs[i].x, cs[i].y, cs[i].z, cs[i].w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float u = x[4 * i + 2 * k], v = x[4 * i + 2 * k + 1];
        x[4 * i + 2 * k] = __fsub_rn(__fmul_rn(u, t4[2 * k]), __fmul_rn(v, t4[2 * k + 1]));
        x[4 * i + 2 * k + 1] = __fadd_rn(__fmul_rn(v, t4[2 * k]), __fmul_rn(u, t4[2 * k + 1]));
      }
    }
  }
  if (is_q && live) store8(static_cast<T*>(a.q_out) + (static_cast<size_t>(row) * a.n_head + h) * HD + sub * 8, x);
  if (__all_sync(0xffffffffu, is_q)) return;
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (is_q || !live) return;
  const bool nan = isnan(hi);
  if (!nan && (lo < -kKvMax || hi > kKvMax)) {
    lo = fminf(fmaxf(lo, -kKvMax), kKvMax);
    hi = fminf(fmaxf(hi, -kKvMax), kKvMax);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -kKvMax), kKvMax);
  }
  const __half sh = __float2half_rn(fmaxf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), __fdiv_rn(fmaxf(-lo, hi), 127.f)));
  const float s = __half2float(sh);
  float z = 0.f;
  uint32_t packed = 0;
  if (s > 0.f && !nan) {
    z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), -127.f), 127.f);
    float r[8];
    Quotients(s).round(x, r);
#pragma unroll
    for (int i = 0; i < 8; ++i)  // a sum of whole numbers, exact
      packed |= static_cast<uint32_t>(fminf(fmaxf(r[i] + z, 0.f), 15.f)) << (4 * i);
  }
  const int kh = is_v ? h - a.n_head - a.c.n_kv_head : h - a.n_head;
  uint8_t* block = static_cast<uint8_t*>(a.c.pages) + (static_cast<size_t>(at.page) * a.c.n_kv_head + kh) * B::kBytes +
                   (is_v ? B::kHalf : 0);
  const int slot = at.pos % kPage;
  *reinterpret_cast<uint32_t*>(block + slot * B::kRow + sub * 4) = packed;
  if (sub % 4 == 0)
    *reinterpret_cast<__half2*>(block + kPage * B::kRow + slot * B::kPar + sub / 4 * 4) =
        __halves2half2(nan ? __float2half_rn(NAN) : sh, __float2half_rn(z));
}

// A block takes one row of the call and some of its heads; its warps take heads in turn.  The first load of a head
// does not wait for the row's place.  One pass: a head is read once, and its sums and extremes are shuffles in a
// quarter or half of a warp.  5916 fp16 rows of 32 + 2 x 8 heads: 47.8 us, 2.6 TB/s; bound by instructions (the norm of
// keys to the last bit, the quotients and codes), not by the bytes, which would take 19.
template <typename T, int HD>
__global__ void __launch_bounds__(256) k_kv4_append(const AppendArgs a) {
  constexpr int kPer = 32 / kLanes<HD>;  // heads that a warp takes at a time
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, sub = lane % kLanes<HD>;
  const int heads = a.n_head + 2 * a.c.n_kv_head, row = blockIdx.x;
  const T* src = static_cast<const T*>(a.qkv) + static_cast<size_t>(row) * a.stride + sub * 8;
  const int step = gridDim.y * blockDim.x / 32 * kPer;
  int h0 = (blockIdx.y * (blockDim.x / 32) + warp) * kPer;
  if (h0 >= heads) return;
  auto load = [&](int h, float (&x)[8]) {
    if (h < heads) {
      load8(src + static_cast<size_t>(h) * HD, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
  };
  float x[8], y[8];
  load(h0 + lane / kLanes<HD>, x);
  const Place at = place_of(a.c, row, a.n_pos);
  if (!at.live) return;
  if (at.page < 0) {
    if (lane == 0) kv4_bad(a.c.status);
    return;
  }
  const float4* rope = reinterpret_cast<const float4*>(a.rope) + (static_cast<size_t>(at.pos) * (HD / 2) + sub * 4) / 2;
  const float4 cs[2] = {__ldg(rope), __ldg(rope + 1)};  // the same for all heads
  for (; h0 < heads; h0 += step) {
    const int h = h0 + lane / kLanes<HD>;
    if (h0 + step < heads) load(h + step, y);
    append_item<T, HD>(a, row, at, h, sub, h < heads, cs, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i];
  }
}

// A warp takes a row's keys and values of 32 / kLanes heads.  5916 rows of 8 heads: 8.3 us, 3.9 TB/s of what it reads
// and writes; a warp's loads are three in a chain (bounds, page, codes) before its only stores.
template <int HD>
__global__ void __launch_bounds__(256) k_kv4_read(const s2_kv4 c, __half* __restrict__ k_out,
                                                  __half* __restrict__ v_out) {
  using B = Kv4Block<HD>;
  constexpr int kPer = 32 / kLanes<HD>;
  const int lane = threadIdx.x % 32, sub = lane % kLanes<HD>;
  const int groups = (c.n_kv_head + kPer - 1) / kPer;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int row = static_cast<int>(item / groups), h = static_cast<int>(item % groups) * kPer + lane / kLanes<HD>;
  if (row >= c.n_rows) return;
  const Place at = place_of(c, row, 0x7fffffff);
  if (!at.live) return;
  if (at.page < 0 && lane == 0) kv4_bad(c.status);
  if (h >= c.n_kv_head) return;
  const uint8_t* block = static_cast<const uint8_t*>(c.pages) +
                         (static_cast<size_t>(max(at.page, 0)) * c.n_kv_head + h) * B::kBytes;
  const int slot = at.pos % kPage;
  uint32_t code[2] = {0, 0}, par[2] = {0, 0};
  if (at.page >= 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      code[i] = *reinterpret_cast<const uint32_t*>(block + i * B::kHalf + slot * B::kRow + sub * 4);
      par[i] = *reinterpret_cast<const uint32_t*>(block + i * B::kHalf + kPage * B::kRow + slot * B::kPar + sub / 4 * 4);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2 p = *reinterpret_cast<const __half2*>(&par[i]);
    const float s = __low2float(p), z = __high2float(p);
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = s * (static_cast<float>(code[i] >> (4 * k) & 15) - z);
    store8((i ? v_out : k_out) + (static_cast<size_t>(h) * c.n_rows + row) * HD + sub * 8, x);
  }
}

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" long long s2_kv4_page_bytes(int n_kv_head, int head_dim) {
  if (n_kv_head < 1 || n_kv_head > 65535 || (head_dim != 64 && head_dim != 128)) return -1;
  return static_cast<long long>(n_kv_head) * (head_dim == 64 ? Kv4Block<64>::kBytes : Kv4Block<128>::kBytes);
}

extern "C" int s2_kv4_append(const s2_kv4* cache, const void* qkv, int dtype, long long qkv_stride, int n_head,
                             const float* rope, int n_pos, const float* q_norm, const float* k_norm, float eps,
                             void* q_out, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (kv4_bad_args(cache) || !qkv || !esz || !rope || n_pos < 1 || n_head < 0 || (n_head > 0 && !q_out) ||
      !(eps >= 0.f) || !std::isfinite(eps))
    return S2_EINVAL;
  const long long heads = n_head + 2ll * cache->n_kv_head;
  if (n_head > 65535 || qkv_stride < heads * cache->head_dim) return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(qkv) % 16 != 0 || qkv_stride * esz % 16 != 0 ||
      reinterpret_cast<uintptr_t>(q_out) % 16 != 0 || reinterpret_cast<uintptr_t>(rope) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(q_norm) % 16 != 0 || reinterpret_cast<uintptr_t>(k_norm) % 16 != 0)
    return S2_EINVAL;
  const AppendArgs a{*cache, qkv, qkv_stride, n_head, rope, n_pos, q_norm, k_norm, eps, q_out};
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // Few rows: a warp for every 2 (hd 128) or 4 heads.  Many: one block of four warps a row, each of which finds the
    // row's place and its rotation once and loads a head ahead.  Few and many, us, fp16: 48 heads of 128, 256 rows 5.3
    // and 6.6, 512 7.4 and 7.4, 1024 11.9 and 9.7, 4096 42.4 and 31.7; 15 heads of 64, 512 rows 3.7 and 3.7, 4096 13.5 and
    // 10.3.  (With two warps a row 5916 rows took 49.3 us, with four 46.6, with eight 50.5.)
    const int turns = static_cast<int>((heads * cache->head_dim / 8 + 255) / 256);
    const bool many = cache->n_rows >= 512;
    const dim3 grid(cache->n_rows, many ? 1 : turns);
    const int threads = many ? 128 : 256;
    if (cache->head_dim == 64)
      k_kv4_append<T, 64><<<grid, threads, 0, st>>>(a);
    else
      k_kv4_append<T, 128><<<grid, threads, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

extern "C" int s2_kv4_read(const s2_kv4* cache, void* k, void* v, CUstream_st* stream) {
  if (kv4_bad_args(cache) || !k || !v) return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(k) % 16 != 0 || reinterpret_cast<uintptr_t>(v) % 16 != 0) return S2_EINVAL;
  const int per = 32 / (cache->head_dim / 8);  // heads of a warp
  const long long grid = (static_cast<long long>(cache->n_rows) * ((cache->n_kv_head + per - 1) / per) + 7) / 8;
  if (grid > 0x7fffffffll) return S2_EINVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64)
    k_kv4_read<64><<<static_cast<unsigned>(grid), 256, 0, st>>>(*cache, static_cast<__half*>(k), static_cast<__half*>(v));
  else
    k_kv4_read<128><<<static_cast<unsigned>(grid), 256, 0, st>>>(*cache, static_cast<__half*>(k), static_cast<__half*>(v));
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
