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

// Sum of squares of the warp's elements to well below one fp32 rounding (hi + lo pairs, products
// split with an FMA): a key is quantised after its norm, and a scale that is off in the last place
// would move codes of elements next to a rounding border.
template <int E>
__device__ __forceinline__ float sum_squares(const float (&x)[E]) {
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float p = __fmul_rn(x[i], x[i]);
    lo += __fmaf_rn(x[i], x[i], -p);
    float h, l;
    two_sum(hi, p, h, l);
    hi = h;
    lo += l;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, hi, o), ol = __shfl_xor_sync(0xffffffffu, lo, o);
    float h, l;
    two_sum(hi, oh, h, l);
    hi = h;
    lo = lo + ol + l;
  }
  return hi + lo;
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

// One warp per (row, head) of [q | k | v].  A lane holds hd / 32 consecutive elements, so rotation
// pairs stay in a lane and a quantisation group is 8 (hd 128) or 16 (hd 64) neighbouring lanes.
template <typename T, int HD>
__global__ void __launch_bounds__(256) k_kv4_append(const AppendArgs a) {
  constexpr int E = HD / 32, GL = kKvGroup / E;
  using B = Kv4Block<HD>;
  const int lane = threadIdx.x % 32;
  const int heads = a.n_head + 2 * a.c.n_kv_head;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int row = static_cast<int>(item / heads), h = static_cast<int>(item % heads);
  if (row >= a.c.n_rows) return;
  const int seq = seq_of_row(a.c.q_start, a.c.n_seq, row);
  if (seq >= a.c.n_seq) return;
  const int pos = a.c.lengths[seq] - (a.c.q_start[seq + 1] - row);
  const bool is_q = h < a.n_head, is_v = h >= a.n_head + a.c.n_kv_head;
  int page = -1;
  if (row >= a.c.q_start[seq] && pos >= 0 && pos < a.n_pos && pos / kPage < a.c.table_cols)
    page = a.c.table[static_cast<size_t>(seq) * a.c.table_cols + pos / kPage];
  if (page < 0 || page >= a.c.n_pages) {
    if (lane == 0) kv4_bad(a.c.status);
    return;
  }
  const T* src = static_cast<const T*>(a.qkv) + row * a.stride + static_cast<size_t>(h) * HD + lane * E;
  float x[E];
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = to_f(src[i]);
  if (!is_v) {
    const float* w = is_q ? a.q_norm : a.k_norm;
    if (w) {
      const float mean = sum_squares<E>(x) * (1.f / HD);
      const float r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(mean, a.eps)));
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), __ldg(w + lane * E + i));
    }
    const float2* cs = reinterpret_cast<const float2*>(a.rope) + static_cast<size_t>(pos) * (HD / 2) + lane * E / 2;
#pragma unroll
    for (int i = 0; i < E; i += 2) {  // each product rounded by itself, as the cache's definition has it
      const float2 t = __ldg(cs + i / 2);
      const float u = x[i], v = x[i + 1];
      x[i] = __fsub_rn(__fmul_rn(u, t.x), __fmul_rn(v, t.y));
      x[i + 1] = __fadd_rn(__fmul_rn(v, t.x), __fmul_rn(u, t.y));
    }
  }
  if (is_q) {
    T* dst = static_cast<T*>(a.q_out) + (static_cast<size_t>(row) * a.n_head + h) * HD + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) dst[i] = from_f<T>(x[i]);
    return;
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    nan = nan || isnan(x[i]);
    x[i] = fminf(fmaxf(x[i], -kKvMax), kKvMax);
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < E; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    nan = __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), o) || nan;
  }
  const __half sh = __float2half_rn(fmaxf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), __fdiv_rn(fmaxf(-lo, hi), 127.f)));
  const float s = __half2float(sh);
  const bool some = s > 0.f && !nan;
  const float z = some ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), -127.f), 127.f) : 0.f;
  uint32_t packed = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float c = some ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)) + z, 0.f), 15.f) : 0.f;
    packed |= static_cast<uint32_t>(c) << (4 * i);
  }
  const int kh = is_v ? h - a.n_head - a.c.n_kv_head : h - a.n_head;
  uint8_t* block = static_cast<uint8_t*>(a.c.pages) + (static_cast<size_t>(page) * a.c.n_kv_head + kh) * B::kBytes +
                   (is_v ? B::kHalf : 0);
  uint8_t* codes = block + (pos % kPage) * B::kRow + lane * E / 2;
  if constexpr (E == 4)
    *reinterpret_cast<uint16_t*>(codes) = static_cast<uint16_t>(packed);
  else
    *codes = static_cast<uint8_t>(packed);
  if (lane % GL == 0) {
    const __half2 par = __halves2half2(nan ? __float2half_rn(NAN) : sh, __float2half_rn(z));
    *reinterpret_cast<__half2*>(block + kPage * B::kRow + (pos % kPage) * B::kPar + lane / GL * 4) = par;
  }
}

// One warp per (row, KV head): keys and values of the row's position.
template <int HD>
__global__ void __launch_bounds__(256) k_kv4_read(const s2_kv4 c, __half* __restrict__ k_out,
                                                  __half* __restrict__ v_out) {
  constexpr int E = HD / 32, GL = kKvGroup / E;
  using B = Kv4Block<HD>;
  const int lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int row = static_cast<int>(item / c.n_kv_head), h = static_cast<int>(item % c.n_kv_head);
  if (row >= c.n_rows) return;
  const int seq = seq_of_row(c.q_start, c.n_seq, row);
  if (seq >= c.n_seq) return;
  const int pos = c.lengths[seq] - (c.q_start[seq + 1] - row);
  int page = -1;
  if (row >= c.q_start[seq] && pos >= 0 && pos / kPage < c.table_cols)
    page = c.table[static_cast<size_t>(seq) * c.table_cols + pos / kPage];
  const bool ok = page >= 0 && page < c.n_pages;
  if (!ok && lane == 0) kv4_bad(c.status);
  const uint8_t* block = static_cast<const uint8_t*>(c.pages) +
                         (static_cast<size_t>(ok ? page : 0) * c.n_kv_head + h) * B::kBytes;
#pragma unroll
  for (int part = 0; part < 2; ++part, block += B::kHalf) {
    __half* dst = (part ? v_out : k_out) + (static_cast<size_t>(h) * c.n_rows + row) * HD + lane * E;
    float s = 0.f, z = 0.f;
    uint32_t codes = 0;
    if (ok) {
      const uint8_t* p = block + (pos % kPage) * B::kRow + lane * E / 2;
      codes = E == 4 ? *reinterpret_cast<const uint16_t*>(p) : *p;
      const __half2 par =
          *reinterpret_cast<const __half2*>(block + kPage * B::kRow + (pos % kPage) * B::kPar + lane / GL * 4);
      s = __low2float(par);
      z = __high2float(par);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) dst[i] = __float2half_rn(s * (static_cast<float>(codes >> (4 * i) & 15) - z));
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
  const long long grid = (cache->n_rows * heads + 7) / 8;
  if (n_head > 65535 || grid > 0x7fffffffll || qkv_stride < heads * cache->head_dim) return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(qkv) % 16 != 0 || qkv_stride * esz % 16 != 0 ||
      reinterpret_cast<uintptr_t>(q_out) % 16 != 0 || reinterpret_cast<uintptr_t>(rope) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(q_norm) % 16 != 0 || reinterpret_cast<uintptr_t>(k_norm) % 16 != 0)
    return S2_EINVAL;
  const AppendArgs a{*cache, qkv, qkv_stride, n_head, rope, n_pos, q_norm, k_norm, eps, q_out};
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->head_dim == 64)
      k_kv4_append<T, 64><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
    else
      k_kv4_append<T, 128><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

extern "C" int s2_kv4_read(const s2_kv4* cache, void* k, void* v, CUstream_st* stream) {
  if (kv4_bad_args(cache) || !k || !v) return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(k) % 16 != 0 || reinterpret_cast<uintptr_t>(v) % 16 != 0) return S2_EINVAL;
  const long long grid = (static_cast<long long>(cache->n_rows) * cache->n_kv_head + 7) / 8;
  if (grid > 0x7fffffffll) return S2_EINVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64)
    k_kv4_read<64><<<static_cast<unsigned>(grid), 256, 0, st>>>(*cache, static_cast<__half*>(k), static_cast<__half*>(v));
  else
    k_kv4_read<128><<<static_cast<unsigned>(grid), 256, 0, st>>>(*cache, static_cast<__half*>(k), static_cast<__half*>(v));
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
