// Attention over the paged 4-bit cache (see kv4.cuh for the layout).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "kv4.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

struct AttnArgs {
  s2_kv4 c;
  const void* q;
  int n_head;
  float scale;
  void* out;
};

template <int HD>
__device__ __forceinline__ void kv4_lane(const uint8_t* half_block, int slot, int lane, float (&x)[HD / 32]) {
  constexpr int E = HD / 32, GL = kKvGroup / E;
  using B = Kv4Block<HD>;
  const uint8_t* p = half_block + slot * B::kRow + lane * E / 2;
  const uint32_t codes = E == 4 ? *reinterpret_cast<const uint16_t*>(p) : *p;
  const __half2 par = *reinterpret_cast<const __half2*>(half_block + kPage * B::kRow + slot * B::kPar + lane / GL * 4);
#pragma unroll
  for (int i = 0; i < E; ++i)
    x[i] = round_f16(__low2float(par) * (static_cast<float>(codes >> (4 * i) & 15) - __high2float(par)));
}

// One warp per (row, query head), one position at a time with the running maximum and sum.
template <typename T, int HD>
__global__ void __launch_bounds__(256) k_kv4_attention(const AttnArgs a) {
  constexpr int E = HD / 32;
  using B = Kv4Block<HD>;
  const int lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int row = static_cast<int>(item / a.n_head), h = static_cast<int>(item % a.n_head);
  if (row >= a.c.n_rows) return;
  const int seq = seq_of_row(a.c.q_start, a.c.n_seq, row);
  if (seq >= a.c.n_seq || row < a.c.q_start[seq]) return;
  int seen = a.c.lengths[seq] - (a.c.q_start[seq + 1] - row) + 1;
  if (seen > static_cast<long long>(a.c.table_cols) * kPage) {
    if (lane == 0) kv4_bad(a.c.status);
    seen = a.c.table_cols * kPage;
  }
  const size_t at = (static_cast<size_t>(row) * a.n_head + h) * HD + lane * E;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) q[i] = to_f(static_cast<const T*>(a.q)[at + i]) * a.scale;
  const int kh = h / (a.n_head / a.c.n_kv_head);
  for (int t = 0; t < seen; ++t) {
    const int page = a.c.table[static_cast<size_t>(seq) * a.c.table_cols + t / kPage];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) kv4_bad(a.c.status);
      continue;
    }
    const uint8_t* block = static_cast<const uint8_t*>(a.c.pages) +
                           (static_cast<size_t>(page) * a.c.n_kv_head + kh) * B::kBytes;
    float x[E], s = 0.f;
    kv4_lane<HD>(block, t % kPage, lane, x);
#pragma unroll
    for (int i = 0; i < E; ++i) s += q[i] * x[i];
    s = warp_sum(s);
    const float mn = fmaxf(m, s), keep = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * keep + p;
    kv4_lane<HD>(block + B::kHalf, t % kPage, lane, x);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * keep + p * x[i];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) static_cast<T*>(a.out)[at + i] = from_f<T>(l > 0.f ? o[i] / l : l);
}

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" size_t s2_kv4_attention_workspace(int n_seq, int n_rows, int n_head, int n_kv_head, int head_dim,
                                             int max_len) {
  (void)n_seq, (void)n_rows, (void)n_head, (void)n_kv_head, (void)head_dim, (void)max_len;
  return 0;
}

extern "C" int s2_kv4_attention(const s2_kv4* cache, const void* q, int dtype, int n_head, float scale, int max_len,
                                void* out, void* workspace, size_t ws_bytes, CUstream_st* stream) {
  const int esz = dtype_bytes(dtype);
  if (kv4_bad_args(cache) || !q || !out || !esz || n_head < 1 || n_head > 65535 ||
      n_head % cache->n_kv_head != 0 || !std::isfinite(scale) || max_len < 0)
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(q) % 16 != 0 || reinterpret_cast<uintptr_t>(out) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return S2_EINVAL;
  (void)ws_bytes;
  const long long grid = (static_cast<long long>(cache->n_rows) * n_head + 7) / 8;
  if (grid > 0x7fffffffll) return S2_EINVAL;
  const AttnArgs a{*cache, q, n_head, scale, out};
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (cache->head_dim == 64)
      k_kv4_attention<T, 64><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
    else
      k_kv4_attention<T, 128><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
