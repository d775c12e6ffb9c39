// Rows as 8-bit integers with a scale each: the quantiser, RMSNorm with the residual's sum and the
// feed-forward's gate with such an output, and reading back.
//   step = max(max|v| / 127, 2^-126),   scale = fp32(step),   code_i = rint(v_i / step), ties (to 2^-42) to even
//   v = x                                          (quantiser)
//   v = h w / sqrt(mean(h^2) + eps), h = x + residual rounded to its type
//   v = silu(x_i) x_{f+i}, silu(g) = g / (1 + exp(-g))
// A row of codes is padded with zeros to a multiple of 16.  A row that holds, or comes to, something that
// is not finite gets scale NaN and codes 0.
//
// A code is that of the exact quotient, not of one that went through fp32: v / step is taken in fp32, and
// where that lies nearer to a border between two codes than it may be off, the code is decided by
// sums that are exact, or good to 2^-44.  So a code depends on its row alone, not on how the row was split or how
// a machine function rounds.  It costs four instructions an element, and the decision itself for one element in 2^12
// (gate) to 2^14.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

enum Op { kQuantize, kNorm, kNormResidual, kGate };

struct RowArgs {
  const void* x;
  const void* residual;
  const float* weight;
  void* total;
  int8_t* codes;
  float* scales;
  long long x_stride, residual_stride, rows;
  int cols, pitch;  // pitch: cols rounded up to 16
  float eps;
  bool vec;         // rows may be read 16 bytes at a time
};

// ------------------------------------------------------------- two-term numbers

struct Two {  // hi + lo, |lo| at most half a last place of hi
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two fast_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const Two p = two_prod(a.hi, b.hi);
  return fast_sum(p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo)));
}
// c + a, |c| >= |a|
__device__ __forceinline__ Two add(Two c, Two a) {
  const Two s = two_sum(c.hi, a.hi);
  return fast_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(c.lo, a.lo)));
}
__device__ __forceinline__ Two div(Two a, Two b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const float rest = __fadd_rn(__fmaf_rn(-q, b.hi, a.hi), __fmaf_rn(-q, b.lo, a.lo));
  return fast_sum(q, __fdiv_rn(rest, b.hi));
}

// 1 / n! and ln 2 in terms
struct Factorial {
  static constexpr double at(int n) { return n < 2 ? 1.0 : at(n - 1) * n; }
};
template <int n>
__device__ __forceinline__ Two inverse_factorial() {
  constexpr double v = 1.0 / Factorial::at(n);
  constexpr float hi = static_cast<float>(v), lo = static_cast<float>(v - hi);
  return {hi, lo};
}

// silu(g) * u to about 2^-44.  exp(-|g|) = 2^n exp(r), |r| <= ln 2 / 2, exp(r) by its Taylor series: the terms from
// r^7 on, 2^-23 of the sum, in fp32, the others in two terms.
__device__ __noinline__ Two gate_exactly(float g, float u) {
  constexpr double kLn2 = 0.693147180559945309417232121458;
  constexpr float kA = static_cast<float>(static_cast<int>(kLn2 * 32768) / 32768.0);  // 15 bits: n times it is exact
  constexpr float kB = static_cast<float>(kLn2 - kA), kC = static_cast<float>(kLn2 - kA - kB);
  const float a = fabsf(g), n = rintf(a * static_cast<float>(1.0 / kLn2));
  if (g >= 0.f && a > 60.f) return two_prod(g, u);  // 1 + exp(-g) is 1 to 2^-86
  const Two nb = two_prod(n, kB);
  // r = n ln 2 - |g|; n A - |g| is exact
  Two r = two_sum(__fsub_rn(__fmul_rn(n, kA), a), nb.hi);
  r = fast_sum(r.hi, __fadd_rn(r.lo, __fmaf_rn(n, kC, nb.lo)));
  float p = static_cast<float>(1.0 / Factorial::at(12));
  p = __fmaf_rn(p, r.hi, static_cast<float>(1.0 / Factorial::at(11)));
  p = __fmaf_rn(p, r.hi, static_cast<float>(1.0 / Factorial::at(10)));
  p = __fmaf_rn(p, r.hi, static_cast<float>(1.0 / Factorial::at(9)));
  p = __fmaf_rn(p, r.hi, static_cast<float>(1.0 / Factorial::at(8)));
  p = __fmaf_rn(p, r.hi, static_cast<float>(1.0 / Factorial::at(7)));
  Two e = add(inverse_factorial<6>(), two_prod(p, r.hi));
  e = add(inverse_factorial<5>(), mul(e, r));
  e = add(inverse_factorial<4>(), mul(e, r));
  e = add(inverse_factorial<3>(), mul(e, r));
  e = add(inverse_factorial<2>(), mul(e, r));
  e = add(Two{1.f, 0.f}, mul(e, r));
  e = add(Two{1.f, 0.f}, mul(e, r));
  const float half = -n * 0.5f, up = exp2f(floorf(half)), up2 = exp2f(-n - floorf(half));  // 2^-n, perhaps below 2^-126
  const Two small{e.hi * up * up2, e.lo * up * up2};
  const Two below = add(Two{1.f, 0.f}, small);
  Two v = two_prod(g, u);
  if (g < 0.f) v = mul(v, e);
  v = div(v, below);
  if (g < 0.f) v = {v.hi * up * up2, v.lo * up * up2};
  return v;
}

// ------------------------------------------------------------------- the rows' values

// eight elements of a row from column c on, zeros past the last
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, bool vec, float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    uint4 raw[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) raw[i] = *(reinterpret_cast<const uint4*>(row + c) + i);
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_f(row[c + i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void save8(T* row, int c, int cols, bool vec, const float (&v)[8]) {
  if (vec && c + 8 <= cols) {
    uint4 raw[sizeof(T) / 2];
    T* e = reinterpret_cast<T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f<T>(v[i]);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) *(reinterpret_cast<uint4*>(row + c) + i) = raw[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = from_f<T>(v[i]);
  }
}

template <typename T, Op kOp>
struct Row {
  const T* x;
  const T* residual;
  T* total;
  const float* weight;
  int cols;
  bool vec;
  __device__ __forceinline__ Row(const RowArgs& a, long long row)
      : x(static_cast<const T*>(a.x) + row * a.x_stride),
        residual(static_cast<const T*>(a.residual) + (kOp == kNormResidual ? row * a.residual_stride : 0)),
        total(static_cast<T*>(a.total) + (kOp == kNormResidual ? row * a.cols : 0)),
        weight(a.weight), cols(a.cols), vec(a.vec) {}

  // Values of columns c .. c + 7 (of a norm h f w g, without its row's factor), and the sum of the squares of h f.  The first
  // time the residual's sum is made and written; after that it is read, so it may have overwritten what it came from.
  template <bool kFirst>
  __device__ __forceinline__ void values(int c, float f, float g, float (&v)[8], float& squares) const {
    if constexpr (kOp == kGate) {
      float u[8];
      load8(x, c, cols, vec, v);
      load8(x + cols, c, cols, vec, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = expf(-fabsf(v[i])), s = __fdividef(v[i], 1.f + e);
        v[i] = (v[i] >= 0.f ? s : s * e) * u[i];
      }
    } else if constexpr (kOp == kQuantize) {
      load8(x, c, cols, vec, v);
    } else {
      if constexpr (kOp == kNormResidual && kFirst) {
        float d[8];
        load8(x, c, cols, vec, d);
        load8(residual, c, cols, vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(from_f<T>(v[i] + d[i]));
        save8(total, c, cols, vec, v);
      } else {
        load8(kOp == kNormResidual ? total : x, c, cols, vec, v);
      }
      float w[8];
      load8(weight, c, cols, vec, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float h = v[i] * f;
        squares = __fmaf_rn(h, h, squares);
        v[i] = __fmul_rn(h, w[i] * g);
      }
    }
  }

  // One column's value to 2^-44 or exactly, as its magnitude
  __device__ __forceinline__ Two exactly(int c, float f, float g) const {
    Two v;
    if constexpr (kOp == kGate) {
      v = gate_exactly(to_f(x[c]), to_f(x[cols + c]));
    } else if constexpr (kOp == kQuantize) {
      v = {to_f(x[c]), 0.f};
    } else {
      v = two_prod(to_f((kOp == kNormResidual ? total : x)[c]) * f, __ldg(weight + c) * g);
    }
    return v.hi < 0.f ? Two{-v.hi, -v.lo} : v;
  }
};

// Elements nearer to a border than this are decided exactly.  t = v * (127 / peak) is off by at most 127 times the
// roundings in it, 2^-24 each: two (quantiser), four (norm), sixteen (gate, where expf and the division are good to two last
// places, four of them, and exp(-|g|) enters twice): 1.5e-5, 3.1e-5, 1.22e-4.
template <Op kOp>
constexpr float kMargin = kOp == kQuantize ? 0x1p-15f : kOp == kGate ? 0x1.2p-13f : 0x1p-14f;

// The magnitude's code where t, its quotient in fp32, lies next to a border: 254 v against (2 l + 1) most.
__device__ __forceinline__ float decide(Two v, Two most, float t) {
  const float l = floorf(t), b = 2.f * l + 1.f;
  if (most.hi > 0x1p100f || most.hi < 0x1p-60f) {  // keep the products' last places within fp32's range
    const float s = most.hi > 1.f ? 0x1p-64f : 0x1p64f;
    v = {v.hi * s, v.lo * s};
    most = {most.hi * s, most.lo * s};
  }
  const Two p = two_prod(254.f, v.hi), q = two_prod(b, most.hi);
  const float d = __fadd_rn(__fsub_rn(p.hi, q.hi),
                            __fadd_rn(__fsub_rn(p.lo, q.lo), __fsub_rn(__fmul_rn(254.f, v.lo), __fmul_rn(b, most.lo))));
  // A half, to what these sums are good to: halves are met in earnest (elements of 16 bits with the gate, or the norm's
  // weight, of their row's largest), and a quotient of 24-bit numbers is 2^-31 away from one if it is none.
  if (fabsf(d) <= p.hi * 0x1p-42f) return 2.f * rintf(0.5f * (l + 0.5f));  // the even one
  return d > 0.f ? l + 1.f : l;
}

// For one-warp rows and one-block rows
template <bool kBlock>
__device__ __forceinline__ uint32_t most_of(uint32_t v, uint32_t* shared) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (kBlock) {
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
    __syncthreads();
    const int lane = threadIdx.x % 32;
    v = __reduce_max_sync(0xffffffffu, lane < static_cast<int>(blockDim.x / 32) ? shared[lane] : 0u);
  }
  return v;
}
template <bool kBlock>
__device__ __forceinline__ float sum_of(float v, float* shared) {  // in a fixed order
  v = warp_sum(v);
  if constexpr (kBlock) {
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
    __syncthreads();
    const int lane = threadIdx.x % 32;
    v = warp_sum(lane < static_cast<int>(blockDim.x / 32) ? shared[lane] : 0.f);
  }
  return v;
}
// hi + lo in the order of their sizes (hi >= 0)
__device__ __forceinline__ unsigned long long ordered(Two v) {
  const uint32_t l = __float_as_uint(v.lo);
  return static_cast<unsigned long long>(__float_as_uint(v.hi)) << 32 | (l & 0x80000000u ? ~l : l | 0x80000000u);
}
__device__ __forceinline__ Two from_ordered(unsigned long long k) {
  const uint32_t l = static_cast<uint32_t>(k);
  return {__uint_as_float(static_cast<uint32_t>(k >> 32)), __uint_as_float(l & 0x80000000u ? l & 0x7fffffffu : ~l)};
}

// A row is a warp's (up to kHeld * 256 columns) or a block's.  A thread holds kHeld times eight elements; what lies
// past them is computed again for its codes.
template <typename T, Op kOp, int kHeld, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) k_q8_rows(const RowArgs a) {
  __shared__ uint32_t shared_most[32];
  __shared__ float shared_sum[32];
  __shared__ unsigned long long shared_exact[kBlock ? 1 : 8];
  constexpr bool kNorms = kOp == kNorm || kOp == kNormResidual;
  const int team = kBlock ? blockDim.x : 32, me = kBlock ? threadIdx.x : threadIdx.x % 32;
  const long long row = kBlock ? blockIdx.x : static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (!kBlock && row >= a.rows) return;
  unsigned long long* exact = shared_exact + (kBlock ? 0 : threadIdx.x / 32);
  if (me == 0) *exact = 0;
  if constexpr (!kBlock) __syncwarp();
  const Row<T, kOp> in(a, row);

  float held[kHeld][8];
  float f = 1.f, g = 1.f, squares = 0.f;
  uint32_t top = 0;  // bits of the largest magnitude; infinities and NaN are the largest
  auto look = [&](const float(&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int c = (h * team + me) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) held[h][i] = 0.f;
    if (c < a.cols) in.template values<true>(c, f, g, held[h], squares);
    look(held[h]);
  }
  for (int c = (kHeld * team + me) * 8; c < a.cols; c += team * 8) {
    float v[8];
    in.template values<true>(c, f, g, v, squares);
    look(v);
  }
  top = most_of<kBlock>(top, shared_most);
  float r = 1.f;
  if constexpr (kNorms) {
    float sum = sum_of<kBlock>(squares, shared_sum);
    if (top == 0x7f800000u || isinf(sum)) {  // perhaps only past fp32's range: once more with what is too large times 2^-80
      if (isinf(sum)) f = 0x1p-80f;
      if (top == 0x7f800000u) g = 0x1p-80f;
      squares = 0.f, top = 0;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int c = (h * team + me) * 8;
        if (c < a.cols) in.template values<false>(c, f, g, held[h], squares);
        look(held[h]);
      }
      for (int c = (kHeld * team + me) * 8; c < a.cols; c += team * 8) {
        float v[8];
        in.template values<false>(c, f, g, v, squares);
        look(v);
      }
      if constexpr (kBlock) __syncthreads();
      top = most_of<kBlock>(top, shared_most);
      sum = sum_of<kBlock>(squares, shared_sum);
    }
    // 1 / f times the row's factor
    r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(a.cols)), a.eps * f * f)));
  }
  const float most = __uint_as_float(top);
  const float largest = most * r * (g == 1.f ? 1.f : 0x1p80f);
  int8_t* codes = a.codes + row * a.pitch;
  if (!(largest <= 3.4028234663852886e38f)) {  // not finite
    for (int c = me * 8; c < a.pitch; c += team * 8) *reinterpret_cast<uint2*>(codes + c) = make_uint2(0, 0);
    if (me == 0) a.scales[row] = __uint_as_float(0x7fc00000u);
    return;
  }
  float step = fminf(__fdiv_rn(largest, 127.f), 0x1.020406p+121f);  // what 127 times is finite
  const bool tiny = step < 0x1p-126f;  // the quotient is v 2^126 then
  if (tiny) step = 0x1p-126f;
  if (me == 0) a.scales[row] = step;

  // the largest magnitude to more than fp32
  Two peak{most, 0.f};
  if constexpr (kOp != kQuantize) {
    if (!tiny) {
      const float near = most * (1.f - 0x1p-18f);
      auto candidates = [&](const float(&v)[8], int c) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          float one = v[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) one = i == j ? v[j] : one;
          if (fabsf(one) >= near) atomicMax(exact, ordered(in.exactly(c + i, f, g)));
        }
      };
      auto any = [&](const float(&v)[8]) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
        return m >= near;
      };
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (any(held[h])) candidates(held[h], (h * team + me) * 8);
      for (int c = (kHeld * team + me) * 8; c < a.cols; c += team * 8) {
        float v[8], unused = 0.f;
        in.template values<false>(c, f, g, v, unused);
        if (any(v)) candidates(v, c);
      }
    }
    if constexpr (kBlock)
      __syncthreads();
    else
      __syncwarp();
    if (!tiny) peak = from_ordered(*reinterpret_cast<volatile unsigned long long*>(exact));
  }

  const float inverse = tiny ? 0x1p126f : __fdiv_rn(127.f, peak.hi);
  auto encode = [&](const float(&v)[8], int c) {
    if (c >= a.pitch) return;
    float t[8], k[8];
    uint32_t near = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = kNorms && tiny ? v[i] * r * inverse : v[i] * inverse;
      k[i] = rintf(t[i]);
      near |= (fabsf(t[i] - k[i]) > 0.5f - kMargin<kOp> ? 1u : 0u) << i;
    }
    if (near && !tiny) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        if (!(near >> i & 1)) continue;
        float one = t[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) one = i == j ? t[j] : one;
        const float code = copysignf(decide(in.exactly(c + i, f, g), peak, fabsf(one)), one);
#pragma unroll
        for (int j = 0; j < 8; ++j) k[j] = i == j ? code : k[j];
      }
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i / 4] |= (static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(k[i], -127.f), 127.f))) & 255u) << (i % 4 * 8);
    *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h) encode(held[h], (h * team + me) * 8);
  for (int c = (kHeld * team + me) * 8; c < a.pitch; c += team * 8) {
    float v[8], unused = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (c < a.cols) in.template values<false>(c, f, g, v, unused);
    encode(v, c);
  }
}

// Rows of up to 1024 columns by a warp each, longer ones by a block whose threads hold 16 elements.
template <Op kOp>
int launch_rows(const RowArgs& a, int dtype, cudaStream_t st) {
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (a.cols <= 1024) {
      k_q8_rows<T, kOp, 4, false><<<static_cast<unsigned>((a.rows + 7) / 8), 256, 0, st>>>(a);
    } else {
      const int threads = min(1024, (a.pitch / 8 + 63) / 64 * 32);
      k_q8_rows<T, kOp, 2, true><<<static_cast<unsigned>(a.rows), threads, 0, st>>>(a);
    }
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

// A thread reads 16 codes.
template <typename T>
__global__ void __launch_bounds__(256) k_q8_read(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                 long long items, int per, int cols, bool vec, T* __restrict__ out) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= items) return;
  const long long row = i / per;
  const int c = static_cast<int>(i - row * per) * 16;
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(codes) + i);
  const float s = __ldg(scales + row);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = s * static_cast<float>(static_cast<int8_t>(w[2 * h + e / 4] >> (e % 4 * 8)));
    if (c + 8 * h < cols) save8(out + row * cols, c + 8 * h, cols, vec, v);
  }
}

constexpr int kColsMost = 1 << 24;

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool bad_rows(const void* x, int dtype, long long stride, long long rows, long long width, int cols, const void* codes,
              const void* scales) {
  const int esz = dtype_bytes(dtype);
  return !x || !esz || !codes || !scales || rows < 1 || rows > 0x7fffffffll || cols < 1 || cols > kColsMost ||
         stride < width || !aligned(x, esz) || !aligned(codes, 16) || !aligned(scales, 4);
}
bool wide(const void* p, long long stride, int esz) { return aligned(p, 16) && stride * esz % 16 == 0; }
int pitch_of(int cols) { return (cols + 15) / 16 * 16; }

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_quantize_q8(const void* x, int dtype, long long x_stride, long long rows, int cols, int8_t* codes,
                              float* scales, CUstream_st* stream) {
  if (bad_rows(x, dtype, x_stride, rows, cols, cols, codes, scales)) return S2_EINVAL;
  const int esz = dtype_bytes(dtype);
  const RowArgs a{x, nullptr, nullptr, nullptr, codes, scales, x_stride, 0, rows, cols, pitch_of(cols), 0.f,
                  wide(x, x_stride, esz)};
  return launch_rows<kQuantize>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int s2_rms_norm_q8(const void* x, int dtype, long long x_stride, const void* residual,
                              long long residual_stride, const float* weight, float eps, long long rows, int cols,
                              void* total, int8_t* codes, float* scales, CUstream_st* stream) {
  if (bad_rows(x, dtype, x_stride, rows, cols, cols, codes, scales) || !weight || !aligned(weight, 4) ||
      !(eps >= 0.f) || !std::isfinite(eps))
    return S2_EINVAL;
  const int esz = dtype_bytes(dtype);
  if ((residual != nullptr) != (total != nullptr) ||
      (residual && (residual_stride < cols || !aligned(residual, esz) || !aligned(total, esz))))
    return S2_EINVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  RowArgs a{x, residual, weight, total, codes, scales, x_stride, residual_stride, rows, cols, pitch_of(cols), eps,
            wide(x, x_stride, esz) && aligned(weight, 16)};
  if (!residual) return launch_rows<kNorm>(a, dtype, st);
  a.vec = a.vec && wide(residual, residual_stride, esz) && wide(total, cols, esz);
  return launch_rows<kNormResidual>(a, dtype, st);
}

extern "C" int s2_swiglu_q8(const void* x, int dtype, long long x_stride, long long rows, int cols, int8_t* codes,
                            float* scales, CUstream_st* stream) {
  if (bad_rows(x, dtype, x_stride, rows, 2ll * cols, cols, codes, scales)) return S2_EINVAL;
  const int esz = dtype_bytes(dtype);
  const RowArgs a{x, nullptr, nullptr, nullptr, codes, scales, x_stride, 0, rows, cols, pitch_of(cols), 0.f,
                  wide(x, x_stride, esz) && static_cast<long long>(cols) * esz % 16 == 0};
  return launch_rows<kGate>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int s2_dequantize_q8(const int8_t* codes, const float* scales, long long rows, int cols, void* out, int dtype,
                                CUstream_st* stream) {
  if (bad_rows(out, dtype, cols, rows, cols, cols, codes, scales)) return S2_EINVAL;
  const int per = pitch_of(cols) / 16;
  const long long items = rows * per, grid = (items + 255) / 256;
  if (grid > 0x7fffffffll) return S2_EINVAL;
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    k_q8_read<T><<<static_cast<unsigned>(grid), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        codes, scales, items, per, cols, wide(out, cols, sizeof(T)), static_cast<T*>(out));
  });
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}
