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

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "convert.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "s2_internal.h"
#include "tc05.cuh"

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
  float eps, per_col;  // per_col: 1 / cols
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

// x = m 2^e, 1 <= |m| < 2
struct Split {
  float m;
  int e;
};
__device__ __forceinline__ Split split(float x) {
  const bool small = fabsf(x) < 0x1p-126f;
  const uint32_t b = __float_as_uint(small ? x * 0x1p64f : x);
  return {__uint_as_float((b & 0x807fffffu) | 0x3f800000u), static_cast<int>(b >> 23 & 255u) - (small ? 191 : 127)};
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126..127
// v 2^e, kept within what can be compared with numbers of about 1
__device__ __forceinline__ Two scaled(Two v, int e) {
  const float s = power_of_two(min(max(e, -100), 100));
  return {v.hi * s, v.lo * s};
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

// silu(g) * u * 2^unit to about 2^-44, from the factors' significands: neither g u, which passes fp32's range where silu(g) u does
// not, nor the last places of a small product are lost.  exp(-|g|) = 2^-n exp(r), |r| <= ln 2 / 2, exp(r) by its Taylor series:
// the terms from r^7 on, 2^-23 of the sum, in fp32, the others in two terms.
__device__ __noinline__ Two gate_exactly(float g, float u, int unit) {
  constexpr double kLn2 = 0.693147180559945309417232121458;
  constexpr float kA = static_cast<float>(static_cast<int>(kLn2 * 32768) / 32768.0);  // 15 bits: n times it is exact
  constexpr float kB = static_cast<float>(kLn2 - kA), kC = static_cast<float>(kLn2 - kA - kB);
  const float a = fabsf(g), n = rintf(a * static_cast<float>(1.0 / kLn2));
  const Split gs = split(g), us = split(u);
  unit += gs.e + us.e;
  if (g >= 0.f && a > 60.f) return scaled(two_prod(gs.m, us.m), unit);  // 1 + exp(-g) is 1 to 2^-86
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
  const int down = -static_cast<int>(fminf(n, 200.f));
  const Two below = add(Two{1.f, 0.f}, scaled(e, down));
  Two v = two_prod(gs.m, us.m);
  if (g < 0.f) v = mul(v, e);
  return scaled(div(v, below), unit + (g < 0.f ? down : 0));
}

// ------------------------------------------------------------------- the rows' values

// kKeep: through L1, for elements that are read once more.
template <bool kKeep, typename U>
__device__ __forceinline__ U get_from(const U* p) {
  if constexpr (kKeep)
    return *p;
  else
    return __ldcg(p);
}

// eight elements as they lie in memory
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
  // Of columns c .. c + 7 of a row, zeros past the last.  Rows start anywhere: the aligned 16-byte blocks around an eight are
  // loaded and shifted by `skew`, the bytes of the row's start past a block's (the same for all eights of a row).  The row's first
  // and last eights, whose blocks may reach out of it, are loaded by elements.  (By elements alone: 20000 x 700 bf16 gate 60 us.)
  template <bool kKeep>
  __device__ __forceinline__ void load(const T* row, int c, int cols, int skew) {
    const uint4* block = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(row + c) - skew);
    if (skew == 0 && c + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = get_from<kKeep>(block + i);
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    } else if (c > 0 && c + 16 <= cols) {
      uint32_t b[kWords + 4];
#pragma unroll
      for (int i = 0; i <= kWords / 4; ++i) {
        const uint4 u = get_from<kKeep>(block + i);
        b[4 * i] = u.x, b[4 * i + 1] = u.y, b[4 * i + 2] = u.z, b[4 * i + 3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < kWords + 3; ++i) b[i] = skew & 4 ? b[i + 1] : b[i];
#pragma unroll
      for (int i = 0; i < kWords + 1; ++i) b[i] = skew & 8 ? b[i + 2] : b[i];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? b[i] : __funnelshift_r(b[i], b[i + 1], skew % 4 * 8);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = c + i < cols ? __float_as_uint(get_from<kKeep>(reinterpret_cast<const float*>(row) + c + i)) : 0u;
    } else {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 2 * i < cols ? get_from<kKeep>(e + c + 2 * i) : 0u, hi = c + 2 * i + 1 < cols ? get_from<kKeep>(e + c + 2 * i + 1) : 0u;
        w[i] = lo | hi << 16;
      }
    }
  }
  __device__ static __forceinline__ int skew_of(const T* row) { return static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15); }
  // in pieces of 16, 4 or 2 bytes
  __device__ __forceinline__ void store(T* row, int c, int cols, int skew) const {
    if (skew == 0 && c + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(row + c)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if (skew % 4 == 0 && c + 8 <= cols) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(row + c)[i] = w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= cols) break;
        if constexpr (sizeof(T) == 4)
          row[c + i] = __uint_as_float(w[i]);
        else
          reinterpret_cast<uint16_t*>(row)[c + i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
        v[i] = i % 2 ? f.y : f.x;
      } else {
        v[i] = i % 2 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {  // rounded to T
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
        }
      }
    }
  }
};

// silu(g) u = (u / (1 + e)) g, times e for negative g, e = exp(-|g|) = 2^(-|g| log2 e) with the product's rounding taken back.  Off by
// up to: e, four last places' halves from ex2 and 1.5 more; the sum one, its reciprocal two, three products.  An e below 2^-126
// (g beyond 87.3) is zero.  The product with log2 e is rounded towards zero, which of gates past 2.36e38 leaves fp32's largest
// number instead of an infinity, whose rounding is not a number (|g| taken as 128 at most: 2048 x 9728 bf16 30.0 us, so 29.7).
// The gate comes last: u g may pass fp32's range where the value does not, silu(g) of a small g lose places below it that a large u brings
// back; u sigmoid(g) loses at most 88 2^-150 of the value, 2^-17 of the least step.
// (expf and __fdividef: 12 instructions more, 33.0 us against 29.8 for 2048 x 9728 bf16.)
__device__ __forceinline__ float gate_fast(float g, float u) {
  constexpr double kLog2 = 1.44269504088896340735992468100;
  constexpr float kHi = static_cast<float>(kLog2), kLo = static_cast<float>(kLog2 - kHi), kLn2 = 0.69314718f;
  const float a = -fabsf(g), y = __fmul_rz(a, kHi), rest = __fmaf_rn(a, kLo, __fmaf_rn(a, kHi, -y));
  float e, d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  e = __fmaf_rn(e, __fmul_rn(rest, kLn2), e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(1.f + e));
  return __fmul_rn(__fmul_rn(u, __fmul_rn(d, g >= 0.f ? 1.f : e)), g);
}

// maximum of which a NaN is one
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T, Op kOp>
struct Row {
  static constexpr bool kTwo = kOp == kGate || kOp == kNormResidual, kNorms = kOp == kNorm || kOp == kNormResidual;
  // Elements next to a border are read again, after a residual's sum from where it was written.  (2048 x 9728 gate through L1 29.4 us,
  // past it 30.7; 5916 x 2560 fp32 norm with a residual 37.5 and 33.8.)
  static constexpr bool kKeep = kOp != kNormResidual;
  const T* x;
  const T* other;  // the residual, or the gate's second half
  T* total;
  const float* weight;
  int cols, skew, other_skew, total_skew, weight_skew;
  __device__ __forceinline__ Row(const RowArgs& a, long long row)
      : x(static_cast<const T*>(a.x) + row * a.x_stride),
        other(kOp == kGate ? x + a.cols : static_cast<const T*>(a.residual) + (kTwo ? row * a.residual_stride : 0)),
        total(static_cast<T*>(a.total) + (kOp == kNormResidual ? row * a.cols : 0)),
        weight(a.weight), cols(a.cols), skew(Eight<T>::skew_of(x)), other_skew(Eight<T>::skew_of(other)),
        total_skew(Eight<T>::skew_of(total)), weight_skew(Eight<float>::skew_of(weight)) {}

  // What eight values are made of: loaded first, for all that a thread holds.
  struct In {
    Eight<T> x;
    std::conditional_t<kTwo, Eight<T>, uint32_t> other;
    std::conditional_t<kNorms, Eight<float>, uint32_t> weight;
  };
  __device__ __forceinline__ void load(int c, In& in) const {
    in.x.template load<kKeep>(x, c, cols, skew);
    if constexpr (kTwo) in.other.template load<kKeep>(other, c, cols, other_skew);
    if constexpr (kNorms) in.weight.template load<true>(weight, c, cols, weight_skew);
  }
  // Values of columns c .. c + 7 (of a norm h w, without its row's factor), and the sum of the squares of h.  The residual's
  // sum is written, and read from there when values are made again: it may have overwritten what it came from.
  __device__ __forceinline__ void values(int c, In& in, float (&v)[8], float& squares) const {
    in.x.get(v);
    if constexpr (kOp == kGate) {
      float u[8];
      in.other.get(u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = gate_fast(v[i], u[i]);
    }
    if constexpr (kOp == kNormResidual) {
      float r[8];
      in.other.get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
      in.x.set(v);
      in.x.store(total, c, cols, total_skew);
      in.x.get(v);
    }
    if constexpr (kNorms) {
      float w[8];
      in.weight.get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        squares = __fmaf_rn(v[i], v[i], squares);
        v[i] = __fmul_rn(v[i], w[i]);
      }
    }
  }
  // A norm's h and weights of columns c .. c + 7, once more
  __device__ __forceinline__ void operands(int c, float (&h)[8], float (&w)[8]) const {
    Eight<T> hs;
    Eight<float> ws;
    if constexpr (kOp == kNormResidual)
      hs.template load<false>(total, c, cols, total_skew);
    else
      hs.template load<kKeep>(x, c, cols, skew);
    ws.template load<true>(weight, c, cols, weight_skew);
    hs.get(h);
    ws.get(w);
  }
  // Values once more
  __device__ __forceinline__ void again(int c, float (&v)[8]) const {
    if constexpr (kNorms) {
      float w[8];
      operands(c, v, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], w[i]);
    } else {
      In in;
      float unused;
      load(c, in);
      values(c, in, v, unused);
    }
  }

  // One column's value (of a norm h w) times 2^unit, to 2^-44 or exactly
  __device__ __forceinline__ Two exactly(int c, int unit) const {
    if constexpr (kOp == kGate) {
      return gate_exactly(to_f(x[c]), to_f(other[c]), unit);
    } else if constexpr (kOp == kQuantize) {
      return {to_f(x[c]) * power_of_two(unit), 0.f};
    } else {
      const Split h = split(to_f((kOp == kNormResidual ? total : x)[c])), w = split(weight[c]);
      return scaled(two_prod(h.m, w.m), h.e + w.e + unit);
    }
  }
};

__device__ __forceinline__ Two magnitude(Two v) { return v.hi < 0.f ? Two{-v.hi, -v.lo} : v; }

// Elements nearer to a border than this are decided exactly.  v * (127 / most) is off by at most 127 times the roundings in
// v, most and their quotient, 2^-24 each: one (quantiser; 7.6e-6), three (norm; 2.3e-5), and twelve each in v and most (gate;
// 1.9e-4) or, where most is known better, fourteen (1.06e-4).
template <Op kOp, bool kPeakFirst>
constexpr float kMargin = kOp == kQuantize ? 0x1p-16f : kOp == kGate ? (kPeakFirst ? 0x1p-13f : 0x1p-12f) : 0x1p-15f;

// The magnitude's code where v per, its quotient in fp32, lies next to a border: 254 v against (2 l + 1) most.
__device__ __forceinline__ float decide(Two v, Two most, float per) {
  const float l = floorf(v.hi * per), b = 2.f * l + 1.f;
  const Two p = two_prod(254.f, v.hi), q = two_prod(b, most.hi);
  const float d = __fadd_rn(__fsub_rn(p.hi, q.hi),
                            __fadd_rn(__fsub_rn(p.lo, q.lo), __fsub_rn(__fmul_rn(254.f, v.lo), __fmul_rn(b, most.lo))));
  // A half, to what these sums are good to: halves are met in earnest (elements of 16 bits with the gate, or the norm's
  // weight, of their row's largest), and a quotient of 24-bit numbers is 2^-31 away from one if it is none.
  if (fabsf(d) <= p.hi * 0x1p-42f) return 2.f * rintf(0.5f * (l + 0.5f));  // the even one
  return d > 0.f ? l + 1.f : l;
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

// A row is a team's: 8 or 32 lanes of a warp, or a block.  Reductions are in a fixed order.
template <int kTeam>  // 0: the block
struct Team {
  __device__ static __forceinline__ unsigned mask() {
    return kTeam == 8 ? 0xffu << (threadIdx.x & 24u) : 0xffffffffu;
  }
  // the largest of a magnitude (infinities and NaN are the largest) and the sum of s
  template <bool kSum>
  __device__ static __forceinline__ void reduce(float& most, float& s, float2* shared) {
    constexpr int kLanes = kTeam == 8 ? 8 : 32;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      if constexpr (kTeam == 8) most = max_nan(most, __shfl_xor_sync(mask(), most, o));
      if constexpr (kSum) s += __shfl_xor_sync(mask(), s, o);
    }
    if constexpr (kTeam != 8) most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if constexpr (kTeam == 0) {
      const int lane = threadIdx.x % 32;
      if (lane == 0) shared[threadIdx.x / 32] = make_float2(most, s);
      __syncthreads();
      const float2 t = lane < static_cast<int>(blockDim.x / 32) ? shared[lane] : make_float2(0.f, 0.f);
      most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t.x)));
      if constexpr (kSum) s = warp_sum(t.y);
    }
  }
  // of a block in *shared, which was zero
  __device__ static __forceinline__ unsigned long long largest(unsigned long long key, unsigned long long* shared) {
    if constexpr (kTeam == 0) {
      if (key) atomicMax(shared, key);
      __syncthreads();
      key = *reinterpret_cast<volatile unsigned long long*>(shared);
    } else {
#pragma unroll
      for (int o = kTeam / 2; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(mask(), key, o));
    }
    return key;
  }
};

constexpr float kMost = 3.4028234663852886e38f;
// at most what 127 times is finite
__device__ __forceinline__ float scale_of(float largest) { return fminf(fmaxf(__fdiv_rn(largest, 127.f), 0x1p-126f), 0x1.020406p+121f); }

// A norm's row whose squares or products leave fp32's range, or the places that it has near its lower end: h is taken times 2^h_up, h w
// times 2^product_up, which bring the largest to 1 .. 4, from their significands and exponents.  Sums are in the order of k_q8_rows.
// Such rows are rare, so nothing is held; they have a function of their own, and it takes its columns one by one, so that the others
// keep their registers (as a second round of k_q8_rows itself: norm of 5916 x 2560 with a residual, bf16 26.2 us, so 24.1; fp32 42.8
// and 34.5; by eights 26.3 and 38.2.  Of such rows alone bf16 103, by eights 91).
template <typename T, Op kOp, int kTeam>
__device__ __noinline__ void norm_by_exponents(const RowArgs a, long long row, float2* shared, float2* shared_too,
                                               unsigned long long* exact) {
  using R = Row<T, kOp>;
  const R in(a, row);
  const int team = kTeam == 0 ? blockDim.x : kTeam, me = kTeam == 0 ? threadIdx.x : threadIdx.x % kTeam;
  int8_t* codes = a.codes + row * a.pitch;
  constexpr int kZero = 400;  // all exponents are above -400
  const T* const from = kOp == kNormResidual ? in.total : in.x;
  auto each = [&](auto f) {  // of this thread's columns
#pragma unroll 1
    for (int c = me * 8; c < a.cols; c += team * 8)
#pragma unroll 1
      for (int i = c; i < min(c + 8, a.cols); ++i) f(to_f(from[i]), a.weight[i]);
  };
  float h_most = 0.f, product_most = 0.f, unused = 0.f;
  each([&](float h, float w) {
    const int e = split(h).e + kZero, p = split(w).e + e;
    if (h != 0.f) h_most = fmaxf(h_most, static_cast<float>(e));
    if (h != 0.f && w != 0.f) product_most = fmaxf(product_most, static_cast<float>(p));
  });
  Team<kTeam>::template reduce<false>(h_most, unused, shared_too);
  Team<kTeam>::template reduce<false>(product_most, unused, shared);
  int h_up = h_most > 0.f ? kZero - static_cast<int>(h_most) : 0;
  if (a.eps > 0.f) h_up = min(h_up, -(split(a.eps).e >> 1));  // beside eps, what is lower than half of its exponent does not count
  const int product_up = kZero - static_cast<int>(product_most), back = h_up - product_up;
  auto product = [&](float h, float w) {
    const Split p = split(h), q = split(w);
    return h == 0.f || w == 0.f ? Two{0.f, 0.f} : scaled(two_prod(p.m, q.m), p.e + q.e + product_up);
  };
  float squares = 0.f, most = 0.f;
  unsigned long long key = 0;
  each([&](float h, float w) {
    const Split p = split(h);
    const float t = h == 0.f ? 0.f : p.m * power_of_two(min(max(p.e + h_up, -126), 1));
    squares = __fmaf_rn(t, t, squares);
    key = max(key, ordered(magnitude(product(h, w))));
    most += __fadd_rn(__fsub_rn(h, h), __fsub_rn(w, w));  // not a number where one of them is not finite
  });
  most = fabsf(most + __uint_as_float(static_cast<uint32_t>(key >> 32)));
  Team<kTeam>::template reduce<true>(most, squares, shared_too);
  const float r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(squares, static_cast<float>(a.cols)), ldexpf(a.eps, 2 * h_up))));
  const float largest = ldexpf(most * r, back);
  const bool finite = largest <= kMost;
  if (me == 0) a.scales[row] = finite ? scale_of(largest) : __uint_as_float(0x7fc00000u);
  if (!finite || most == 0.f) {
    for (int c = me * 8; c < a.pitch; c += team * 8) *reinterpret_cast<uint2*>(codes + c) = make_uint2(0, 0);
    return;
  }
  const bool tiny = largest < 127 * 0x1p-126f;
  const Two peak = from_ordered(Team<kTeam>::largest(key, exact));
  const float per = tiny ? r * power_of_two(max(126 + back, -126)) : __fdiv_rn(127.f, peak.hi);
#pragma unroll 1
  for (int c = me * 8; c < a.pitch; c += team * 8) {
    unsigned long long word = 0;
#pragma unroll 1
    for (int i = c; i < min(c + 8, a.cols); ++i) {
      const Two v = product(to_f(from[i]), a.weight[i]);
      const float t = fabsf(v.hi * per);
      float k = rintf(t);
      if (!tiny && fabsf(t - k) > 0.5f - kMargin<kOp, false>) k = decide(magnitude(v), peak, per);
      word |= static_cast<unsigned long long>(static_cast<uint8_t>(static_cast<int>(copysignf(k, v.hi)))) << 8 * (i - c);
    }
    *reinterpret_cast<unsigned long long*>(codes + c) = word;
  }
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, it rounds to a whole number, which the sum's low bits then hold

// One pass over memory: a row's threads hold its values while they agree on the largest (and a norm's sum of squares), and then
// encode them.  A thread holds kHeld times eight elements; what lies past them is made again for its codes.
// Quantised and normed rows of fp32 run near the copy's rate.  Others are bound by latency that nothing hides: a row's loads, meetings and
// codes do not overlap with another's in its block, and 40 to 49 % of the warps that an SM holds are there.  (Profiled: 16 warp
// instructions for 32 values of the quantiser, 39 of a norm with a residual, 33 of the gate, that is 20, 15 and 17 us of issue slots, of
// which 60 to 70 % are taken; 22, 16 and 15 us of bytes; no pipe is full.)  Measured, operands not in L2 (GB300, copies run at
// 6.7 TB/s): quantising 19456 x 2560 bf16 33.4 us (4.5 TB/s), 9728 x 2560 fp32 19.6 (6.4); norm with a residual of 5916 x 2560 bf16 24.2
// (4.4), fp32 34.5 (5.7); gate of 2048 x 9728 bf16 29.7 (3.4), 1024 x 9728 fp32 21.6 (4.1); one row of 2560 2.4, of 9728 4.3.
template <typename T, Op kOp, int kHeld, int kTeam, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) k_q8_rows(const RowArgs a) {
  __shared__ float2 shared[2][kTeam == 0 ? 32 : 1];
  __shared__ unsigned long long exact;
  using R = Row<T, kOp>;
  constexpr bool kNorms = R::kNorms;
  // Whether the largest magnitude is made exact before any code: a gate's long row has an element next to a border more often
  // than not, others have none.
  constexpr bool kPeakFirst = kTeam == 0 && kOp == kGate;
  pdl_trigger();
  pdl_wait();
  const int team = kTeam == 0 ? blockDim.x : kTeam, me = kTeam == 0 ? threadIdx.x : threadIdx.x % kTeam;
  const long long row = kTeam == 0 ? blockIdx.x : (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kTeam;
  if (kTeam != 0 && row >= a.rows) return;
  if (kTeam == 0 && me == 0) exact = 0;
  const R in(a, row);
  auto column = [&](int h) { return (h * team + me) * 8; };
  float held[kHeld][8];
  float squares = 0.f, most = 0.f;
  auto look = [&](const float(&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max_nan(most, fabsf(v[i]));
  };
  {
    typename R::In raw[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (column(h) < a.cols) in.load(column(h), raw[h]);
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) held[h][i] = 0.f;
      if (column(h) < a.cols) {
        in.values(column(h), raw[h], held[h], squares);
        look(held[h]);
      }
    }
  }
#pragma unroll 1
  for (int c = column(kHeld); c < a.cols; c += team * 8) {
    float v[8];
    typename R::In raw;
    in.load(c, raw);
    in.values(c, raw, v, squares);
    look(v);
  }
  float mine = most;
  Team<kTeam>::template reduce<kNorms>(most, squares, shared[0]);
  float r = 1.f;  // of a norm the row's factor, to a few last places
  if constexpr (kNorms) {
    // Sums and products in fp32 are good while nothing that counts leaves its range: squares past it, or so small that what falls below
    // it counts beside eps; products past it, or so small that codes would not have fp32's places.  (Where the step is its least, products
    // are off by up to 2^-24 r of it; rows of zeros are such, and any product that is 0 here is one of them while r is up to 2^22.)
    const float mean = __fmaf_rn(squares, a.per_col, a.eps);
    r = rsqrtf(mean);
    const bool small = most < 0x1p-110f && (r > (most == 0.f ? 0x1p22f : 0x1p10f) || most * r >= 0x1p-120f);
    if (isinf(most) || isinf(squares) || mean < 0x1p-100f || small) {
      norm_by_exponents<T, kOp, kTeam>(a, row, shared[0], shared[1], &exact);
      return;
    }
  }
  int8_t* codes = a.codes + row * a.pitch;
  if (!(most * r <= kMost)) {  // not finite
    for (int c = me * 8; c < a.pitch; c += team * 8) *reinterpret_cast<uint2*>(codes + c) = make_uint2(0, 0);
    if (me == 0) a.scales[row] = __uint_as_float(0x7fc00000u);
    return;
  }
  const bool tiny = most * r < 127 * 0x1p-126f;  // the step is its least, the quotient is v 2^126
  const float early = r;
  if (me == 0) {
    if (kNorms) r = __fdiv_rn(1.f, __fsqrt_rn(__fadd_rn(__fdiv_rn(squares, static_cast<float>(a.cols)), a.eps)));
    a.scales[row] = scale_of(most * r);
  }
  if (kNorms && tiny) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) held[h][i] *= early;
  }

  // What codes go by, the largest magnitude or what has the least step, to more than fp32: of what comes near to it, the largest.  What
  // is taken exactly is held times 2^unit, which brings that to 1 .. 4.
  const float top = tiny ? 127 * 0x1p-126f : most;
  const int unit = 127 - min(static_cast<int>(__float_as_uint(top) >> 23), 253);
  Two peak{top * power_of_two(unit), 0.f};
  auto find_peak = [&] {
    const float near = most * (1.f - 0x1p-18f);
    unsigned long long key = 0;
    uint32_t mask = 0;  // bit 8 h + i
    if (kOp != kGate || mine >= near) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) mask |= (fabsf(held[h][i]) >= near ? 1u : 0u) << (8 * h + i);
    }
    for (; mask; mask &= mask - 1) {
      const int i = __ffs(mask) - 1;
      key = max(key, ordered(magnitude(in.exactly(column(i / 8) + i % 8, unit))));
    }
#pragma unroll 1
    for (int c = column(kHeld); c < a.cols; c += team * 8) {
      float v[8];
      in.again(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) mask |= (fabsf(v[i]) >= near ? 1u : 0u) << i;
      for (; mask; mask &= mask - 1) key = max(key, ordered(magnitude(in.exactly(c + __ffs(mask) - 1, unit))));
    }
    peak = from_ordered(Team<kTeam>::largest(key, &exact));
  };
  if constexpr (kPeakFirst) {
    if (!tiny) find_peak();  // the block's threads agree on that
  }
  const float per = __fdiv_rn(127.f, peak.hi), inverse = per * power_of_two(unit);
  // (of a tiny row the quantiser's quotients are exact, and a norm's are what fp32 has)
  const float border = tiny && kOp != kGate ? 1.f : 0.5f - kMargin<kOp, kPeakFirst>;
  // eight codes; the mask of those next to a border
  auto encode = [&](int c, const float(&v)[8]) {
    float k[8], d[8], far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      k[i] = __fmaf_rn(v[i], inverse, kMagic);
      d[i] = fabsf(__fmaf_rn(v[i], inverse, -(k[i] - kMagic)));
      far = fmaxf(far, d[i]);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = __byte_perm(__byte_perm(__float_as_uint(k[4 * i]), __float_as_uint(k[4 * i + 1]), 0x0040),
                         __byte_perm(__float_as_uint(k[4 * i + 2]), __float_as_uint(k[4 * i + 3]), 0x0040), 0x5410);
    *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
    uint32_t mask = 0;
    if (far > border) {
#pragma unroll
      for (int i = 0; i < 8; ++i) mask |= (d[i] > border ? 1u : 0u) << i;
    }
    return mask;
  };
  auto correct = [&](int c) {
    const Two v = in.exactly(c, unit), m = magnitude(v);
    codes[c] = static_cast<int8_t>(copysignf(decide(m, peak, per), v.hi));
  };
  uint32_t mask = 0;
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (column(h) < a.pitch) mask |= encode(column(h), held[h]) << (8 * h);
  if constexpr (kOp != kQuantize && !kPeakFirst) {
    // (a thread with columns that it does not hold does not know of them yet)
    bool some = mask != 0 || column(kHeld) < a.cols;
    if constexpr (kTeam == 0)
      some = __syncthreads_or(some);
    else
      some = __any_sync(Team<kTeam>::mask(), some);
    if (some && !tiny) find_peak();
  }
  for (; mask; mask &= mask - 1) {
    const int i = __ffs(mask) - 1;
    correct(column(i / 8) + i % 8);
  }
#pragma unroll 1
  for (int c = column(kHeld); c < a.pitch; c += team * 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (c < a.cols) in.again(c, v);
    if (kNorms && tiny) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= early;
    }
    for (mask = encode(c, v); mask; mask &= mask - 1) correct(c + __ffs(mask) - 1);
  }
}

// threads: a block's, kThreads at most
template <typename T, Op kOp, int kHeld, int kTeam, int kThreads, int kBlocks>
int launch_teams(const RowArgs& a, int threads, cudaStream_t st) {
  static_assert(kHeld <= 4, "masks of 32 bits");
  const int rows_per = kTeam == 0 ? 1 : threads / (kTeam == 0 ? 1 : kTeam);
  return launch_ahead(k_q8_rows<T, kOp, kHeld, kTeam, kThreads, kBlocks>, dim3(static_cast<unsigned>((a.rows + rows_per - 1) / rows_per)),
                      dim3(1), threads, 0, st, a);
}

template <Op kOp>
int launch_rows(const RowArgs& a, int dtype, cudaStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int eights = a.pitch / 8;
    auto threads = [&](int each) { return (eights + 32 * each - 1) / (32 * each) * 32; };
    // us.  Short rows: eight lanes a row up to 128 columns (300000 x 64 24 us; a warp a row 88), a warp up to 1024 (gate of 20000 x 700
    // bf16 33; a block 43).  A quantiser's rows up to 4096 columns, and long ones of 16 bits: 32 elements a thread (19456 x 2560
    // bf16 33.2, with 16 35.2; gate of 2048 x 9728 29.5, 34.2).  Others 16: an fp32 thread would hold too much (gate of 1024 x 9728
    // 22.1, with 32 28.5), and so would a norm's.
    if constexpr (kOp == kQuantize || kOp == kGate) {
      if (a.cols <= 128) return launch_teams<T, kOp, 2, 8, 128, 8>(a, 128, st);
      if (a.cols <= 1024) return launch_teams<T, kOp, 4, 32, 128, 8>(a, 128, st);
      if (a.cols <= 4096) {
        if constexpr (kOp == kQuantize)
          return launch_teams<T, kOp, 4, 0, 128, 6>(a, threads(4), st);
        else
          return launch_teams<T, kOp, 2, 0, 256, 4>(a, threads(2), st);
      }
      if constexpr (sizeof(T) == 2)
        return launch_teams<T, kOp, 4, 0, 320, 3>(a, std::min(320, threads(4)), st);
      else
        return launch_teams<T, kOp, 2, 0, 640, 2>(a, std::min(640, threads(2)), st);
    } else {
      if (a.cols <= 1024) return launch_teams<T, kOp, 4, 32, 128, 6>(a, 128, st);
      // (64 registers are too few for fp32 rows with a residual: 5916 x 2560 36.6, with up to 80 34.4.)
      constexpr int kBlocks = sizeof(T) == 4 && kOp == kNormResidual ? 3 : 4;
      if (a.cols <= 4096) return launch_teams<T, kOp, 2, 0, 256, kBlocks>(a, threads(2), st);
      // Norms past 4096 columns: two blocks an SM (2048 x 9728 bf16 without a residual 25.7, with one block 40.8); with a residual
      // smaller ones (bf16 36.8, 42.5; 2000 x 5000 fp32 26.0, 29.2; of one row 3.5 and 4.1, where 640 threads take 3.1).  Nothing here
      // goes by the rows: a row's sums, and so its scale's last place, are the same in any batch.
      if constexpr (kOp == kNorm)
        return launch_teams<T, kOp, 2, 0, 640, 2>(a, std::min(640, threads(2)), st);
      else if constexpr (sizeof(T) == 2)
        return launch_teams<T, kOp, 3, 0, 416, 2>(a, std::min(416, threads(3)), st);
      else
        return launch_teams<T, kOp, 2, 0, 512, 2>(a, std::min(512, threads(2)), st);
    }
  });
}

// Eight values of the output, taken as one row of rows * cols, from up to two 8-byte words of codes.
template <typename T>
__device__ __forceinline__ void read_eight(const int8_t* __restrict__ codes, const float* __restrict__ scales, long long at,
                                           long long all, int cols, int pitch, bool wide, T* __restrict__ out) {
  if (at >= all) return;
  // (32-bit division where it does)
  long long row = at >> 32 ? at / cols : static_cast<uint32_t>(at) / static_cast<uint32_t>(cols);
  int c = static_cast<int>(at - row * cols);
  float v[8];
  if (c + 8 <= cols) {
    const uint2* w = reinterpret_cast<const uint2*>(codes + row * pitch + (c & ~7));
    uint2 lo = __ldcg(w), hi = c & 7 ? __ldcg(w + 1) : make_uint2(0, 0);
    const uint32_t b[4] = {lo.x, lo.y, hi.x, hi.y};
    const float s = __ldcg(scales + row);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t p = c & 4 ? b[i + 1] : b[i], q = c & 4 ? b[i + 2 < 4 ? i + 2 : 3] : b[i + 1];
      const uint32_t u = __funnelshift_r(p, q, c % 4 * 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = s * static_cast<float>(static_cast<int8_t>(u >> (8 * e)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = at + i < all ? __ldcg(scales + row) * static_cast<float>(__ldcg(reinterpret_cast<const signed char*>(codes) + row * pitch + c)) : 0.f;
      if (++c == cols) c = 0, ++row;
    }
  }
  Eight<T> o;
  o.set(v);
  o.store(out + at, 0, static_cast<int>(min(all - at, 8ll)), wide ? 0 : 1);
}
template <typename T>
__global__ void __launch_bounds__(256) k_q8_read(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                 long long all, int cols, int pitch, bool wide, T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  read_eight(codes, scales, (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) * 8, all, cols, pitch, wide, out);
}
// Rows of whole 16 columns, and an output that starts on 16 bytes: 16 codes a thread (19456 x 2560 bf16 24.3 us, 6.1 TB/s; by
// eights 30.3).
template <typename T>
__global__ void __launch_bounds__(256) k_q8_read16(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                   long long items, int per, T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= items) return;
  const long long row = i >> 32 ? i / per : static_cast<uint32_t>(i) / static_cast<uint32_t>(per);
  const uint4 raw = __ldcg(reinterpret_cast<const uint4*>(codes) + i);
  const float s = __ldcg(scales + row);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = s * static_cast<float>(static_cast<int8_t>(w[2 * h + e / 4] >> (e % 4 * 8)));
    Eight<T> o;
    o.set(v);
    o.store(out + i * 16, 8 * h, 16, 0);
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
// Whether `total`, contiguous, meets rows of which it is not the whole.
bool meets(const void* total, const void* x, long long stride, long long rows, int cols, int esz) {
  if (total == x && (stride == cols || rows == 1)) return false;
  const long long begin = static_cast<long long>(reinterpret_cast<uintptr_t>(total) - reinterpret_cast<uintptr_t>(x));  // past x
  const long long end = begin + rows * cols * esz, row = static_cast<long long>(cols) * esz, step = stride * esz;
  const long long first = begin < row ? 0 : (begin - row) / step + 1;  // the first row that ends behind its begin
  return first < rows && first * step < end;
}
int pitch_of(int cols) { return (cols + 15) / 16 * 16; }

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_quantize_q8(const void* x, int dtype, long long x_stride, long long rows, int cols, int8_t* codes,
                              float* scales, CUstream_st* stream) {
  if (bad_rows(x, dtype, x_stride, rows, cols, cols, codes, scales)) return S2_EINVAL;
  const RowArgs a{x, nullptr, nullptr, nullptr, codes, scales, x_stride, 0, rows, cols, pitch_of(cols), 0.f, 0.f};
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
      (residual && (residual_stride < cols || !aligned(residual, esz) || !aligned(total, esz) ||
                    meets(total, x, x_stride, rows, cols, esz) || meets(total, residual, residual_stride, rows, cols, esz))))
    return S2_EINVAL;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const RowArgs a{x, residual, weight, total, codes, scales, x_stride, residual_stride, rows, cols, pitch_of(cols), eps,
                  1.f / cols};
  return residual ? launch_rows<kNormResidual>(a, dtype, st) : launch_rows<kNorm>(a, dtype, st);
}

extern "C" int s2_swiglu_q8(const void* x, int dtype, long long x_stride, long long rows, int cols, int8_t* codes,
                            float* scales, CUstream_st* stream) {
  if (bad_rows(x, dtype, x_stride, rows, 2ll * cols, cols, codes, scales)) return S2_EINVAL;
  const RowArgs a{x, nullptr, nullptr, nullptr, codes, scales, x_stride, 0, rows, cols, pitch_of(cols), 0.f, 0.f};
  return launch_rows<kGate>(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int s2_dequantize_q8(const int8_t* codes, const float* scales, long long rows, int cols, void* out, int dtype,
                                CUstream_st* stream) {
  if (bad_rows(out, dtype, cols, rows, cols, cols, codes, scales)) return S2_EINVAL;
  const long long all = rows * cols;
  const bool sixteens = cols % 16 == 0 && aligned(out, 16);
  const long long items = sixteens ? all / 16 : (all + 7) / 8, grid = (items + 255) / 256;
  if (grid > 0x7fffffffll) return S2_EINVAL;
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    T* const to = static_cast<T*>(out);
    const dim3 blocks(static_cast<unsigned>(grid));
    return sixteens ? launch_ahead(k_q8_read16<T>, blocks, dim3(1), 256, 0, st, codes, scales, items, cols / 16, to)
                    : launch_ahead(k_q8_read<T>, blocks, dim3(1), 256, 0, st, codes, scales, all, cols, pitch_of(cols),
                                   aligned(out, 16), to);
  });
}
