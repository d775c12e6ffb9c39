// Attention over the paged 4-bit cache (see kv4.cuh for the layout):
//   o = sum_t softmax_t(scale * q . k_t) v_t  over the positions t that a row sees,
// in one pass over the cache with the running maximum and sum of the softmax.
//
// Two kernels, by the columns of a sequence; a column is a (row, query head) pair of a KV head:
//  - few (decode steps): mma.sync.m16n8k16 (fp16 operands, fp32 sums) with the cache as the A operand, which is
//    expanded from its codes in registers on the way.  tcgen05 would want it in shared or tensor memory first, and a
//    row of a decode step brings 4 to 8 columns where its smallest M or N has use for more.
//      S^T[16 positions][8 columns] = K[16][hd] Q^T[hd][8]
//      O^T[hd][8] += V^T[hd][16] P^T[16][8]
//  - many (pieces of prompts): tcgen05, the cache expanded once for 128 columns (k_kv4_tc, below).
// A weight of the softmax is two fp16 terms (22 bits), whose products with the values are added: rounded to one, 2^-11 of
// it, weights made fp16 results 2.4e-4 off 64 bits, where their own rounding is 2.1e-4, and took 20 % of them (4 % of bf16
// ones) to a neighbour of the rounded 64-bit result; now 0.3 % (0.03 %).  In the kernel for few a lane's two columns are
// then a weight's terms, four columns a tile, which costs nothing where a sequence has no more than four; with more,
// eight columns a tile and twice the products.  (8 x 30000 positions, four query heads a KV head: 79 us so, 85 with eight
// columns, 78 with one term; pieces of prompts 57 us, 54 with one term; 512 rows over 30000 397 and 378.)
// fp32 queries are two fp16 terms as well, a column each in the kernel for few, whose scores are added.  16-bit queries
// are exact in fp16: each row is scaled by a power of two.  Weights are kept as 2^6 exp2(s - m), m the running maximum or
// up to 8 (log2) below it: what falls off fp16's end is 2^-30 and less of the largest, and a maximum that rises a little
// costs no rescaling of the output.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "convert.cuh"
#include "kv4.cuh"
#include "ptx.cuh"
#include "s2_internal.h"
#include "tc05.cuh"

namespace s2 {
namespace {

constexpr int kStep = 16;       // positions of one pair of products
constexpr int kHalfPage = 32;   // positions that a warp copies at a time: two steps
constexpr int kDepth = 2;       // half pages that a warp holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightShift = 6.f, kSlack = 8.f;

struct AttnArgs {
  s2_kv4 c;
  const void* q;
  int n_head;
  int group;         // query heads of a KV head
  float scale;
  void* out;
  int n_split, split_pages;
  float* part_o;     // [row][head][split][hd]
  float2* part_ml;   // [row][head][split]
  int tries;         // of a wait
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 bits_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scale and zero point of the two fp16 values that are expanded together.
struct Pair {
  __half2 s, z1024, z64;  // scales, 1024 + zero, -(64 + zero)
  // a, b: {fp16 scale, fp16 zero} of the low and the high value
  __device__ __forceinline__ Pair(uint32_t a, uint32_t b) {
    s = bits_h2(__byte_perm(a, b, 0x5410));
    const __half2 z = bits_h2(__byte_perm(a, b, 0x7632));
    z1024 = __hadd2(z, __float2half2_rn(1024.f));
    z64 = __hsub2(__float2half2_rn(-64.f), z);
  }
};

// The four nibble pairs of w (the nibbles of its low half with those of its high half) as
// fp16(scale * (code - zero)).  0x6400 | code is 1024 + code in fp16 and 0x6400 | code << 4 is
// 1024 + 16 code, so code - zero comes out of one exact subtraction or FMA; the product is the one rounding.
__device__ __forceinline__ void expand(uint32_t w, const Pair& p, uint32_t (&v)[4]) {
  const uint32_t m = 0x64006400u;
  const uint32_t w8 = w >> 8;
  const __half2 sixteenth = __float2half2_rn(0.0625f);
  v[0] = h2_bits(__hmul2(p.s, __hsub2(bits_h2((w & 0x000f000fu) | m), p.z1024)));
  v[1] = h2_bits(__hmul2(p.s, __hfma2(bits_h2((w & 0x00f000f0u) | m), sixteenth, p.z64)));
  v[2] = h2_bits(__hmul2(p.s, __hsub2(bits_h2((w8 & 0x000f000fu) | m), p.z1024)));
  v[3] = h2_bits(__hmul2(p.s, __hfma2(bits_h2((w8 & 0x00f000f0u) | m), sixteenth, p.z64)));
}

// Half a page of the cache in shared memory.  Keys are read 16 bytes (a quarter row) a lane, rows packed;
// values a word or two of four rows a lane, rows padded so that the rows of the four lanes of a group
// start 32 bytes apart modulo 128: both without bank conflicts.
template <int HD>
struct Stage {
  using B = Kv4Block<HD>;
  static constexpr int kVRow = B::kRow + 16;
  static constexpr int kK = 0, kKPar = kHalfPage * B::kRow, kV = kKPar + kHalfPage * B::kPar,
                       kVPar = kV + kHalfPage * kVRow;
  static constexpr int kBytes = kVPar + kHalfPage * B::kPar;
};

// a warp's copy of half `half` of a page block
template <int HD>
__device__ __forceinline__ void copy_half(uint8_t* st, const uint8_t* block, int half, int lane) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int per = B::kRow / 16;  // 16-byte units of a row
  const uint8_t* k = block + half * (kHalfPage * B::kRow) + lane * 16;
  uint8_t* to = st + lane * 16;
#pragma unroll
  for (int i = 0; i < per; ++i) cp_async16(to + S::kK + i * 512, k + i * 512);
  to = st + S::kV + lane / per * S::kVRow + lane % per * 16;
#pragma unroll
  for (int i = 0; i < per; ++i) cp_async16(to + i * (32 / per) * S::kVRow, k + B::kHalf + i * 512);
  constexpr int np = kHalfPage * B::kPar / 16;  // 32 or 16
  const uint8_t* par = block + kPage * B::kRow + half * (kHalfPage * B::kPar);
  if constexpr (np == 32) {
    cp_async16(st + S::kKPar + lane * 16, par + lane * 16);
    cp_async16(st + S::kVPar + lane * 16, par + B::kHalf + lane * 16);
  } else {
    const bool v = lane >= np;
    cp_async16(st + (v ? S::kVPar : S::kKPar) + lane % np * 16, par + (v ? B::kHalf : 0) + lane % np * 16);
  }
}

// A row's scores are computed from its query times `up`, and multiplied by `down`: the largest element goes to
// 2^13 .. 2^14, exact and far from fp16's ends.  `down` is positive (a negative scale turns the query, a scale of 0
// makes it 0), so that a masked score stays -inf.
struct QueryScale {
  float up, down;
  __device__ __forceinline__ QueryScale(float top, float scale) {
    const int e = top > 0.f && isfinite(top) ? min(13 - ilogbf(top), 126) : 0;
    up = scale == 0.f ? 0.f : ldexpf(scale < 0.f ? -1.f : 1.f, e);
    down = scale == 0.f ? 1.f : fmaxf(ldexpf(1.f, -e) * (fabsf(scale) * kLog2e), 1e-37f);
  }
};

// The query columns of a warp as B operand: lane (g = lane / 4, c = lane % 4) holds column g of each
// group of 8 at the elements that lane c expands of a key row.
template <typename T, int HD>
__device__ __forceinline__ float load_q(const T* q, bool live, bool low, float scale, int c, uint32_t (&f)[HD / 8]) {
  constexpr int E = HD / 4;
  float x[E], top = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    x[i] = live ? to_f(q[c * E + i]) : 0.f;
    top = fmaxf(top, fabsf(x[i]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const QueryScale qs(top, scale);
#pragma unroll
  for (int j = 0; j < E / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = x[8 * j + i] * qs.up, b = x[8 * j + i + 4] * qs.up;
      if (low) {
        a -= round_f16(a);
        b -= round_f16(b);
      }
      f[4 * j + i] = h2_bits(__floats2half2_rn(a, b));
    }
  return qs.down;
}

// S^T of one step: scores of rows g, g + 8 at columns 2c, 2c + 1
template <int HD>
__device__ __forceinline__ void scores(uint32_t st, int step, int g, int c, const uint32_t (&q)[HD / 8],
                                       float (&s)[4]) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int W = HD / 32;  // words of a lane's quarter row
  uint32_t r0[W], r1[W];
  const uint32_t a = st + S::kK + (step * kStep + g) * B::kRow + c * (HD / 8);
  if constexpr (W == 4) {
    const uint4 x = lds128(a), y = lds128(a + 8 * B::kRow);
    r0[0] = x.x, r0[1] = x.y, r0[2] = x.z, r0[3] = x.w;
    r1[0] = y.x, r1[1] = y.y, r1[2] = y.z, r1[3] = y.w;
  } else {
    const uint2 x = lds64(a), y = lds64(a + 8 * B::kRow);
    r0[0] = x.x, r0[1] = x.y;
    r1[0] = y.x, r1[1] = y.y;
  }
  const uint32_t par = st + S::kKPar + (step * kStep + g) * B::kPar + c * (HD / 4) / kKvGroup * 4;
  const uint32_t p0 = lds32(par), p1 = lds32(par + 8 * B::kPar);
  const Pair pa(p0, p0), pb(p1, p1);
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    uint32_t x[4], y[4];
    expand(r0[j], pa, x);
    expand(r1[j], pb, y);
    mma_f16_16816(s, x[0], y[0], x[1], y[1], q[4 * j], q[4 * j + 1]);
    mma_f16_16816(s, x[2], y[2], x[3], y[3], q[4 * j + 2], q[4 * j + 3]);
  }
}

// Whether parameters of the step's values are no numbers (for the whole warp): each lane looks at its share.
template <int HD>
__device__ __forceinline__ bool odd_values(uint32_t st, int step, int lane) {
  using S = Stage<HD>;
  const uint32_t a = st + S::kVPar + step * kStep * Kv4Block<HD>::kPar;
  auto odd = [](uint32_t w) { return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u; };
  uint32_t bad;
  if constexpr (HD == 128) {
    const uint2 w = lds64(a + lane * 8);
    bad = odd(w.x) | odd(w.y);
  } else {
    bad = odd(lds32(a + lane * 4));
  }
  return __any_sync(0xffffffffu, bad != 0);
}

// O^T += V^T P^T of one step.  Lane (g, c) expands elements g * hd/8 .. + hd/8 - 1 of rows 2c, 2c + 1, 2c + 8,
// 2c + 9; element 2i of those is row g, element 2i + 1 row g + 8 of the i-th tile.  Where not kPlain, the
// parameters of rows from `valid` on (behind the sequence: their weights are zero, but what is there may be no
// number) and those that are no numbers count as zero.  p: the terms of the weights (kTwo: one, of columns in pairs).
// kApart: the step's products start at zero and are added to O outside the tensor core, which cuts a sum off at its
// last bit at every addition (as k_kv4_tc's).
template <int HD, bool kPlain, bool kApart, bool kTwo>
__device__ __forceinline__ void values(uint32_t st, int step, int g, int c, int valid, const uint32_t (&p)[2][2],
                                       float (&o)[HD / 16][4]) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int W = HD / 64;  // words of a row that a lane expands
  uint32_t w[4][W], par[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = 2 * c + (k & 1) + (k >> 1) * 8;
    const uint32_t a = st + S::kV + (step * kStep + row) * S::kVRow + g * (HD / 16);
    if constexpr (W == 2) {
      const uint2 x = lds64(a);
      w[k][0] = x.x, w[k][1] = x.y;
    } else {
      w[k][0] = lds32(a);
    }
    par[k] = lds32(st + S::kVPar + (step * kStep + row) * B::kPar + g * (HD / 8) / kKvGroup * 4);
    if (!kPlain && (row >= valid || (par[k] & 0x7c00u) == 0x7c00u || (par[k] & 0x7c000000u) == 0x7c000000u)) par[k] = 0;
  }
  const Pair lo(par[0], par[1]), hi(par[2], par[3]);
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t x[4], y[4];
      const uint32_t sel = h ? 0x7632 : 0x5410;
      expand(__byte_perm(w[0][j], w[1][j], sel), lo, x);
      expand(__byte_perm(w[2][j], w[3][j], sel), hi, y);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float(&to)[4] = o[4 * j + 2 * h + i];
        if constexpr (kApart) {
          float d[4];
          mma_f16_16816_first(d, x[2 * i], x[2 * i + 1], y[2 * i], y[2 * i + 1], p[0][0], p[0][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) to[k] += d[k];
        } else {
          if constexpr (!kTwo) mma_f16_16816(to, x[2 * i], x[2 * i + 1], y[2 * i], y[2 * i + 1], p[1][0], p[1][1]);
          mma_f16_16816(to, x[2 * i], x[2 * i + 1], y[2 * i], y[2 * i + 1], p[0][0], p[0][1]);
        }
      }
    }
}

// The running state of a warp's columns.  A lane's columns are 2c, 2c + 1 (kTwo: the two terms of one), the same in the
// scores and in the output tiles.
template <int HD, bool kTwo>
struct Rows {
  static constexpr int NC = kTwo ? 1 : 2;  // a lane's logical columns
  static constexpr float kNone = 3e38f;    // `lift` before a column has seen a position
  float o[HD / 16][4];
  float lift[NC];  // kWeightShift - m, m the running maximum (log2 units): a weight is exp2(score + lift)
  float l[NC], f[NC];  // this lane's part of the sum, score factor
  int lim[NC];             // positions seen

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < HD / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) lift[j] = kNone, l[j] = 0.f;
  }
  __device__ __forceinline__ float maximum(int j) const {
    return lift[j] == kNone ? -INFINITY : kWeightShift - lift[j];
  }

  // one step at position t0: s becomes the weights, as B operand, in two terms (kTwo: a column each)
  __device__ __forceinline__ void softmax(float (&s)[4], int t0, int g, bool cut, uint32_t (&p)[2][2]) {
    if constexpr (kTwo) s[0] += s[1], s[2] += s[3];
    if (cut) {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (t0 + g + 8 * r >= lim[j]) s[2 * r + j] = -INFINITY;
    }
    float e[2][NC], top = -INFINITY;  // [row g, row g + 8][column]
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      e[0][j] = __fmaf_rn(s[j], f[j], lift[j]);
      e[1][j] = __fmaf_rn(s[2 + j], f[j], lift[j]);
      top = fmaxf(top, fmaxf(e[0][j], e[1][j]));
    }
    if (__any_sync(0xffffffffu, top > kWeightShift + kSlack)) rise(s, e);
    float w[2][2];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      w[0][j] = ex2(e[0][j]);
      w[1][j] = ex2(e[1][j]);
      l[j] += w[0][j] + w[1][j];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if constexpr (kTwo) w[r][1] = w[r][0] - round_f16(w[r][0]);
      const __half2 h = __floats2half2_rn(w[r][0], w[r][1]);
      p[0][r] = movmatrix_trans(h2_bits(h));
      if constexpr (!kTwo) {
        const float2 f = __half22float2(h);
        p[1][r] = movmatrix_trans(h2_bits(__floats2half2_rn(w[r][0] - f.x, w[r][1] - f.y)));
      }
    }
  }

  // the maxima raised to the step's, output and sums rescaled
  __device__ __forceinline__ void rise(const float (&s)[4], float (&e)[2][NC]) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const float x0 = s[j] * f[j], x1 = s[2 + j] * f[j];
      float top = fmaxf(x0, x1);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float m = maximum(j), mn = fmaxf(m, top);
      if (mn > -INFINITY) {  // the same in all lanes of the column
        const float keep = ex2(m - mn);
        lift[j] = kWeightShift - mn;
        l[j] *= keep;
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          if constexpr (kTwo) {
            o[i][0] *= keep, o[i][1] *= keep, o[i][2] *= keep, o[i][3] *= keep;
          } else {
            o[i][j] *= keep, o[i][2 + j] *= keep;
          }
        }
      }
      e[0][j] = __fmaf_rn(s[j], f[j], lift[j]);
      e[1][j] = __fmaf_rn(s[2 + j], f[j], lift[j]);
    }
  }

  // a value row of the step that is no number: every column that sees it is none either, in its group's elements
  __device__ __forceinline__ void poison(uint32_t st, int step, int t0, int valid, int g) {
    using S = Stage<HD>;
    for (int r = 0; r < valid; ++r) {
      const uint32_t par = lds32(st + S::kVPar + (step * kStep + r) * Kv4Block<HD>::kPar + g * (HD / 8) / kKvGroup * 4);
      if ((par & 0x7c00u) != 0x7c00u && (par & 0x7c000000u) != 0x7c000000u) continue;
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t0 + r < lim[kTwo ? 0 : j % 2]) o[i][j] = NAN;
    }
  }

  __device__ __forceinline__ void finish_sums() {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    }
  }
};

// Where a tile of columns lies: its sequence, that one's rows q0 .. q1 - 1 and length, and the first of the tile's
// columns there.  Tiles are counted over the sequences in order; seq -1 where there are fewer.  Bounds and lengths
// come in one round of loads.
struct Tile {
  int seq, first, q0, q1, len;
};
__device__ __forceinline__ Tile find_tile(const s2_kv4& k, int group, int cols, int t) {
  const int lane = threadIdx.x % 32;
  int before = 0;
  for (int base = 0; base < k.n_seq; base += 32) {
    const int s = base + lane;
    int q0 = 0, q1 = 0, len = 0;
    if (s < k.n_seq) q0 = __ldg(k.q_start + s), q1 = __ldg(k.q_start + s + 1), len = __ldg(k.lengths + s);
    const int tiles = (min(max(q1 - q0, 0), k.n_rows) * group + cols - 1) / cols;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > t);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return {base + l, (t - before - __shfl_sync(0xffffffffu, upto - tiles, l)) * cols,
              __shfl_sync(0xffffffffu, q0, l), __shfl_sync(0xffffffffu, q1, l), __shfl_sync(0xffffffffu, len, l)};
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return {-1, 0, 0, 0, 0};
}

// pages of a sequence's table, 32 at a time in the lanes of a warp
struct Pages {
  const int32_t* row;
  int n, n_pages, base = -64, mine = -1;
  __device__ __forceinline__ int id(int p, int32_t* status) {
    if (p < base || p >= base + 32) {
      base = p & ~31;
      const int at = base + static_cast<int>(threadIdx.x % 32);
      mine = at < n ? __ldg(row + at) : -1;
      if (at < n && (mine < 0 || mine >= n_pages)) {
        mine = -1;
        kv4_bad(status);
      }
    }
    return __shfl_sync(0xffffffffu, mine, p - base);
  }
};

constexpr int kWarps = 4;
template <int HD>
constexpr int kDecodeSmem = std::max(kWarps * kDepth * Stage<HD>::kBytes, kWarps * 8 * (HD + 4 + 2) * 4);

// Few columns: a block takes one tile of 8 columns (kTwo: 4 of two terms each, see above) of one KV head over a range of
// pages, two at a time.  Each of its four warps takes half a page with its own copies in flight, so the warps never wait
// on one another until their states are joined.  8 sequences of 30000 positions, 32 query heads on 8, hd 128: 79 us, 3.9
// TB/s of the cache (fp32 queries 82); 32 of 512 .. 4096: 31 us.  Bound by a step's chain (scores, exponential, turned
// weights, output) on the instructions that expand codes, 53 million a call of the first, each of which serves four query
// heads here: sixteen warps an SM fill 66 % of the issue slots with them; the copies alone take 55 us.
template <typename T, int HD, bool kTwo>
__global__ void __launch_bounds__(128) k_kv4_decode(const AttnArgs a) {
  constexpr bool kApart = sizeof(T) == 4;
  constexpr int CT = kTwo ? 4 : 8;  // logical columns
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int kORow = HD + 4;  // floats of a column's output in the joining buffer
  extern __shared__ __align__(16) uint8_t sm[];
  pdl_trigger();  // the joining kernel may find its rows
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int kh = blockIdx.y, split = blockIdx.z;
  const Tile tile = find_tile(a.c, a.group, CT, blockIdx.x);
  if (tile.seq < 0) return;
  const int q0 = tile.q0, q1 = tile.q1;
  if (q0 < 0 || q1 > a.c.n_rows) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    return;
  }
  const int cols = (q1 - q0) * a.group;
  int len = tile.len;
  const int over = len - (q1 - q0);  // row i sees over + i + 1 positions
  if (len > a.c.table_cols * kPage) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    len = a.c.table_cols * kPage;
  }
  len = max(len, 0);
  const int pages = (len + kPage - 1) / kPage;
  const int p0 = split * a.split_pages, p1 = split == a.n_split - 1 ? pages : min(pages, p0 + a.split_pages);
  if (p0 >= p1 && split > 0) return;
  const bool whole = a.n_split == 1 || pages <= a.split_pages;  // nothing to join

  uint8_t* ring = sm + warp * kDepth * S::kBytes;
  Pages pg{a.c.table + static_cast<size_t>(tile.seq) * a.c.table_cols, pages, a.c.n_pages};
  const uint8_t* heads = static_cast<const uint8_t*>(a.c.pages) + static_cast<size_t>(kh) * B::kBytes;
  uint32_t usable = 0;  // by turn modulo 32: copied
  const int half = warp & 1, turns = (p1 - p0 + 1) / 2;
  auto issue = [&](int turn) {
    const int p = p0 + 2 * turn + warp / 2;
    if (turn < turns) {
      const int id = pg.id(p < p1 ? p : p0, a.c.status);
      const bool ok = p < p1 && id >= 0 && p * kPage + half * kHalfPage < len;
      usable = ok ? usable | 1u << (turn & 31) : usable & ~(1u << (turn & 31));
      if (ok)
        copy_half<HD>(ring + turn % kDepth * S::kBytes, heads + static_cast<size_t>(id) * a.c.n_kv_head * B::kBytes,
                      half, lane);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue(i);

  Rows<HD, kTwo> st;
  st.init();
  uint32_t qf[HD / 8];
  {
    const int col = tile.first + (kTwo ? g / 2 : g);
    const bool live = col < cols;
    const int row = q0 + (live ? col / a.group : 0), h = kh * a.group + (live ? col % a.group : 0);
    const float down = load_q<T, HD>(static_cast<const T*>(a.q) + (static_cast<size_t>(row) * a.n_head + h) * HD, live,
                                     kTwo && (g & 1), a.scale, c, qf);
#pragma unroll
    for (int j = 0; j < st.NC; ++j) {
      const int mine = tile.first + (kTwo ? c : 2 * c + j);
      st.f[j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j));
      st.lim[j] = mine < cols ? min(over + mine / a.group + 1, len) : 0;
    }
  }
  const int first_lim = min(over + tile.first / a.group + 1, len);  // the least that a live column sees

  for (int turn = 0; turn < turns; ++turn) {
    issue(turn + kDepth - 1);
    cp_async_wait_group<kDepth - 1>();
    __syncwarp();
    if (usable >> (turn & 31) & 1) {
      const uint32_t at = smem_u32(ring + turn % kDepth * S::kBytes);
      const int first = (p0 + 2 * turn + warp / 2) * kPage + half * kHalfPage;
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const int t0 = first + step * kStep, valid = min(len - t0, kStep);
        if (valid <= 0) break;
        float s[4];
        uint32_t pf[2][2];
        scores<HD>(at, step, g, c, qf, s);
        // where every column sees the whole step, a value that is no number reaches all of them anyway
        const bool cut = t0 + kStep > first_lim;
        st.softmax(s, t0, g, cut, pf);
        const bool odd = cut && odd_values<HD>(at, step, lane);
        if (!odd && valid == kStep) {
          values<HD, true, kApart, kTwo>(at, step, g, c, valid, pf, st.o);
        } else {
          values<HD, false, kApart, kTwo>(at, step, g, c, valid, pf, st.o);
          if (odd) st.poison(at, step, t0, valid, g);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait_all();
  st.finish_sums();
  __syncthreads();
  // join the warps: [warp][column] of (output, maximum, sum)
  float* jo = reinterpret_cast<float*>(sm);
  float* jm = jo + kWarps * CT * kORow;
#pragma unroll
  for (int j = 0; j < st.NC; ++j) {
    const int col = kTwo ? c : 2 * c + j;
    float* dst = jo + (warp * CT + col) * kORow + g * (HD / 8);
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {
      if constexpr (kTwo) {
        dst[2 * i] = st.o[i][0] + st.o[i][1];
        dst[2 * i + 1] = st.o[i][2] + st.o[i][3];
      } else {
        dst[2 * i] = st.o[i][j];
        dst[2 * i + 1] = st.o[i][2 + j];
      }
    }
    if (g == 0) {
      jm[(warp * CT + col) * 2] = st.maximum(j);
      jm[(warp * CT + col) * 2 + 1] = st.l[j];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < CT * HD; i += blockDim.x) {
    const int col = i / HD, e = i % HD, mine = tile.first + col;
    if (mine >= cols) break;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, jm[(w * CT + col) * 2]);
    const float base = m == -INFINITY ? 0.f : m;
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(jm[(w * CT + col) * 2] - base);
      o += f * jo[(w * CT + col) * kORow + e];
      l += f * jm[(w * CT + col) * 2 + 1];
    }
    const size_t at = static_cast<size_t>(q0 + mine / a.group) * a.n_head + kh * a.group + mine % a.group;
    if (whole) {
      static_cast<T*>(a.out)[at * HD + e] = from_f<T>(l == 0.f ? 0.f : o / l);
    } else {
      a.part_o[(at * a.n_split + split) * HD + e] = o;
      if (e == 0) a.part_ml[at * a.n_split + split] = make_float2(m, l);
    }
  }
}

// ---- many columns: a block takes 128 columns of one KV head, each a row of tcgen05 products, a page at a time:
//   S[128][64] = Q[128][hd] K[64][hd]^T      Q and K in shared memory
//   O[128][hd] += P[128][64] V[64][hd]       P in tensor memory, V^T in shared memory
// Four warps have a column a thread: its scores, its maximum, its sum and its row of the output, all in tensor
// memory lanes of its own, so the softmax has no shuffles.  Four more expand every page once for all columns (a
// thread 64 key codes and 32 values of two positions; its codes wait in registers while the page before is used),
// and a ninth issues the products, so that expanding, exponentials and products overlap.  The two blocks of an SM
// share its tensor memory.  Weights are two fp16 terms, and so are fp32 queries: their products run twice, into the same
// sums, the small terms first.  The tensor core cuts every sum off at its last bit, a few 1e-8 each, in
// one direction; so with fp32 queries a page's output starts at zero, and the threads of its rows add it to the one so
// far, which has tensor memory of its own (pieces of prompts over up to 3000 positions: 2.7e-6 off 64 bits without,
// 2.7e-7 with, for 1 to 10 % of the time).
// Operands lie in the 128-byte-swizzled layout; the elements of eight key codes in the order 0 4 1 5 2 6 3 7,
// queries alike.
// 512 bf16 rows over 30000 positions: 397 us, 640 TFLOP/s (fp32 705); five pieces of prompts (874 rows over up to 42
// pages): 57 us, with the joining, 66 where the cache is not in L2.  Bound by a page's chain of scores, exponentials (one
// thread a column) and output.
constexpr int kTcCols = 128;
template <int HD, int TN>
struct Tc {
  static constexpr int kAtoms = HD / 64;                // 128-byte columns of Q and K
  static constexpr int kQAtom = kTcCols * 128, kKAtom = kPage * 128;
  static constexpr int kQ = 0, kK = kQ + TN * kAtoms * kQAtom, kV = kK + kAtoms * kKAtom, kVBuf = HD * 128,
                       kOdd = kV + 3 * kVBuf, kBars = kOdd + 4 * 4 * kPage, kBytes = kBars + 128 + 1024;
  // tensor memory columns: the output, two pages' scores, whose place their weights take, and (fp32 queries) the
  // output of the pages before the last one
  static constexpr uint32_t kO = 0, kS = HD, kBefore = kS + 2 * kPage, kUsed = kBefore + (TN == 2 ? HD : 0),
                            kCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= kCols && TN * 32 <= kPage, "tensor memory");
};

// Warp-wide: 32 consecutive tensor memory columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// (complete after tmem_st_wait)
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// What a thread holds of a page: hd/64 groups of 32 keys of a row, and 32 (hd 64: 16) values of positions l and
// l + 32, l its lane, with their parameters.  Neighbouring lanes read neighbouring 16 bytes of keys and, of values,
// neighbouring rows.  (Positions l and l + 32 share a word of the weights and of V^T: its K index 2l, 2l + 1.)
template <int HD>
struct PageCodes {
  static constexpr int kU = HD / 64, kGroups = HD / kKvGroup;
  uint4 k[kU];
  uint32_t kp[kU], vp[2];
  uint2 v[2][kU];
  // `rows` of the page are in the sequence
  __device__ __forceinline__ void load(const uint8_t* block, int rows) {
    using B = Kv4Block<HD>;
    const int tid = threadIdx.x % kTcCols, lane = tid % 32, warp = tid / 32;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int unit = tid + i * kTcCols;
      const bool in = unit / kGroups < rows;
      k[i] = in ? __ldg(reinterpret_cast<const uint4*>(block) + unit) : make_uint4(0, 0, 0, 0);
      kp[i] = in ? __ldg(reinterpret_cast<const uint32_t*>(block + kPage * B::kRow) + unit) : 0;
    }
    const uint8_t* vb = block + B::kHalf;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = lane + 32 * t;
      const bool in = r < rows;
      const uint8_t* p = vb + r * B::kRow + warp * (kU * 8);
      if constexpr (kU == 2) {
        const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
        v[t][0] = make_uint2(u.x, u.y), v[t][1] = make_uint2(u.z, u.w);
      } else {
        v[t][0] = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
      }
      vp[t] = in ? __ldg(reinterpret_cast<const uint32_t*>(vb + kPage * B::kRow + r * B::kPar) + warp * HD / 128) : 0;
    }
  }
  // Into the operands' layouts.
  __device__ __forceinline__ void expand_keys(uint8_t* kt) const {
    const int tid = threadIdx.x % kTcCols;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int unit = tid + i * kTcCols, row = unit / kGroups, group = unit % kGroups;
      const Pair pk(kp[i], kp[i]);
      const bool turn = group / 2;  // the two atoms' chunks share banks: the second's go in another order
      const uint32_t kw[4] = {turn ? k[i].z : k[i].x, turn ? k[i].w : k[i].y, turn ? k[i].x : k[i].z, turn ? k[i].y : k[i].w};
      uint8_t* to = kt + group / 2 * (kPage * 128) + row * 128;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[4];
        expand(kw[j], pk, x);
        const int chunk = group % 2 * 4 + (turn ? j ^ 2 : j);
        *reinterpret_cast<uint4*>(to + ((chunk ^ (row & 7)) * 16)) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  // Values whose parameters are no numbers become zeros; returns whether there are.
  __device__ __forceinline__ bool expand_values(uint8_t* vt, uint16_t* odd_rows) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % 4;
    uint16_t odd = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if ((vp[t] & 0x7c00u) == 0x7c00u || (vp[t] & 0x7c000000u) == 0x7c000000u) {
        odd |= 1u << (8 * t);
        vp[t] = 0;
      }
    odd_rows[warp * 32 + lane] = odd;
    const Pair pv(vp[0], vp[1]);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const uint32_t w0[2] = {v[0][i].x, v[0][i].y}, w1[2] = {v[1][i].x, v[1][i].y};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[4];
          expand(__byte_perm(w0[j], w1[j], h ? 0x7632 : 0x5410), pv, x);
          const int dim = warp * (kU * 16) + i * 16 + j * 8 + h * 4;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint32_t*>(vt + (dim + e) * 128 + (((lane / 4) ^ ((dim + e) & 7)) * 16) + lane % 4 * 4) = x[e];
        }
    }
    return odd != 0;
  }
};

// 96 registers a thread: two blocks an SM.  fp32 queries at head size 128 have tensor memory and shared memory for one.
constexpr int kTcThreads = 2 * kTcCols + 32;
template <typename T, int HD>
__global__ void __maxnreg__(sizeof(T) == 4 && HD == 128 ? 168 : 96) k_kv4_tc(const AttnArgs a) {
  constexpr int TN = sizeof(T) == 4 ? 2 : 1;
  constexpr bool kApart = TN == 2;
  using B = Kv4Block<HD>;
  using M = Tc<HD, TN>;
  extern __shared__ __align__(16) uint8_t smraw[];
  pdl_trigger();
  uint8_t* sm = smraw + (-smem_u32(smraw) & 1023u);
  // Barriers.  Operands of page n: filled[n % 2]; its scores: scored[n % 2] (the products' arrival and their
  // issuer's); its weights: weighed[n % 2]; the output with it: summed[n % 2].  A barrier completes again only after
  // all that wait for it have seen it, since each of them has a part in what comes before its next completion.
  uint64_t* filled = reinterpret_cast<uint64_t*>(sm + M::kBars);
  uint64_t *scored = filled + 2, *weighed = filled + 4, *summed = filled + 6, *drained = filled + 8;
  uint32_t* tbase = reinterpret_cast<uint32_t*>(filled + 9);
  int* place = reinterpret_cast<int*>(tbase + 1);                  // [n % 4]: page n in the sequence, -1 after the last
  uint8_t* odd_any = reinterpret_cast<uint8_t*>(place + 4);        // [n % 4][warp]: values that are no numbers
  volatile int* failed = place + 8;                                // a wait gave up
  uint16_t* odd_rows = reinterpret_cast<uint16_t*>(sm + M::kOdd);  // [n % 4][warp][lane], a byte a position
  const int warp = threadIdx.x / 32;
  const int kh = blockIdx.y, split = blockIdx.z;
  const Tile tile = find_tile(a.c, a.group, kTcCols, blockIdx.x);
  if (tile.seq < 0) return;
  const int q0 = tile.q0, q1 = tile.q1;
  if (q0 < 0 || q1 > a.c.n_rows) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    return;
  }
  const int cols = (q1 - q0) * a.group;
  int len = tile.len;
  const int over = len - (q1 - q0);  // row i sees over + i + 1 positions
  if (len > a.c.table_cols * kPage) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    len = a.c.table_cols * kPage;
  }
  len = max(len, 0);
  const int pages = (len + kPage - 1) / kPage;
  const int p0 = split * a.split_pages;
  int p1 = split == a.n_split - 1 ? pages : min(pages, p0 + a.split_pages);
  if (p0 >= p1 && split > 0) return;
  const bool whole = a.n_split == 1 || pages <= a.split_pages;  // nothing to join
  // no column of the tile sees more than its last one, nor less than its first
  const int last = min(tile.first + kTcCols, cols) - 1;
  p1 = min(p1, (max(min(over + last / a.group + 1, len), 0) + kPage - 1) / kPage);
  const int least = min(over + tile.first / a.group + 1, len);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(filled + i, 4);
      mbar_init(scored + i, 2);
      mbar_init(weighed + i, kTcCols);
      mbar_init(summed + i, 1);
    }
    mbar_init(drained, 1);
    *failed = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tbase, M::kCols);
    tmem_relinquish();
  }

  // Where a wait gives up its warp goes on without waiting (all it touches is its block's own) and says so in `failed`,
  // which the block's results go by: they are NaN then, and the call reports it.
  bool ok = true;
  auto wait = [&](uint64_t* bar, int n) { return mbar_wait_short(bar + (n & 1), n >> 1 & 1, a.tries); };
  if (warp == 8) {
    // ---------------------------------------------------------------- issuing the products
    named_bar(2, kTcThreads);  // queries, barriers and tensor memory are there
    if (threadIdx.x % 32 == 0) {
      tc_fence_after();
      const uint32_t tm = *tbase;
      for (int n = 0;; ++n) {
        ok = ok && wait(filled, n);
        const bool end = !ok || place[n & 3] < 0;
        if (!end) {
          if (n > 1) ok = wait(summed, n - 2);  // the weights of page n - 2 lie there
          tc_fence_after();
          const uint32_t ts = tm + M::kS + (n & 1) * kPage;
#pragma unroll
          for (int t = TN - 1; t >= 0; --t)
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              tc_mma(ts, desc_sw128(smem_u32(sm + M::kQ) + (t * M::kAtoms + k / 4) * M::kQAtom + k % 4 * 32),
                     desc_sw128(smem_u32(sm + M::kK) + k / 4 * M::kKAtom + k % 4 * 32), idesc_f16(kTcCols, kPage),
                     t < TN - 1 || k > 0);
          tc_commit(scored + (n & 1));
        } else {
          mbar_arrive(scored + (n & 1));
        }
        mbar_arrive(scored + (n & 1));
        if (n > 0) {  // the output with page n - 1
          const int o = n - 1;
          ok = ok && wait(weighed, o);
          tc_fence_after();
          const uint32_t tp = tm + M::kS + (o & 1) * kPage;
#pragma unroll
          for (int t = 1; t >= 0; --t)
#pragma unroll
            for (int k = 0; k < kPage / 16; ++k)
              tc_mma_tmem_a(tm + M::kO, tp + t * 32 + k * 8, desc_sw128(smem_u32(sm + M::kV) + o % 3 * M::kVBuf + k * 32),
                            idesc_f16(kTcCols, HD), (!kApart && o > 0) || t < 1 || k > 0);
          tc_commit(summed + (o & 1));
        }
        if (end) break;
      }
      tc_commit(drained);  // no end before that of the products
      if (!mbar_wait_short(drained, 0) || !ok) *failed = 1;
    }
    __syncwarp();
    named_bar(3, kTcThreads);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- expanding
    const int lane = threadIdx.x % 32;
    const int32_t* table = a.c.table + static_cast<size_t>(tile.seq) * a.c.table_cols;
    const uint8_t* heads = static_cast<const uint8_t*>(a.c.pages) + static_cast<size_t>(kh) * B::kBytes;
    PageCodes<HD> held;
    int next = p0;
    int id = next < p1 ? __ldg(table + next) : -1;  // of page `next`, on its way a page ahead
    // the codes of the next page that is there; `next` ends at p1
    auto fetch = [&] {
      for (; next < p1; ++next) {
        const int now = id;
        id = next + 1 < p1 ? __ldg(table + next + 1) : -1;
        if (now >= 0 && now < a.c.n_pages) {
          held.load(heads + static_cast<size_t>(now) * a.c.n_kv_head * B::kBytes, len - next * kPage);
          return;
        }
        if (lane == 0) kv4_bad(a.c.status);
      }
    };
    fetch();
    named_bar(2, kTcThreads);
    for (int n = 0;; ++n) {
      const bool end = next >= p1;
      // values first: there are three buffers of them, while the keys wait for the scores of the page before
      if (n > 2) ok = ok && wait(summed, n - 3);  // the values of page n - 3 are used up
      __syncwarp();
      bool odd = false;
      if (!end) odd = held.expand_values(sm + M::kV + n % 3 * M::kVBuf, odd_rows + (n & 3) * 2 * kPage);
      if (n > 0) ok = ok && wait(scored, n - 1);  // the keys before are used up
      __syncwarp();
      if (!end) held.expand_keys(sm + M::kK);
      odd = __any_sync(0xffffffffu, odd);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        odd_any[(n & 3) * 4 + warp - 4] = odd;
        if (warp == 4) place[n & 3] = end ? -1 : next;
        mbar_arrive(filled + (n & 1));
      }
      if (end) break;
      ++next;
      fetch();
    }
    if (!ok) *failed = 1;
    named_bar(3, kTcThreads);
  } else {
    // ---------------------------------------------------------------- a column a thread
    const int col = tile.first + threadIdx.x;
    const bool live = col < cols;
    const size_t at = static_cast<size_t>(q0 + (live ? col / a.group : 0)) * a.n_head + kh * a.group + (live ? col % a.group : 0);
    const int lim = live ? min(over + col / a.group + 1, len) : 0;
    float factor;
    {
      // eight loads of a row under way together; rows are read twice
      constexpr int kPer = 16 / sizeof(T), kUnits = 8;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + at * HD);
      uint4 u[kUnits];
      float top = 0.f;
      constexpr int kTurns = HD / kPer / kUnits > 0 ? HD / kPer / kUnits : 1, kTurn = HD / kPer / kTurns;
#pragma unroll
      for (int h = 0; h < kTurns; ++h) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i) u[i] = __ldg(q + h * kTurn + i);
        const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
        for (int i = 0; i < kTurn * kPer; ++i) top = fmaxf(top, fabsf(to_f(e[i])));
      }
      const QueryScale qs(live ? top : 0.f, a.scale);
      factor = qs.down;
#pragma unroll
      for (int h = 0; h < kTurns; ++h) {
        if (kTurns > 1)
#pragma unroll
          for (int i = 0; i < kTurn; ++i) u[i] = __ldg(q + h * kTurn + i);
        const T* v = reinterpret_cast<const T*>(u);
#pragma unroll
        for (int g = 0; g < kTurn * kPer / 8; ++g) {
          const int i = h * (kTurn * kPer / 8) + g;
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = live ? to_f(v[g * 8 + k]) * qs.up : 0.f;
          uint8_t* to = sm + M::kQ + i / 8 * M::kQAtom + threadIdx.x * 128 + (((i % 8) ^ (threadIdx.x & 7)) * 16);
#pragma unroll
          for (int t = 0; t < TN; ++t) {
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              r[k] = h2_bits(__floats2half2_rn(x[k], x[k + 4]));
              x[k] -= round_f16(x[k]);
              x[k + 4] -= round_f16(x[k + 4]);
            }
            *reinterpret_cast<uint4*>(to + t * M::kAtoms * M::kQAtom) = make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    named_bar(2, kTcThreads);
    tc_fence_after();
    const uint32_t tlane = *tbase + (static_cast<uint32_t>(warp * 32) << 16);

    float lift = 3e38f, l = 0.f;  // as Rows
    uint32_t poison = 0;          // groups of the output that are no numbers
    int n = 0;
    for (;; ++n) {
      ok = __all_sync(0xffffffffu, wait(scored, n));
      const int p = ok ? place[n & 3] : -1;
      if (p < 0) break;
      tc_fence_after();
      const uint32_t tscore = tlane + M::kS + (n & 1) * kPage;
      float s[kPage];
      tmem_ld32(tscore, *reinterpret_cast<float(*)[32]>(s));
      tmem_ld32(tscore + 32, *reinterpret_cast<float(*)[32]>(s + 32));
      if ((p + 1) * kPage > least) {
        const int seen = lim - p * kPage;
#pragma unroll
        for (int i = 0; i < kPage; ++i)
          if (i >= seen) s[i] = -INFINITY;
      }
      if (*reinterpret_cast<const uint32_t*>(odd_any + (n & 3) * 4))
        for (int i = 0; i < kPage && p * kPage + i < lim; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (odd_rows[(n & 3) * 2 * kPage + w * 32 + i % 32] >> (8 * (i / 32)) & 1) poison |= 1u << (w * HD / 128);
      float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i < kPage; ++i) tops[i % 4] = fmaxf(tops[i % 4], s[i]);
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * factor;
      const bool rise = top + lift > kWeightShift + kSlack;
      float keep = 1.f;
      // the output so far times `keep`; where it is apart, with the last page's
      auto carry = [&] {
        ok = __all_sync(0xffffffffu, wait(summed, n - 1));
        if (!ok) return;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          float o[16];
          uint32_t r[16];
          tmem_ld16(tlane + M::kO + c, o);
          if (kApart && n > 1) {
            float before[16];
            tmem_ld16(tlane + M::kBefore + c, before);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] += before[i];
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(o[i] * keep);
          tmem_st16(tlane + (kApart ? M::kBefore : M::kO) + c, r);
        }
      };
      if (__any_sync(0xffffffffu, rise)) {
        const float m = lift == 3e38f ? -INFINITY : kWeightShift - lift, mn = fmaxf(m, top);
        if (rise) {
          keep = ex2(m - mn);
          lift = kWeightShift - mn;
          l *= keep;
        }
        __syncwarp();
        if (!kApart && n > 0) {
          carry();
          if (!ok) break;
        }
      }
      float2 sum[2] = {};
      const float2 f2 = make_float2(factor, factor), lift2 = make_float2(lift, lift), minus = make_float2(-1.f, -1.f);
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float2 e0 = __ffma2_rn(make_float2(s[c + i], s[c + i + 1]), f2, lift2);
          float2 e1 = __ffma2_rn(make_float2(s[c + i + 32], s[c + i + 33]), f2, lift2);
          e0 = make_float2(ex2(e0.x), ex2(e0.y)), e1 = make_float2(ex2(e1.x), ex2(e1.y));
          sum[i / 2 % 2] = __fadd2_rn(sum[i / 2 % 2], __fadd2_rn(e0, e1));
          const __half2 h0 = __floats2half2_rn(e0.x, e1.x), h1 = __floats2half2_rn(e0.y, e1.y);
          const float2 g0 = __half22float2(h0), g1 = __half22float2(h1);
          hi[i] = h2_bits(h0), hi[i + 1] = h2_bits(h1);
          const float2 r0 = __ffma2_rn(make_float2(g0.x, g1.x), minus, e0), r1 = __ffma2_rn(make_float2(g0.y, g1.y), minus, e1);
          lo[i] = h2_bits(__floats2half2_rn(r0.x, r1.x)), lo[i + 1] = h2_bits(__floats2half2_rn(r0.y, r1.y));
        }
        tmem_st8(tscore + c, hi);
        tmem_st8(tscore + 32 + c, lo);
      }
      l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      tmem_st_wait();
      if (kApart && n > 0) {
        carry();
        if (!ok) break;
      }
      tc_fence_before();
      mbar_arrive(weighed + (n & 1));
    }
    if (!ok) *failed = 1;
    named_bar(3, kTcThreads);  // all products have ended, and all waits
    mbar_wait_short(drained, 0);  // for this thread's order with the products; it does not wait any more
    tc_fence_after();
    if (*failed) {
      ok = false;
      l = NAN;
      if (a.c.status && threadIdx.x == 0) atomicCAS(a.c.status, 0, static_cast<int>(S2_ETIMEOUT));
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
    for (int c = 0; c < HD; c += 16) {
      float o[16] = {};
      __syncwarp();
      if (n > 0) tmem_ld16(tlane + M::kO + c, o);
      if (kApart && n > 1) {
        float before[16];
        tmem_ld16(tlane + M::kBefore + c, before);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] += before[i];
      }
      if (poison >> (c / 32) & 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = NAN;
      if (live && whole) {
        constexpr int kPer = 16 / sizeof(T);
        T* out = static_cast<T*>(a.out) + at * HD + c;
#pragma unroll
        for (int i = 0; i < 16; i += kPer) {
          uint4 u;
          T* e = reinterpret_cast<T*>(&u);
#pragma unroll
          for (int k = 0; k < kPer; ++k) e[k] = from_f<T>(l == 0.f ? 0.f : o[i + k] * inv);
          *reinterpret_cast<uint4*>(out + i) = u;
        }
      } else if (live) {
        float4* out = reinterpret_cast<float4*>(a.part_o + (at * a.n_split + split) * HD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
    }
    if (live && !whole)
      a.part_ml[at * a.n_split + split] = make_float2(lift == 3e38f || !ok ? -INFINITY : kWeightShift - lift, l);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*tbase, M::kCols);
  }
}

// What joins a row's splits: how many of them there are (1 or 0: written by its one block).  For every thread of the
// block, before anything ends.
__device__ __forceinline__ int row_splits(const AttnArgs& a, int row) {
  const int seq = seq_of_row(a.c.q_start, a.c.n_seq, row);
  const bool live = seq < a.c.n_seq && row >= __ldg(a.c.q_start + seq) && __ldg(a.c.q_start + seq + 1) <= a.c.n_rows;
  const int len = live ? min(max(__ldg(a.c.lengths + seq), 0), a.c.table_cols * kPage) : 0;
  pdl_wait();  // no end before the splits'
  return min(((len + kPage - 1) / kPage + a.split_pages - 1) / a.split_pages, a.n_split);
}

// Many splits (more than 16): a block a (row, query head), a thread an element of every fourth of them; the four
// parts are added in order.  One row over 30000 positions: 36 -> 22 us against one part.
constexpr int kJoinParts = 4, kJoinMany = 16;
template <typename T, int HD>
__global__ void __launch_bounds__(HD * kJoinParts) k_kv4_join_many(const AttnArgs a) {
  __shared__ float so[kJoinParts][HD], sl[kJoinParts];
  const int row = blockIdx.x, e = threadIdx.x % HD, part = threadIdx.x / HD;
  const int n = row_splits(a, row);
  if (n <= 1) return;
  const size_t item = static_cast<size_t>(row) * a.n_head + blockIdx.y;
  const float2* ml = a.part_ml + item * a.n_split;
  const float* po = a.part_o + item * a.n_split * HD + e;
  float m = -INFINITY;
  for (int s = threadIdx.x % 32; s < n; s += 32) m = fmaxf(m, __ldcg(&ml[s].x));
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  float o = 0.f, l = 0.f;
#pragma unroll 4
  for (int s = part; s < n; s += kJoinParts) {
    const float2 v = __ldcg(ml + s);
    const float f = ex2(v.x - base);
    l += f * v.y;
    o += f * __ldcg(po + static_cast<size_t>(s) * HD);
  }
  so[part][e] = o;
  if (e == 0) sl[part] = l;
  __syncthreads();
  if (part > 0) return;
  o = l = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinParts; ++i) o += so[i][e], l += sl[i];
  static_cast<T*>(a.out)[item * HD + e] = from_f<T>(l == 0.f ? 0.f : o / l);
}

// Up to 16 splits: a warp a query head, eight heads of a row a block, so that a row with nothing to join costs
// little and one with something has all its heads under way (874 rows, 60 of them split: 23 us -> 6).
template <typename T, int HD>
__global__ void __launch_bounds__(256) k_kv4_join_few(const AttnArgs a) {
  constexpr int E = HD / 32;
  const int row = blockIdx.x, lane = threadIdx.x % 32, h = blockIdx.y * 8 + threadIdx.x / 32;
  const int n = row_splits(a, row);
  if (n <= 1 || h >= a.n_head) return;
  const size_t item = static_cast<size_t>(row) * a.n_head + h;
  const float2 ml = lane < n ? __ldcg(a.part_ml + item * a.n_split + lane) : make_float2(-INFINITY, 0.f);
  const float* po = a.part_o + item * a.n_split * HD + lane;
  const float m = warp_max(ml.x);
  const float f = ex2(ml.x - (m == -INFINITY ? 0.f : m));
  const float l = warp_sum(lane < n ? f * ml.y : 0.f);
  float o[E] = {};
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float w = __shfl_sync(0xffffffffu, f, s);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] += w * __ldcg(po + static_cast<size_t>(s) * HD + 32 * i);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    static_cast<T*>(a.out)[item * HD + lane + 32 * i] = from_f<T>(l == 0.f ? 0.f : o[i] / l);
}

// How a call's work is cut.  The kernel for many columns takes over where a sequence has more than 16 columns on
// average (rows times query heads of a KV head; fp32 queries count twice, and there it is 40).  32 query heads on 8, us
// of the kernel for few and of that for many:
//   sequences x positions      8 x 4000    1 x 30000   32 x 1000   8 x 200
//   bf16 hd 128, 16 columns    38.5 35.9   40.6 34.4   32.4 33.4   13.1 11.5
//                24            48.3 36.5   49.2 34.8   46.6 33.6   15.0 11.9
//   bf16 hd 64,  16            22.2 29.1   26.2 28.4   20.1 27.1    8.6  9.5
//                24            30.3 29.5   31.5 28.8   28.7 27.5    9.7  9.9
//   fp32 hd 128, 32            50.2 60.2   45.1 57.0   48.4 59.0   13.5 12.3
//                48            69.0 61.1   63.2 57.8   71.7 59.8   19.1 13.5
//   fp32 hd 64,  32            30.8 35.0   29.1 33.2   29.1 33.2    8.6 10.3
//                48            42.2 35.3   40.2 34.0   41.8 33.3   10.2 10.6
// Splits, of at least two pages (an even number: they are taken two at a time), at most 128:
//  - few columns: the blocks that the 152 SMs hold at once (4 an SM), twice that where there are many items of what
//    may be different lengths (32 of 512..4096: 32 us against 46);
//  - many columns: the blocks that they hold at once (2 an SM; fp32 queries at head size 128 have one, and two rounds).
//    Two where that gives one, there are few rounds and max_len is 32 pages or more: a sequence much longer than the
//    others is a chain of pages by itself (five pieces, 60 rows over 42 pages and four over 20: 56 us, unsplit 67; 30 rows
//    over 59 and four of 160 over 20: 59, 82).  Lengths are not known here, and where they are alike two splits cost more
//    than they give, the more the shorter (8 x 100 rows over 47 pages: 102 us, unsplit 84; 5 x 200 over 32: 82, 60; 4 x
//    512 over 8: 82, 39).  42 calls of 1 to 16 sequences, geometric means (with one term a weight): split from 32 pages
//    on 44.7 us, never 45.4, always 51.6.
// The workspace is sized for the most splits that any length up to max_len can get, so that it does not shrink with
// a larger max_len.
struct Plan {
  bool many, pairs;
  int tiles, n_split, split_pages;
  size_t o_bytes, bytes;
};
Plan plan(int n_seq, int n_rows, int n_head, int n_kv_head, int head_dim, int max_len, bool two) {
  Plan p{};
  const long long group = n_head / n_kv_head, columns = n_rows * group * (two ? 2 : 1);
  p.many = columns > (two ? 40ll : 16ll) * n_seq;
  p.pairs = two || columns <= 4ll * n_seq;
  const int cols = p.many ? kTcCols : p.pairs ? 4 : 8;
  p.tiles = static_cast<int>(std::min(n_rows * group / cols + n_seq, n_rows * ((group + cols - 1) / cols)));
  const int pages = static_cast<int>((static_cast<long long>(max_len) + kPage - 1) / kPage);
  const long long items = static_cast<long long>(p.tiles) * n_kv_head;
  const long long room = p.many ? 152 * 2 : items < 152 ? 152 * 4 : 152 * 8;
  const long long least = p.many && items < 152 * 4 && pages >= 32 ? 2 : 1;
  const int want = static_cast<int>(std::min(std::max(least, room / items), 128ll));
  p.split_pages = std::max(2, (pages + want - 1) / want);
  p.split_pages += p.split_pages & 1;
  p.n_split = std::max(1, (pages + p.split_pages - 1) / p.split_pages);
  const int most = std::min(want, (pages + 1) / 2);
  if (most > 1) {
    const size_t parts = static_cast<size_t>(n_rows) * n_head * most;
    p.o_bytes = parts * head_dim * 4;
    p.bytes = p.o_bytes + parts * 8;
  }
  return p;
}

template <typename T, int HD>
int launch(const AttnArgs& a, const Plan& p, cudaStream_t st) {
  const dim3 grid(p.tiles, a.c.n_kv_head, p.n_split);
  if (p.many) {
    constexpr int smem = Tc<HD, sizeof(T) == 4 ? 2 : 1>::kBytes;
    if (!allow_smem<k_kv4_tc<T, HD>, smem>()) return S2_ECUDA;
    k_kv4_tc<T, HD><<<grid, kTcThreads, smem, st>>>(a);
  } else {
    constexpr int smem = kDecodeSmem<HD>;
    auto go = [&](auto pairs) {
      if (!allow_smem<k_kv4_decode<T, HD, decltype(pairs)::value>, smem>()) return false;
      k_kv4_decode<T, HD, decltype(pairs)::value><<<grid, 32 * kWarps, smem, st>>>(a);
      return true;
    };
    bool ok;
    if constexpr (sizeof(T) == 4)
      ok = go(std::true_type{});
    else
      ok = p.pairs ? go(std::true_type{}) : go(std::false_type{});
    if (!ok) return S2_ECUDA;
  }
  if (p.n_split > 1) {
    cudaLaunchConfig_t cfg{};
    const bool many = p.n_split > kJoinMany;
    cfg.gridDim = dim3(a.c.n_rows, many ? a.n_head : (a.n_head + 7) / 8);
    cfg.blockDim = dim3(many ? HD * kJoinParts : 256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, many ? k_kv4_join_many<T, HD> : k_kv4_join_few<T, HD>, a) != cudaSuccess)
      return S2_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? S2_OK : S2_ECUDA;
}

// rows * heads stays in 32 bits, so that columns and tiles do
bool bad_sizes(int n_seq, int n_rows, int n_head, int n_kv_head, int head_dim, int max_len) {
  return n_seq < 1 || n_rows < 1 || n_head < 1 || n_head > 65535 || n_kv_head < 1 || n_head % n_kv_head != 0 ||
         (head_dim != 64 && head_dim != 128) || max_len < 0 ||
         static_cast<long long>(n_rows) * n_head + n_seq > 0x3fffffffll;
}

}  // namespace
}  // namespace s2

using namespace s2;

extern "C" int s2_set_wait_limit(int tries) {
  wait_tries.store(tries < 0 ? kWaitTries : tries, std::memory_order_relaxed);
  return S2_OK;
}

extern "C" size_t s2_kv4_attention_workspace(int n_seq, int n_rows, int n_head, int n_kv_head, int head_dim,
                                             int max_len) {
  if (bad_sizes(n_seq, n_rows, n_head, n_kv_head, head_dim, max_len)) return 0;
  if (max_len == 0) max_len = 0x7fffffff;
  // the more of what 16-bit and fp32 queries need
  return std::max(plan(n_seq, n_rows, n_head, n_kv_head, head_dim, max_len, false).bytes,
                  plan(n_seq, n_rows, n_head, n_kv_head, head_dim, max_len, true).bytes);
}

extern "C" int s2_kv4_attention(const s2_kv4* cache, const void* q, int dtype, int n_head, float scale, int max_len,
                                void* out, void* workspace, size_t ws_bytes, CUstream_st* stream) {
  if (kv4_bad_args(cache) || !q || !out || !dtype_bytes(dtype) || !std::isfinite(scale) ||
      bad_sizes(cache->n_seq, cache->n_rows, n_head, cache->n_kv_head, cache->head_dim, max_len))
    return S2_EINVAL;
  if (reinterpret_cast<uintptr_t>(q) % 16 != 0 || reinterpret_cast<uintptr_t>(out) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return S2_EINVAL;
  if (max_len == 0 || max_len > cache->table_cols * kPage) max_len = cache->table_cols * kPage;
  const Plan p = plan(cache->n_seq, cache->n_rows, n_head, cache->n_kv_head, cache->head_dim, max_len, dtype == S2_F32);
  if (p.bytes > 0 && (!workspace || ws_bytes < p.bytes)) return S2_EINVAL;
  AttnArgs a{*cache, q, n_head, n_head / cache->n_kv_head, scale, out, p.n_split, p.split_pages, nullptr, nullptr, 0};
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.o_bytes);
  a.tries = wait_tries.load(std::memory_order_relaxed);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return cache->head_dim == 64 ? launch<T, 64>(a, p, st) : launch<T, 128>(a, p, st);
  });
}
