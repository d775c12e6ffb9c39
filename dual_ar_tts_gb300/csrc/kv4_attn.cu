// Attention over the paged 4-bit cache (see kv4.cuh for the layout):
//   o = sum_t softmax_t(scale * q . k_t) v_t  over the positions t that a row sees,
// in one pass over the cache with the running maximum and sum of the softmax.
//
// Both products are mma.sync.m16n8k16 (fp16 operands, fp32 sums) with the cache as the A operand, which
// is expanded from its codes in registers on the way: tcgen05 would want it in shared or tensor memory
// first, and a row of a decode step brings 4 to 8 columns where its smallest M or N has use for more.
//   S^T[16 positions][8 columns] = K[16][hd] Q^T[hd][8]
//   O^T[hd][8] += V^T[hd][16] P^T[16][8]
// A column is a (row, query head) pair; with fp32 queries it is two, the high and the low fp16 part of the
// query, whose scores are added and whose weights are again split so (a weight then carries 22 bits).
// 16-bit queries are exact in fp16: each row is scaled by a power of two.  Weights are kept as
// 2^6 exp2(s - m), which puts what fp16 drops 2^-30 below the largest.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "convert.cuh"
#include "kv4.cuh"
#include "ptx.cuh"
#include "s2_internal.h"

namespace s2 {
namespace {

constexpr int kStep = 16;       // positions of one pair of products
constexpr int kDepth = 4;       // steps a warp has in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWeightShift = 6.f;

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
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

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

// One step of the cache in shared memory.  Keys are read 16 bytes (a quarter row) a lane, rows packed;
// values a word or two of four rows a lane, rows padded so that the rows of the four lanes of a group
// start 32 bytes apart modulo 128: both without bank conflicts.
template <int HD>
struct Stage {
  using B = Kv4Block<HD>;
  static constexpr int kVRow = B::kRow + 16;
  static constexpr int kK = 0, kKPar = kStep * B::kRow, kV = kKPar + kStep * B::kPar, kVPar = kV + kStep * kVRow;
  static constexpr int kBytes = kVPar + kStep * B::kPar;
};

// a warp's copy of the step at position `slot` of a page block
template <int HD>
__device__ __forceinline__ void copy_step(uint8_t* st, const uint8_t* block, int slot, int lane) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  const uint8_t* k = block + slot * B::kRow;
  const uint8_t* v = k + B::kHalf;
#pragma unroll
  for (int i = lane; i < kStep * B::kRow / 16; i += 32) cp_async16(st + S::kK + i * 16, k + i * 16);
#pragma unroll
  for (int i = lane; i < kStep * B::kRow / 16; i += 32) {
    constexpr int per = B::kRow / 16;
    cp_async16(st + S::kV + i / per * S::kVRow + i % per * 16, v + i * 16);
  }
  constexpr int np = kStep * B::kPar / 16;  // 16 or 8
  const uint8_t* par = block + kPage * B::kRow + slot * B::kPar;
  if (lane < np)
    cp_async16(st + S::kKPar + lane * 16, par + lane * 16);
  else if (lane < 2 * np)
    cp_async16(st + S::kVPar + (lane - np) * 16, par + B::kHalf + (lane - np) * 16);
}

// The query columns of a warp as B operand: lane (g = lane / 4, c = lane % 4) holds column g of each
// group of 8 at the elements that lane c expands of a key row.
template <typename T, int HD>
__device__ __forceinline__ float load_q(const T* q, bool live, bool low, int c, uint32_t (&f)[HD / 8]) {
  constexpr int E = HD / 4;
  float x[E], top = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    x[i] = live ? to_f(q[c * E + i]) : 0.f;
    top = fmaxf(top, fabsf(x[i]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  int e = 0;  // the largest element to 2^13 .. 2^14: exact, and far from fp16's ends
  if (top > 0.f && isfinite(top)) e = min(13 - ilogbf(top), 126);
  const float up = ldexpf(1.f, e);
#pragma unroll
  for (int j = 0; j < E / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = x[8 * j + i] * up, b = x[8 * j + i + 4] * up;
      if (low) {
        a -= round_f16(a);
        b -= round_f16(b);
      }
      f[4 * j + i] = h2_bits(__floats2half2_rn(a, b));
    }
  return ldexpf(1.f, -e);
}

// S^T of one step: scores of rows g, g + 8 at columns 2c, 2c + 1 of each group of 8
template <int HD, int NT>
__device__ __forceinline__ void scores(uint32_t st, int g, int c, const uint32_t (&q)[NT][HD / 8], float (&s)[NT][4]) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int W = HD / 32;  // words of a lane's quarter row
  uint32_t r0[W], r1[W];
  const uint32_t a = st + S::kK + g * B::kRow + c * (HD / 8);
  if constexpr (W == 4) {
    const uint4 x = lds128(a), y = lds128(a + 8 * B::kRow);
    r0[0] = x.x, r0[1] = x.y, r0[2] = x.z, r0[3] = x.w;
    r1[0] = y.x, r1[1] = y.y, r1[2] = y.z, r1[3] = y.w;
  } else {
    const uint2 x = lds64(a), y = lds64(a + 8 * B::kRow);
    r0[0] = x.x, r0[1] = x.y;
    r1[0] = y.x, r1[1] = y.y;
  }
  const uint32_t par = st + S::kKPar + g * B::kPar + c * (HD / 4) / kKvGroup * 4;
  const uint32_t p0 = lds32(par), p1 = lds32(par + 8 * B::kPar);
  const Pair pa(p0, p0), pb(p1, p1);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    uint32_t x[4], y[4];
    expand(r0[j], pa, x);
    expand(r1[j], pb, y);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma_f16_16816(s[n], x[0], y[0], x[1], y[1], q[n][4 * j], q[n][4 * j + 1]);
      mma_f16_16816(s[n], x[2], y[2], x[3], y[3], q[n][4 * j + 2], q[n][4 * j + 3]);
    }
  }
}

// O^T += V^T P^T of one step.  Lane (g, c) expands elements g * hd/8 .. + hd/8 - 1 of rows 2c, 2c + 1, 2c + 8,
// 2c + 9; element 2i of those is row g, element 2i + 1 row g + 8 of the i-th tile.  `valid` rows from the
// step's start are in the sequence; parameters of the others are taken as zero (their weights are zero, but
// what is there may be no number).  Returns whether a parameter is not finite: such rows count as zero here.
template <int HD, int NT>
__device__ __forceinline__ bool values(uint32_t st, int g, int c, int valid, const uint32_t (&p)[NT][2],
                                       float (&o)[NT][HD / 16][4]) {
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int W = HD / 64;  // words of a row that a lane expands
  uint32_t w[4][W], par[4];
  bool odd = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = 2 * c + (k & 1) + (k >> 1) * 8;
    const uint32_t a = st + S::kV + row * S::kVRow + g * (HD / 16);
    if constexpr (W == 2) {
      const uint2 x = lds64(a);
      w[k][0] = x.x, w[k][1] = x.y;
    } else {
      w[k][0] = lds32(a);
    }
    par[k] = lds32(st + S::kVPar + row * B::kPar + g * (HD / 8) / kKvGroup * 4);
    if (row >= valid) par[k] = 0;
    if ((par[k] & 0x7c00u) == 0x7c00u || (par[k] & 0x7c000000u) == 0x7c000000u) {
      odd = true;
      par[k] = 0;
    }
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
      for (int n = 0; n < NT; ++n) {
        mma_f16_16816(o[n][4 * j + 2 * h], x[0], x[1], y[0], y[1], p[n][0], p[n][1]);
        mma_f16_16816(o[n][4 * j + 2 * h + 1], x[2], x[3], y[2], y[3], p[n][0], p[n][1]);
      }
    }
  return odd;
}

// The running state of a warp's columns.  A lane's columns are 2c, 2c + 1 of each group of 8 (with fp32
// queries the two parts of one), the same in the scores and in the output tiles.
template <int HD, int NT, bool kTwo>
struct Rows {
  static constexpr int NC = kTwo ? 1 : 2;  // a lane's logical columns per group of 8
  float o[NT][HD / 16][4];
  float m[NT][NC], l[NT][NC], f[NT][NC];   // maximum (log2 units), this lane's part of the sum, score factor
  int lim[NT][NC];                         // positions seen

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < HD / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j) m[n][j] = -INFINITY, l[n][j] = 0.f;
    }
  }

  // one step at position t0: s becomes the weights, as B operand
  __device__ __forceinline__ void softmax(float (&s)[NT][4], int t0, int g, bool cut, uint32_t (&p)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[2][NC];  // [row g, row g + 8][column]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (kTwo) {
          x[r][0] = (s[n][2 * r] + s[n][2 * r + 1]) * f[n][0];
        } else {
          x[r][0] = s[n][2 * r] * f[n][0];
          x[r][1] = s[n][2 * r + 1] * f[n][1];
        }
        if (cut) {
#pragma unroll
          for (int j = 0; j < NC; ++j)
            if (t0 + g + 8 * r >= lim[n][j]) x[r][j] = -INFINITY;
        }
      }
      float w[2][2];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float top = fmaxf(x[0][j], x[1][j]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float mn = fmaxf(m[n][j], top);
        const float base = mn == -INFINITY ? 0.f : mn - kWeightShift;
        const float keep = ex2(m[n][j] - (mn == -INFINITY ? 0.f : mn));
        m[n][j] = mn;
        w[0][j] = ex2(x[0][j] - base);
        w[1][j] = ex2(x[1][j] - base);
        l[n][j] = l[n][j] * keep + (w[0][j] + w[1][j]);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
          if constexpr (kTwo) {
            o[n][i][0] *= keep, o[n][i][1] *= keep, o[n][i][2] *= keep, o[n][i][3] *= keep;
          } else {
            o[n][i][j] *= keep, o[n][i][2 + j] *= keep;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if constexpr (kTwo) w[r][1] = w[r][0] - round_f16(w[r][0]);
        p[n][r] = movmatrix_trans(h2_bits(__floats2half2_rn(w[r][0], w[r][1])));
      }
    }
  }

  // a value row of the step that is no number: every column that sees it is none either, in its group's elements
  __device__ __forceinline__ void poison(uint32_t st, int t0, int valid, int g) {
    using S = Stage<HD>;
    for (int r = 0; r < valid; ++r) {
      const uint32_t par = lds32(st + S::kVPar + r * Kv4Block<HD>::kPar + g * (HD / 8) / kKvGroup * 4);
      if ((par & 0x7c00u) != 0x7c00u && (par & 0x7c000000u) != 0x7c000000u) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (t0 + r < lim[n][kTwo ? 0 : j % 2]) o[n][i][j] = NAN;
    }
  }

  __device__ __forceinline__ void finish_sums() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 4);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 8);
        l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], 16);
      }
  }
};

// Where a tile of columns lies: its sequence and the first of its columns there.  Tiles are counted over the
// sequences in order; -1 where there are fewer.
struct Tile {
  int seq, first;
};
__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ q_start, int n_seq, int group, int cols, int t) {
  const int lane = threadIdx.x % 32;
  int before = 0;
  for (int base = 0; base < n_seq; base += 32) {
    const int s = base + lane;
    int tiles = 0;
    if (s < n_seq) tiles = (max(__ldg(q_start + s + 1) - __ldg(q_start + s), 0) * group + cols - 1) / cols;
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > t);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return {base + l, (t - before - __shfl_sync(0xffffffffu, upto - tiles, l)) * cols};
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return {-1, 0};
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

// Few columns: a block takes one tile of 8 columns of one KV head over a range of pages.  Warp w takes
// positions 16w .. 16w + 15 of each page with its own copies in flight, so the warps never wait on one
// another until their states are joined.
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_kv4_decode(const AttnArgs a) {
  constexpr bool kTwo = sizeof(T) == 4;
  constexpr int CT = kTwo ? 4 : 8;  // logical columns
  constexpr int kWarps = 4;
  using B = Kv4Block<HD>;
  using S = Stage<HD>;
  constexpr int kORow = HD + 4;  // floats of a column's output in the joining buffer
  constexpr int kRing = kWarps * kDepth * S::kBytes, kJoin = kWarps * CT * (kORow + 2) * 4;
  __shared__ __align__(16) uint8_t sm[kRing > kJoin ? kRing : kJoin];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, c = lane % 4;
  const int kh = blockIdx.y, split = blockIdx.z;
  const Tile tile = find_tile(a.c.q_start, a.c.n_seq, a.group, CT, blockIdx.x);
  if (tile.seq < 0) return;
  const int q0 = __ldg(a.c.q_start + tile.seq), q1 = __ldg(a.c.q_start + tile.seq + 1);
  if (q0 < 0 || q1 > a.c.n_rows) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    return;
  }
  const int cols = (q1 - q0) * a.group;
  int len = __ldg(a.c.lengths + tile.seq);
  const int over = len - (q1 - q0);  // row i sees over + i + 1 positions
  if (len > a.c.table_cols * kPage) {
    if (threadIdx.x == 0) kv4_bad(a.c.status);
    len = a.c.table_cols * kPage;
  }
  len = max(len, 0);
  const int pages = (len + kPage - 1) / kPage;
  const int p0 = split * a.split_pages, p1 = split == a.n_split - 1 ? pages : min(pages, p0 + a.split_pages);
  if (p0 >= p1 && split > 0) return;

  Rows<HD, 1, kTwo> st;
  st.init();
  uint32_t qf[1][HD / 8];
  {
    const int col = tile.first + (kTwo ? g / 2 : g);
    const bool live = col < cols;
    const int row = q0 + (live ? col / a.group : 0), h = kh * a.group + (live ? col % a.group : 0);
    const float down = load_q<T, HD>(static_cast<const T*>(a.q) + (static_cast<size_t>(row) * a.n_head + h) * HD, live,
                                     kTwo && (g & 1), c, qf[0]);
#pragma unroll
    for (int j = 0; j < st.NC; ++j) {
      const int mine = tile.first + (kTwo ? c : 2 * c + j);
      st.f[0][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j)) * a.scale * kLog2e;
      st.lim[0][j] = mine < cols ? min(over + mine / a.group + 1, len) : 0;
    }
  }
  const int first_lim = min(over + tile.first / a.group + 1, len);  // the least that a live column sees

  uint8_t* ring = sm + warp * kDepth * S::kBytes;
  Pages pg{a.c.table + static_cast<size_t>(tile.seq) * a.c.table_cols, pages, a.c.n_pages};
  const uint8_t* heads = static_cast<const uint8_t*>(a.c.pages) + static_cast<size_t>(kh) * B::kBytes;
  uint32_t usable = 0;  // by page modulo 32: copied
  auto issue = [&](int p) {
    if (p < p1) {
      const int id = pg.id(p, a.c.status);
      const bool ok = id >= 0 && p * kPage + warp * kStep < len;
      usable = ok ? usable | 1u << (p & 31) : usable & ~(1u << (p & 31));
      if (ok)
        copy_step<HD>(ring + p % kDepth * S::kBytes, heads + static_cast<size_t>(id) * a.c.n_kv_head * B::kBytes,
                      warp * kStep, lane);
    }
    cp_async_commit();
  };
  for (int i = 0; i < kDepth - 1; ++i) issue(p0 + i);
  for (int p = p0; p < p1; ++p) {
    issue(p + kDepth - 1);
    cp_async_wait_group<kDepth - 1>();
    __syncwarp();
    if (usable >> (p & 31) & 1) {
      const int t0 = p * kPage + warp * kStep;
      const uint32_t at = smem_u32(ring + p % kDepth * S::kBytes);
      float s[1][4];
      uint32_t pf[1][2];
      scores<HD, 1>(at, g, c, qf, s);
      st.softmax(s, t0, g, t0 + kStep > first_lim, pf);
      const int valid = min(len - t0, kStep);
      if (__any_sync(0xffffffffu, values<HD, 1>(at, g, c, valid, pf, st.o))) st.poison(at, t0, valid, g);
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
        dst[2 * i] = st.o[0][i][0] + st.o[0][i][1];
        dst[2 * i + 1] = st.o[0][i][2] + st.o[0][i][3];
      } else {
        dst[2 * i] = st.o[0][i][j];
        dst[2 * i + 1] = st.o[0][i][2 + j];
      }
    }
    if (g == 0) {
      jm[(warp * CT + col) * 2] = st.m[0][j];
      jm[(warp * CT + col) * 2 + 1] = st.l[0][j];
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
    if (a.n_split == 1) {
      static_cast<T*>(a.out)[at * HD + e] = from_f<T>(l == 0.f ? 0.f : o / l);
    } else {
      a.part_o[(at * a.n_split + split) * HD + e] = o;
      if (e == 0) a.part_ml[at * a.n_split + split] = make_float2(m, l);
    }
  }
}

// The splits of each (row, query head), one warp each: their maxima decide the weights of their outputs.
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_kv4_join(const AttnArgs a) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x % 32;
  const long long item = static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int row = static_cast<int>(item / a.n_head);
  if (row >= a.c.n_rows) return;
  const int seq = seq_of_row(a.c.q_start, a.c.n_seq, row);
  if (seq >= a.c.n_seq || row < __ldg(a.c.q_start + seq) || __ldg(a.c.q_start + seq + 1) > a.c.n_rows) return;
  const int len = min(max(__ldg(a.c.lengths + seq), 0), a.c.table_cols * kPage);
  const int pages = (len + kPage - 1) / kPage;
  const int n = min(max((pages + a.split_pages - 1) / a.split_pages, 1), a.n_split);
  const float2* ml = a.part_ml + item * a.n_split;
  const float* po = a.part_o + item * a.n_split * HD + lane * E;
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, __ldcg(&ml[s].x));
  m = warp_max(m);
  const float base = m == -INFINITY ? 0.f : m;
  float o[E] = {}, l = 0.f;
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float2 v = __ldcg(ml + s);
    const float f = ex2(v.x - base);
    l += f * v.y;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] += f * __ldcg(po + s * HD + i);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    static_cast<T*>(a.out)[item * HD + lane * E + i] = from_f<T>(l == 0.f ? 0.f : o[i] / l);
}

// How a call's work is cut.  Splits: enough blocks for twice what the 152 SMs hold at once (4 each), of at
// least two pages, at most 128.  The workspace is sized for the most splits that any length up to max_len can
// get, so that it does not shrink with a larger max_len.
struct Plan {
  int tiles, n_split, split_pages;
  size_t o_bytes, bytes;
};
Plan plan(int n_seq, int n_rows, int n_head, int n_kv_head, int head_dim, int max_len, bool two) {
  Plan p{};
  const int cols = two ? 4 : 8;
  const long long group = n_head / n_kv_head;
  p.tiles = static_cast<int>(std::min(n_rows * group / cols + n_seq, n_rows * ((group + cols - 1) / cols)));
  const int pages = static_cast<int>((static_cast<long long>(max_len) + kPage - 1) / kPage);
  const int want = static_cast<int>(std::min(std::max(1ll, 152 * 8 / (static_cast<long long>(p.tiles) * n_kv_head)), 128ll));
  p.split_pages = std::max(2, (pages + want - 1) / want);
  p.n_split = std::max(1, (pages + p.split_pages - 1) / p.split_pages);
  const int most = std::min(want, (pages + 1) / 2);
  if (most > 1) {
    const size_t items = static_cast<size_t>(n_rows) * n_head * most;
    p.o_bytes = items * head_dim * 4;
    p.bytes = p.o_bytes + items * 8;
  }
  return p;
}

template <typename T, int HD>
int launch(const AttnArgs& a, const Plan& p, cudaStream_t st) {
  k_kv4_decode<T, HD><<<dim3(p.tiles, a.c.n_kv_head, p.n_split), 128, 0, st>>>(a);
  if (p.n_split > 1) {
    const long long warps = static_cast<long long>(a.c.n_rows) * a.n_head;
    k_kv4_join<T, HD><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(a);
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
  AttnArgs a{*cache, q, n_head, n_head / cache->n_kv_head, scale, out, p.n_split, p.split_pages, nullptr, nullptr};
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.o_bytes);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return cache->head_dim == 64 ? launch<T, 64>(a, p, st) : launch<T, 128>(a, p, st);
  });
}
