// The paged 4-bit key/value cache: layout and the rows of a call.
//
// A page holds 64 positions.  Per KV head it is one block: key codes [64][hd / 2] bytes (low nibble =
// even element), key parameters [64][hd / 32] of {fp16 scale, fp16 zero point}, then the same of the
// values.  An element stands for fp16(scale * (code - zero)), the zero point a whole number in -127..127.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/s2frame.h"

namespace s2 {

constexpr int kPage = S2_KV4_PAGE;
constexpr int kKvGroup = 32;         // elements that share a scale and a zero point
constexpr float kKvMax = 57344.f;    // values beyond are held as this: 8 steps of the widest scale stay below fp16's maximum

template <int HD>
struct Kv4Block {
  static constexpr int kRow = HD / 2;                 // code bytes of a position
  static constexpr int kPar = HD / kKvGroup * 4;      // parameter bytes of a position
  static constexpr int kHalf = kPage * (kRow + kPar); // keys or values
  static constexpr int kBytes = 2 * kHalf;
};

// sequence of row i: the count of sequences that end at or before it (the warp's lanes look at 32 at a time)
__device__ __forceinline__ int seq_of_row(const int32_t* __restrict__ q_start, int n_seq, int i) {
  int s = 0;
  for (int base = 0; base < n_seq; base += 32) {
    const int j = base + static_cast<int>(threadIdx.x % 32);
    const unsigned done = __ballot_sync(0xffffffffu, j < n_seq && __ldg(q_start + j + 1) <= i);
    s += __popc(done);
    if (done != 0xffffffffu) break;
  }
  return s;
}

__device__ __forceinline__ void kv4_bad(int32_t* status) {
  if (status) atomicCAS(status, 0, static_cast<int>(S2_EINVAL));
}

inline bool kv4_bad_args(const s2_kv4* c) {
  if (!c || !c->pages || !c->table || !c->q_start || !c->lengths) return true;
  if (c->n_pages < 1 || c->n_kv_head < 1 || (c->head_dim != 64 && c->head_dim != 128) || c->table_cols < 1 ||
      c->n_seq < 1 || c->n_rows < 1)
    return true;
  if (c->table_cols > 0x7fffffff / kPage || c->n_kv_head > 65535) return true;
  return reinterpret_cast<uintptr_t>(c->pages) % 16 != 0 || reinterpret_cast<uintptr_t>(c->table) % 4 != 0 ||
         reinterpret_cast<uintptr_t>(c->q_start) % 4 != 0 || reinterpret_cast<uintptr_t>(c->lengths) % 4 != 0 ||
         reinterpret_cast<uintptr_t>(c->status) % 4 != 0;
}

}  // namespace s2
