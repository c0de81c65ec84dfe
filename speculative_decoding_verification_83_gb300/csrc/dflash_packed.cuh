// dflash_packed.cuh -- what the kernels of the attention over packed sequences
// share: a sequence's extent, what a row sees, and the row kernels that go
// through single rows with exact masks.
#pragma once

#include "dflash_paged.cuh"
#include "dflash_train.h"

namespace dflash {

// Sequence b's first row and count; offsets that do not ascend inside [0, tokens]
// are clamped there, so that no index leaves the arrays.
__device__ __forceinline__ void extent(const int32_t* start, int tokens, int b, int& first, int& n, bool& bad) {
  const int s = start[b], e = start[b + 1];
  first = min(max(s, 0), tokens);
  const int last = min(max(e, first), tokens);
  n = last - first;
  bad |= first != s || last != e;
}
// The sequence that holds row t, or -1. (Offsets that do not ascend name any
// sequence; the caller checks the row against its extent.)
__device__ __forceinline__ int sequence_of(const int32_t* start, int B, int t) {
  int lo = 0, hi = B;  // the last b with start[b] <= t
  if (t < start[0] || t >= start[B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// Keys that query i of n sees of m.
__device__ __forceinline__ int seen_keys(int causal, int n, int m, int i) {
  return causal ? min(m, max(0, m - n + i + 1)) : m;
}
// The first query of n that sees key j of m (causal).
__device__ __forceinline__ int first_query(int causal, int n, int m, int j) { return causal ? max(0, j - (m - n)) : 0; }

// A bf16 output's next 8 bits: the rounding's remainder in units of 2^-8 of the
// output's last place, from the two numbers' bit patterns (of one sign). The backward
// pass needs sum dout out more exactly than bf16 outputs give it: with short
// sequences the outputs' rounding would add as much to dq and dk as all else.
__device__ __forceinline__ int8_t low_bits(float y, uint32_t hi) {
  const int d = ((int)(__float_as_uint(y) - (hi << 16)) + 128) >> 8;
  return (int8_t)max(-128, min(127, d));
}
__device__ __forceinline__ float with_low(uint32_t hi, int low) {
  const bool finite = (hi & 0x7f80u) != 0x7f80u;
  return __uint_as_float((hi << 16) + (finite ? (uint32_t)(low * 256) : 0u));
}

// Rows one by one (dflash_packed.cu): every row, or with `redo` those of the tiles
// whose flag is set that hold a value which is not finite.
int launch_rows_forward(const PackedParams& p, int dtype, int head_dim, const uint32_t* redo, void* stream);
int launch_rows_grad(const PackedParams& p, int head_dim, const uint32_t* redo_q, const uint32_t* redo_kv, void* stream);
int launch_delta(const PackedParams& p, int head_dim, void* stream);

}  // namespace dflash
