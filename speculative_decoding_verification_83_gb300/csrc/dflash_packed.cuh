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

// ---- units of work: a run of rows of one sequence, for each head
struct PackedUnit {
  int row0, rows;  // the unit's first row in its array, its rows
  int i0, n;       // that row's place in its sequence, the sequence's rows
  int other0, m;   // the sequence's rows in the other array: keys of queries, queries of keys
  int unused0, unused1;
};
// The list of the tiles of `rows` queries (or keys), those with the most work first;
// the first word counts them.
struct PackedList {
  int* count;
  PackedUnit* units;
};
__host__ __device__ inline int most_units(int tokens, int B, int rows) { return tokens / rows + (B < tokens ? B : tokens); }
inline size_t list_bytes(int tokens, int B, int rows) {
  return 256 + ((size_t)most_units(tokens, B, rows) * sizeof(PackedUnit) + 255) / 256 * 256;
}
inline PackedList list_at(unsigned char* p) { return {reinterpret_cast<int*>(p), reinterpret_cast<PackedUnit*>(p + 256)}; }

// The tensor cores' kernels leave rows whose masked keys or queries hold values that
// are not finite as NaN (0 times such a value), and a flag for 32 rows with a result that is
// not finite, two or four for each 32 rows (parts of the columns). These kernels go through the flagged rows
// one by one, with exact masks, and set the rows of no sequence to 0.
int launch_redo_forward(const PackedParams& p, int dtype, int head_dim, const PackedList& list, const uint8_t* flags,
                        void* stream);

// The products (dflash_packed_fwd.cu, dflash_packed_bwd.cu).
int launch_forward_tc(const PackedParams& p, int dtype, int head_dim, const PackedList& list, uint8_t* flags, int sms,
                      void* stream);
int launch_dq_tc(const PackedParams& p, int head_dim, const PackedList& list, uint8_t* flags, int sms, void* stream);
// (behind_dq: the kernel before it in the stream is the queries', whose results it does not read)
int launch_dkv_tc(const PackedParams& p, int head_dim, const PackedList& list, uint8_t* flags, bool behind_dq, int sms,
                  void* stream);
constexpr int kForwardRows = 256, kGradRows = 128;  // of a unit
constexpr int kForwardFlags = kForwardRows / 16, kGradFlags = kGradRows / 8;  // of a unit and head
constexpr int kMaxBatch = 2048;

}  // namespace dflash
