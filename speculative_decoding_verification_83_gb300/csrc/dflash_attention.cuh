// dflash_attention.cuh -- what the two attention kernels share: the list of
// work, the workspace of partial results, and the kernel that joins them.
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dflash_paged.cuh"

namespace dflash {

constexpr int kMinRun = 4;  // tiles a CTA takes at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// four e4m3 values as two pairs of f16 values
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// A unit of work is (request, key/value head, `rows` query rows) over all of
// the request's keys, `tile` at a time; units follow each other request by
// request, head by head, row block by row block.
//
// The unit that begins in a CTA's run and goes on in the next CTA's (tiles 0:
// there is none). Every split unit has exactly one such CTA.
struct SplitUnit {
  long long start;  // index of its first tile in the whole list
  int tiles, h, rb, first, n, unused;
};

// A row's statistics over some keys: the largest score m (in powers of 2) and
// the sum l of the weights 2^(x - m).
struct Part {
  float m, l;
};

// Workspace: tiles per CTA (64-bit), a SplitUnit for each CTA, then for each
// CTA two slots of partial results: rows x Part, then rows x D. Slot
// 0 is the segment that begins with the CTA's run, slot 1 one that begins
// inside it.
struct AttnGeometry {
  int rows, tile, ctas;
  __host__ __device__ size_t ml() const { return 256 + ((size_t)ctas * sizeof(SplitUnit) + 255) / 256 * 256; }
  __host__ __device__ size_t o() const { return ml() + ((size_t)ctas * 2 * rows * sizeof(Part) + 255) / 256 * 256; }
  __host__ __device__ size_t bytes(int D) const { return o() + (size_t)ctas * 2 * rows * D * sizeof(float); }
};
// Part b, taken to the reference m; a sum that has seen nothing is 0, or NaN.
__device__ __forceinline__ float part_sum(const Part& b, float m) {
  return b.l == b.l ? (b.m == kNegInf ? 0.0f : b.l * ex2(b.m - m)) : b.l;
}
__device__ __forceinline__ float reciprocal_or_zero(float s) { return s > 0.0f ? 1.0f / s : s == 0.0f ? 0.0f : s; }
__device__ __forceinline__ SplitUnit* split_units(const AttnParams& p) {
  return reinterpret_cast<SplitUnit*>(p.ws + 256);
}

__device__ __forceinline__ int clamped_len(const AttnParams& p, int b, bool& bad) {
  const int L = p.lens[b];
  const long long cap = (long long)p.c.max_pages * p.c.page_size;
  const int top = cap < 0x7fffff00LL ? (int)cap : 0x7fffff00;
  const int c = min(max(L, 0), top);
  bad |= c != L;
  return c;
}
template <int kTileKeys>
__device__ __forceinline__ int tiles_of(int L) {
  return max(1, (L + kTileKeys - 1) / kTileKeys);
}
template <int kUnitRows>
__device__ __forceinline__ int row_blocks(int n, int G) {
  return (int)(((long long)n * G + kUnitRows - 1) / kUnitRows);
}

// ---- values that are not finite (never met in sound data)
// A weight of 0 times such a value would be NaN, for rows that do not see it and
// for rows that see it at a weight below the range of the weights' type. So tiles
// that only some rows see in full have these values replaced by 0 before the
// product, and a unit in which one was replaced, or whose results are not
// finite, is gone through once more: for each column, the first key whose
// value there is +inf, -inf or NaN. A row that sees one of them (at any weight)
// has that as its result, or NaN where it sees infinities of both signs.
constexpr int kNever = 0x7fffffff;

template <class T>
__device__ __forceinline__ bool word_not_finite(uint32_t w) {
  constexpr uint32_t e = std::is_same<T, F16>::value ? 0x7c00u : 0x7f80u;
  return (w & e) == e || ((w >> 16) & e) == e;
}
// e4m3 NaNs (all ones below the sign), or 16-bit values that are not finite, of
// a word become 0; whether there were any
template <class T, bool kF8>
__device__ __forceinline__ bool drop_not_finite(uint32_t& w) {
  bool found = false;
  if (kF8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (((w >> (8 * i)) & 0x7fu) == 0x7fu) {
        w &= ~(0xffu << (8 * i));
        found = true;
      }
  } else if (word_not_finite<T>(w)) {
    constexpr uint32_t e = std::is_same<T, F16>::value ? 0x7c00u : 0x7f80u;
    if ((w & e) == e) w &= 0xffff0000u;
    if (((w >> 16) & e) == e) w &= 0xffffu;
    found = true;
  }
  return found;
}

__device__ __forceinline__ void note(int* first, int key) {
  if (key < *first) atomicMin(first, key);  // (a cache of nothing else meets the atomic rarely)
}
// first[c * D + d]: the first key of [k0, k1) of request b and head h whose value
// d is +inf (c = 0), -inf (1) or NaN (2). `threads` threads share the work.
template <class T, bool kF8, int D>
__device__ __noinline__ void find_not_finite(const AttnParams& p, int b, int h, int k0, int k1, int* first, int tid,
                                             int threads) {
  constexpr int kPieces = (kF8 ? D : 2 * D) / 16, kBatch = 4;
  const long long n = (long long)(k1 - k0) * kPieces;
  for (long long i0 = tid; i0 < n; i0 += (long long)kBatch * threads) {
    int key[kBatch], id[kBatch], slot[kBatch];
    uint4 w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long i = i0 + (long long)j * threads;
      key[j] = k0 + (int)(i / kPieces);
      id[j] = -1;
      if (i >= n) continue;
      int page;
      split_position(p.c, key[j], page, slot[j]);
      id[j] = p.c.table[(long long)b * p.c.table_stride + page];
    }
    const int c = (int)(i0 % kPieces);  // (threads is a multiple of kPieces)
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (id[j] >= 0 && id[j] < p.c.num_pages)
        w[j] = *reinterpret_cast<const uint4*>(p.c.v + ((size_t)row_offset(p.c, id[j], h, slot[j]) + c) * 16u);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t word[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (kF8) {
          for (int k = 0; k < 4; ++k)
            if (((word[e] >> (8 * k)) & 0x7fu) == 0x7fu) note(first + 2 * D + 16 * c + 4 * e + k, key[j]);
        } else if (word_not_finite<T>(word[e])) {
          const float2 f = T::unpack(word[e]);
          const float v[2] = {f.x, f.y};
          for (int k = 0; k < 2; ++k)
            if (!(fabsf(v[k]) < INFINITY))
              note(first + (v[k] > 0.0f ? 0 : v[k] < 0.0f ? 1 : 2) * D + 8 * c + 2 * e + k, key[j]);
        }
      }
    }
  }
}
// Column d of a row that sees the keys before `vis`: 0 where its sum decides.
template <int D>
__device__ __forceinline__ float not_finite_value(const int* first, int d, int vis) {
  const bool pos = first[d] < vis, neg = first[D + d] < vis, nan = first[2 * D + d] < vis;
  return nan || (pos && neg) ? NAN : pos ? INFINITY : neg ? -INFINITY : 0.0f;
}

// Joins the partial results of the units that span CTAs, and writes their rows.
// grid: the CTAs of the kernel before it.
int launch_join(const AttnParams& p, const AttnGeometry& g, int grid, int dtype, bool f8, int head_dim, void* stream);

// The tensor-memory kernel (dflash_attention_tc.cu): units of 32, 64 or 128 rows.
AttnGeometry tc_geometry(int rows, int head_dim);
int launch_attention_tc(const AttnParams& p, int rows, int dtype, bool f8, int head_dim, int sms, void* stream);

}  // namespace dflash
