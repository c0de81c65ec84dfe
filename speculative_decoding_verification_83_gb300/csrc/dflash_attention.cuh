// dflash_attention.cuh -- what the two attention kernels share: the list of
// work, the workspace of partial results, and the kernel that joins them.
#pragma once

#include <cmath>
#include <cstdint>

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

// Joins the partial results of the units that span CTAs, and writes their rows.
// grid: the CTAs of the kernel before it.
int launch_join(const AttnParams& p, const AttnGeometry& g, int grid, int dtype, bool f8, int head_dim, void* stream);

// The tensor-memory kernel (dflash_attention_tc.cu): units of 32, 64 or 128 rows.
AttnGeometry tc_geometry(int rows, int head_dim);
int launch_attention_tc(const AttnParams& p, int rows, int dtype, bool f8, int head_dim, int sms, void* stream);

}  // namespace dflash
