// dflash_packed_mma.cuh -- what the tensor cores' kernels of the attention over
// packed sequences share: bounded waits, pairs of fp32 operations, tensor maps.
#pragma once

#include <cmath>

#include "dflash_packed.cuh"
#include "dflash_tcgen05.cuh"

namespace dflash {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0u && (*failed || global_timer_ns() - t0 > kWaitLimitNs)) {
      *failed = 1;
      return false;
    }
  }
}
// The same for a warp: its lanes go on or give up together, since shuffles and
// votes of the whole warp follow.
__device__ __forceinline__ bool bounded_warp_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, failed));
}

// Two barriers in the time of one: every other lane looks at the second.
__device__ __forceinline__ bool bounded_warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* failed) {
  const bool second = threadIdx.x & 1;
  const bool ok = __all_sync(0xffffffffu, bounded_wait(second ? b : a, second ? pb : pa, failed));
  __syncwarp();
  return ok;
}

// A CTA's units: every gridDim-th of the list, in turn from either end of a round,
// since the list begins with the largest.
__device__ __forceinline__ int unit_of(int round) {
  return round * (int)gridDim.x + (int)(round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
// Two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Inside each group of P lanes, lane t holds the P 16-byte pieces of row t (piece q in
// words 4q .. 4q + 3); afterwards it holds piece t of the group's row i in words 4i ..
// 4i + 3, so that a store's lanes write neighbouring pieces of a few rows.
template <int P>
__device__ __forceinline__ void transpose_pieces(uint32_t (&w)[4 * P], int lane) {
#pragma unroll
  for (int m = P / 2; m > 0; m >>= 1) {
    const bool hi = (lane & m) != 0;
#pragma unroll
    for (int a = 0; a < P; ++a) {
      if (a & m) continue;
      const int b = a | m;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? w[4 * a + e] : w[4 * b + e], m);
        if (hi)
          w[4 * a + e] = got;
        else
          w[4 * b + e] = got;
      }
    }
  }
}
// Writes a warp's 32 rows, P pieces of 16 bytes each (lane t's are row t's), to
// dst + row * stride; rows from `rows` on are left out.
template <int P>
__device__ __forceinline__ void store_rows(uint32_t (&w)[4 * P], unsigned char* dst, long long stride, int rows, int lane) {
  transpose_pieces<P>(w, lane);
  const int r0 = lane & ~(P - 1), t = lane & (P - 1);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (r0 + i < rows)
      *reinterpret_cast<uint4*>(dst + (r0 + i) * stride + 16 * t) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// A [tokens, heads, head_dim] array in boxes of `rows` tokens x 64 values of one head.
inline bool map_heads(CUtensorMap* map, bool bf16, const HeadRows& h, int tokens, int heads, int head_dim, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)h.hs * 2u, (cuuint64_t)h.ts * 2u};
  const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)rows};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, h.p, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dflash
