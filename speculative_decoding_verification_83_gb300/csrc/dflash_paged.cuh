// dflash_paged.cuh -- device-side addressing shared by the paged-cache kernels.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/dflash_verify.h"
#include "dflash_device.cuh"
#include "dflash_ops.h"

namespace dflash {

__device__ __forceinline__ void raise_status(uint32_t* status, uint32_t bits) {
  if (status) atomicOr(status, bits);
}

// Request b's first packed token and its count; offsets that do not ascend
// inside [0, tokens] are clamped there, so that no index leaves the arrays.
__device__ __forceinline__ void request_tokens(const PackedTokens& t, int b, int& first, int& n, bool& bad) {
  if (!t.q_start) {
    first = b * t.q_per;
    n = t.q_per;
    return;
  }
  const int s = t.q_start[b], e = t.q_start[b + 1];
  first = min(max(s, 0), t.tokens);
  const int last = min(max(e, first), t.tokens);
  n = last - first;
  bad |= first != s || last != e;
}

// Page index and slot of a position.
__device__ __forceinline__ void split_position(const PagedView& c, int pos, int& page, int& slot) {
  if (c.page_shift >= 0) {
    page = pos >> c.page_shift;
    slot = pos & (c.page_size - 1);
  } else {
    page = pos / c.page_size;
    slot = pos - page * c.page_size;
  }
}

// Offset of (page, head, slot)'s row of head_dim values, in 16-byte units.
__device__ __forceinline__ uint32_t row_offset(const PagedView& c, int page, int head, int slot) {
  return (uint32_t)page * c.page_s + (uint32_t)head * c.head_s + (uint32_t)slot * c.slot_s;
}

// ---- 16-bit types ---------------------------------------------------------------------
struct Bf16 {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
struct F16 {
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

}  // namespace dflash
