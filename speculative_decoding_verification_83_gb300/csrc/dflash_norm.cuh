// dflash_norm.cuh -- the norm of a head's values, shared by the paged append and
// by the norms with rotation of whole batches. D / 16 neighbouring lanes hold a
// head, two vectors of 8 values each.
#pragma once

#include "dflash_paged.cuh"

namespace dflash {

template <class T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = T::unpack(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7]));
}
// Weights 8 vec .. 8 vec + 7, in the tokens' type or in fp32; 1 where there are none.
template <class T>
__device__ __forceinline__ void weight8(const void* w, bool f32, int vec, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.0f;
  } else if (f32) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * vec], b = reinterpret_cast<const float4*>(w)[2 * vec + 1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    unpack8<T>(reinterpret_cast<const uint4*>(w)[vec], x);
  }
}
// The sum over a head's kLanes lanes, which are all in the call.
template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t mask = (uint32_t)((1ull << kLanes) - 1ull) << (lane & ~(uint32_t)(kLanes - 1));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o);
  return v;
}
// The angle of a pair as (cosine, sine): phase holds turns per token as a 64-bit
// binary fraction, so that the product modulo 2^64 is the fraction of a turn at
// any position; its upper 32 bits are a signed number of half turns.
__device__ __forceinline__ float2 turn_at(unsigned long long phase, int pos) {
  const unsigned long long a = phase * (unsigned long long)(long long)pos;
  float s, c;
  sincospif((float)(int32_t)(uint32_t)(a >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}
// Turns a lane's 8 pairs: between its vectors (split), or neighbours inside them.
// The pairs' angles lie `step` apart; back: by the opposite angle.
__device__ __forceinline__ void turn_pairs(float (&a)[8], float (&b)[8], const float2* tn, int step, bool split, bool back) {
  const float sign = back ? -1.0f : 1.0f;
  if (split) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 cs = tn[e * step];
      const float s = sign * cs.y, r = a[e] * cs.x - b[e] * s, o = b[e] * cs.x + a[e] * s;
      a[e] = r;
      b[e] = o;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 cs = tn[e * step], ct = tn[(4 + e) * step];
      const float s = sign * cs.y, t = sign * ct.y;
      const float r = a[2 * e] * cs.x - a[2 * e + 1] * s, o = a[2 * e + 1] * cs.x + a[2 * e] * s;
      a[2 * e] = r;
      a[2 * e + 1] = o;
      const float r2 = b[2 * e] * ct.x - b[2 * e + 1] * t, o2 = b[2 * e + 1] * ct.x + b[2 * e] * t;
      b[2 * e] = r2;
      b[2 * e + 1] = o2;
    }
  }
}

}  // namespace dflash
