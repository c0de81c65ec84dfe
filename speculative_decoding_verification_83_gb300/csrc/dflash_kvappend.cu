// dflash_kvappend.cu -- new tokens' keys and values into a paged cache, keys
// (and queries) rotated to their positions on the way.
//
// Token i of request b stands at position n = lens[b] + i. The pair (x, y) of
// rotated values number j becomes (x cos a - y sin a, y cos a + x sin a),
// a = n w_j. The pair is (x_j, x_{j + rot/2}), or (x_{2j}, x_{2j+1}) when
// interleaved; values past rot are copied. The angle is taken modulo one turn
// in integers: phases[j] is w_j / 2 pi as a 64-bit binary fraction, so that
// n * phases[j] modulo 2^64 is the fraction of a turn with an error of n
// 2^-65, whatever the position, without 64-bit floating point; its upper 32
// bits, as a signed number of half turns in [-1, 1), go to sincospif.
// Everything is fp32 until the one rounding to the stored type (e4m3: the
// value over its head's scale, saturated at +-448).
#include <cuda_runtime.h>

#include <cstdint>

#include "dflash_paged.cuh"

namespace dflash {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

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

// 8 values to a cache row (16-byte units from base), at value 8 * vec
template <class T, bool kF8>
__device__ __forceinline__ void store_cache(unsigned char* base, uint32_t row, int vec, const float (&x)[8],
                                            float scale) {
  unsigned char* p = base + (size_t)row * 16u;
  if (kF8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)e4m3_pair(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
             (uint32_t)e4m3_pair(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16;
    reinterpret_cast<uint2*>(p)[vec] = make_uint2(w[0], w[1]);
  } else {
    reinterpret_cast<uint4*>(p)[vec] = pack8<T>(x);
  }
}

// One token per blockIdx.x; the token's work is split over blockIdx.y. A work
// item is one pair of 8-value vectors (v and v + D/16) of one head: heads of
// k, then v, then q. Half-split rotation with rot == D pairs the two vectors;
// with rot < D the pairing is inside the first rot values, so the item's
// vectors are chosen by the caller (vector_pair).
template <class T, bool kF8, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  constexpr int kItems = D / 16;  // vector pairs per head
  __shared__ float2 turn[D / 2];
  grid_dependency_sync();
  const int t = blockIdx.x;
  const int half = p.rot >> 1;
  const int b = request_of_token(p.tk, t);
  if (b < 0 || b >= p.tk.B) return;
  int first, n;
  bool bad = false;
  request_tokens(p.tk, b, first, n, bad);
  if (t < first || t >= first + n) return;
  const int len = p.lens[b];
  // positions stay inside the page table's row
  const long long pos64 = (long long)len + (t - first);
  const long long cap = (long long)p.c.max_pages * p.c.page_size;
  if (len < 0 || pos64 >= cap || pos64 > 0x7fffffffLL) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
    return;
  }
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
  const int pos = (int)pos64;
  int page, slot;
  split_position(p.c, pos, page, slot);
  const int id = p.c.table[(long long)b * p.c.table_stride + page];
  const bool have_page = id >= 0 && id < p.c.num_pages;
  if (!have_page && threadIdx.x == 0 && blockIdx.y == 0) raise_status(p.status, DFLASH_STATUS_BAD_PAGE);
  for (int j = threadIdx.x; j < half; j += kAppendThreads) {
    const unsigned long long a = p.phases[j] * (unsigned long long)pos;
    float s, c;
    sincospif((float)(int32_t)(uint32_t)(a >> 32) * 0x1p-31f, &s, &c);
    turn[j] = make_float2(c, s);
  }
  __syncthreads();

  const int heads = 2 * p.c.kv_heads + (p.q ? p.q_heads : 0);
  const int items = heads * kItems;
  for (int w = blockIdx.y * kAppendThreads + threadIdx.x; w < items; w += gridDim.y * kAppendThreads) {
    const int hd = w / kItems, i = w % kItems;
    const bool is_k = hd < p.c.kv_heads, is_v = !is_k && hd < 2 * p.c.kv_heads;
    const int head = is_k ? hd : is_v ? hd - p.c.kv_heads : hd - 2 * p.c.kv_heads;
    const unsigned char* src =
        is_k ? p.k + 2 * ((long long)t * p.k_ts + (long long)head * p.k_hs)
             : is_v ? p.v + 2 * ((long long)t * p.v_ts + (long long)head * p.v_hs)
                    : p.q + 2 * ((long long)t * p.q_ts + (long long)head * p.q_hs);
    // the item's two vectors: a rotated pair (i < rot/16), else two of the
    // rest, which are copied
    const int rv = p.rot / 16;
    int va, vb;
    if (!p.interleaved && i < rv) {
      va = i;
      vb = i + rv;
    } else if (!p.interleaved) {
      va = 2 * rv + 2 * (i - rv);
      vb = va + 1;
    } else {
      va = 2 * i;
      vb = 2 * i + 1;
    }
    float x[8], y[8];
    unpack8<T>(reinterpret_cast<const uint4*>(src)[va], x);
    unpack8<T>(reinterpret_cast<const uint4*>(src)[vb], y);
    if (!is_v && i < rv) {
      if (!p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 cs = turn[8 * i + e];
          const float a = x[e] * cs.x - y[e] * cs.y, o = y[e] * cs.x + x[e] * cs.y;
          x[e] = a;
          y[e] = o;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 cs = turn[8 * i + e], ct = turn[8 * i + 4 + e];
          const float a = x[2 * e] * cs.x - x[2 * e + 1] * cs.y, o = x[2 * e + 1] * cs.x + x[2 * e] * cs.y;
          x[2 * e] = a;
          x[2 * e + 1] = o;
          const float a2 = y[2 * e] * ct.x - y[2 * e + 1] * ct.y, o2 = y[2 * e + 1] * ct.x + y[2 * e] * ct.y;
          y[2 * e] = a2;
          y[2 * e + 1] = o2;
        }
      }
    }
    if (is_k || is_v) {
      if (have_page) {
        const uint32_t row = row_offset(p.c, id, head, slot);
        const float* sc = is_k ? p.c.k_scale : p.c.v_scale;
        const float z = kF8 && sc ? sc[head] : 1.0f;
        unsigned char* base = is_k ? p.c.k : p.c.v;
        store_cache<T, kF8>(base, row, va, x, z);
        store_cache<T, kF8>(base, row, vb, y, z);
      }
    } else {
      uint4* dst = reinterpret_cast<uint4*>(p.q_out + 2 * ((long long)t * p.qo_ts + (long long)head * p.qo_hs));
      dst[va] = pack8<T>(x);
      dst[vb] = pack8<T>(y);
    }
  }
}

template <class T, bool kF8, int D>
int launch(const AppendParams& p, void* stream) {
  const int items = (2 * p.c.kv_heads + (p.q ? p.q_heads : 0)) * (D / 16);
  int split = (items + kAppendThreads - 1) / kAppendThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.tk.tokens, (unsigned)split);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, append_kernel<T, kF8, D>, p);
}

template <class T, bool kF8>
int pick_dim(const AppendParams& p, int d, void* stream) {
  return d == 64 ? launch<T, kF8, 64>(p, stream) : d == 128 ? launch<T, kF8, 128>(p, stream) : launch<T, kF8, 256>(p, stream);
}

}  // namespace

int launch_kv_append(const AppendParams& p, int dtype, int cache_dtype, int head_dim, void* stream) {
  const bool f8 = cache_dtype == DFLASH_E4M3;
  if (dtype == DFLASH_BF16)
    return f8 ? pick_dim<Bf16, true>(p, head_dim, stream) : pick_dim<Bf16, false>(p, head_dim, stream);
  return f8 ? pick_dim<F16, true>(p, head_dim, stream) : pick_dim<F16, false>(p, head_dim, stream);
}

}  // namespace dflash
