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
//
// What bounds it: reading and writing each value once; for few tokens the launch
// and the chain of offset, length, page and slot. So a block reads its values
// first and finds out where they go while they arrive. Measured on one GB300:
// 10223 tokens of 40 query and 8 key/value heads of 128 into an e4m3 cache, half
// of each head rotated, 52 us (5.2 TB/s, 78% of a copy's rate), where one token a
// block, read after its place was known, took 75 us, and two divisions an item 62
// us. Four items a thread are best there (two 51 us, eight 57 us).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dflash_paged.cuh"

namespace dflash {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxGroup = 8;  // tokens per block

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

// A head's scale z, and two reciprocals with the true one between them. Rounding
// is monotonic: where a value's products with both round to the same e4m3 value,
// so does its quotient; elsewhere (about one value in 2^18) it is divided.
// Dividing every value takes 55 us where this takes 52 (the case above).
struct Scale {
  float z, low, high;
};
__device__ __forceinline__ Scale make_scale(float z) {
  const float inv = __frcp_rn(z);
  // no reciprocal with all its bits: 0 and infinity round apart, and all is divided
  if (!(fabsf(inv) >= 0x1p-126f && fabsf(inv) < INFINITY)) return {z, 0.0f, INFINITY};
  // a power of 2 has its own
  if ((__float_as_uint(z) & 0x7fffffu) == 0u) return {z, inv, inv};
  return {z, inv * (1.0f - 0x1p-22f), inv * (1.0f + 0x1p-22f)};
}
__device__ __forceinline__ uint32_t e4m3_4(const float (&x)[8], int i, float f) {
  return (uint32_t)e4m3_pair(x[i] * f, x[i + 1] * f) | (uint32_t)e4m3_pair(x[i + 2] * f, x[i + 3] * f) << 16;
}

// 8 values (e4m3: over the head's scale) to a cache row (16-byte units from base),
// at value 8 * vec
template <class T, bool kF8>
__device__ __forceinline__ void store_cache(unsigned char* base, uint32_t row, int vec, const float (&x)[8],
                                            const Scale& s) {
  unsigned char* p = base + (size_t)row * 16u;
  if (kF8) {
    uint32_t w[2] = {e4m3_4(x, 0, s.low), e4m3_4(x, 4, s.low)};
    if (__builtin_expect((w[0] ^ e4m3_4(x, 0, s.high)) | (w[1] ^ e4m3_4(x, 4, s.high)), 0)) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = (uint32_t)e4m3_pair(x[4 * i] / s.z, x[4 * i + 1] / s.z) |
               (uint32_t)e4m3_pair(x[4 * i + 2] / s.z, x[4 * i + 3] / s.z) << 16;
    }
    reinterpret_cast<uint2*>(p)[vec] = make_uint2(w[0], w[1]);
  } else {
    reinterpret_cast<uint4*>(p)[vec] = pack8<T>(x);
  }
}

// Where a token goes.
struct Place {
  int pos;   // -1: nowhere (it belongs to no request, or its position is bad)
  int page;  // -1: its page is bad
  int slot;
};

// The request that holds packed token t, by one warp: each round looks at 32
// evenly spaced offsets.
__device__ __forceinline__ int request_of_token_warp(const PackedTokens& k, int t) {
  if (!k.q_start) return t / k.q_per;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = k.B;  // the first b with q_start[b] > t is in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const uint32_t over = __ballot_sync(0xffffffffu, at >= hi || k.q_start[at] > t);
    const int f = over ? __ffs(over) - 1 : 32;  // the first place that lies beyond t
    const int new_hi = f < 32 ? min(hi, lo + f * step) : hi;
    lo = f > 0 ? lo + (f - 1) * step + 1 : lo;
    hi = f > 0 ? new_hi : lo;
  }
  return lo - 1;
}

// A block takes `group` tokens and 256 kBatch of their work items; blockIdx.y
// numbers its share. A work item is one pair of 8-value vectors of one head
// (heads of k, then v, then q): the two halves of rotated pairs, or two
// neighbours. The items' values are read before it is known where they go, so
// that the chain of offset, length, page and slot costs no time of its own.
template <class T, bool kF8, int D, int kBatch>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p, int group, uint32_t inv_items) {
  constexpr int kItems = D / 16;  // vector pairs per head
  __shared__ Place place[kMaxGroup];
  __shared__ float2 turn[kMaxGroup * D / 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_sync();
  const int t0 = blockIdx.x * group, nt = min(group, p.tk.tokens - t0);
  const int half = p.rot >> 1, rv = p.rot >> 4;
  const int heads = 2 * p.c.kv_heads + p.q_heads, items = heads * kItems;
  auto token_of = [&](int w) { return (int)__umulhi((uint32_t)w, inv_items); };  // w / items

  // ---- the values
  uint4 x[kBatch], y[kBatch];
#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int w = (blockIdx.y * kBatch + k) * kAppendThreads + tid;
    if (w >= nt * items) continue;
    const int ti = token_of(w), hd = (w - ti * items) / kItems, i = w % kItems;
    const long long t = t0 + ti;
    const unsigned char* src = hd < p.c.kv_heads       ? p.k + 2 * (t * p.k_ts + (long long)hd * p.k_hs)
                               : hd < 2 * p.c.kv_heads ? p.v + 2 * (t * p.v_ts + (long long)(hd - p.c.kv_heads) * p.v_hs)
                                                       : p.q + 2 * (t * p.q_ts + (long long)(hd - 2 * p.c.kv_heads) * p.q_hs);
    const bool split = !p.interleaved && i < rv;
    const int va = p.interleaved || i >= rv ? 2 * i : i, vb = split ? i + rv : va + 1;
    x[k] = reinterpret_cast<const uint4*>(src)[va];
    y[k] = reinterpret_cast<const uint4*>(src)[vb];
  }

  // ---- where the tokens go, and their angles
  for (int ti = warp; ti < nt; ti += kAppendThreads / 32) {
    const int t = t0 + ti, b = request_of_token_warp(p.tk, t);
    Place pl = {-1, -1, 0};
    uint32_t bits = 0;
    if (b >= 0 && b < p.tk.B) {
      int first, n;
      bool bad = false;
      request_tokens(p.tk, b, first, n, bad);
      if (t >= first && t < first + n) {
        const int len = p.lens[b];
        // positions stay inside the page table's row
        const long long pos = (long long)len + (t - first), cap = (long long)p.c.max_pages * p.c.page_size;
        if (bad) bits |= DFLASH_STATUS_BAD_LENGTH;
        if (len < 0 || pos >= cap || pos > 0x7fffffffLL) {
          bits |= DFLASH_STATUS_BAD_LENGTH;
        } else {
          int page;
          pl.pos = (int)pos;
          split_position(p.c, pl.pos, page, pl.slot);
          const int id = p.c.table[(long long)b * p.c.table_stride + page];
          if (id >= 0 && id < p.c.num_pages)
            pl.page = id;
          else
            bits |= DFLASH_STATUS_BAD_PAGE;
        }
      }
    }
    if (lane == 0) {
      place[ti] = pl;
      if (bits && blockIdx.y == 0) raise_status(p.status, bits);
    }
    for (int j = lane; j < half; j += 32) {
      const unsigned long long a = p.phases[j] * (unsigned long long)(unsigned)pl.pos;
      float s, c;
      sincospif((float)(int32_t)(uint32_t)(a >> 32) * 0x1p-31f, &s, &c);
      turn[ti * half + (j & 7) * rv + (j >> 3)] = make_float2(c, s);  // an item's 8 pairs, rv apart
    }
  }
  // Offsets and lengths that no token meets are reported, too: by one block,
  // beginning with the warps that have no token to place.
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0) {
    const long long cap = (long long)p.c.max_pages * p.c.page_size;
    bool bad = false;
    for (int b = kAppendThreads - 1 - tid; b < p.tk.B; b += kAppendThreads) {
      int first, n;
      request_tokens(p.tk, b, first, n, bad);
      bad |= p.lens[b] < 0 || p.lens[b] > cap;
    }
    if (bad) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < kBatch; ++k) {
    const int w = (blockIdx.y * kBatch + k) * kAppendThreads + tid;
    if (w >= nt * items) continue;
    const int ti = token_of(w), hd = (w - ti * items) / kItems, i = w % kItems;
    const Place pl = place[ti];
    if (pl.pos < 0) continue;
    const bool is_k = hd < p.c.kv_heads, is_v = !is_k && hd < 2 * p.c.kv_heads;
    const int head = is_k ? hd : is_v ? hd - p.c.kv_heads : hd - 2 * p.c.kv_heads;
    const bool split = !p.interleaved && i < rv;
    const int va = p.interleaved || i >= rv ? 2 * i : i, vb = split ? i + rv : va + 1;
    float a[8], b[8];
    unpack8<T>(x[k], a);
    unpack8<T>(y[k], b);
    if (!is_v && i < rv) {
      const float2* tn = turn + ti * half + i;
      if (split) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 cs = tn[e * rv];
          const float r = a[e] * cs.x - b[e] * cs.y, o = b[e] * cs.x + a[e] * cs.y;
          a[e] = r;
          b[e] = o;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 cs = tn[e * rv], ct = tn[(4 + e) * rv];
          const float r = a[2 * e] * cs.x - a[2 * e + 1] * cs.y, o = a[2 * e + 1] * cs.x + a[2 * e] * cs.y;
          a[2 * e] = r;
          a[2 * e + 1] = o;
          const float r2 = b[2 * e] * ct.x - b[2 * e + 1] * ct.y, o2 = b[2 * e + 1] * ct.x + b[2 * e] * ct.y;
          b[2 * e] = r2;
          b[2 * e + 1] = o2;
        }
      }
    }
    if (is_k || is_v) {
      if (pl.page >= 0) {
        const uint32_t row = row_offset(p.c, pl.page, head, pl.slot);
        const float* sc = is_k ? p.c.k_scale : p.c.v_scale;
        const Scale z = make_scale(kF8 && sc ? sc[head] : 1.0f);
        unsigned char* base = is_k ? p.c.k : p.c.v;
        store_cache<T, kF8>(base, row, va, a, z);
        store_cache<T, kF8>(base, row, vb, b, z);
      }
    } else {
      uint4* dst =
          reinterpret_cast<uint4*>(p.q_out + 2 * ((long long)(t0 + ti) * p.qo_ts + (long long)head * p.qo_hs));
      dst[va] = pack8<T>(a);
      dst[vb] = pack8<T>(b);
    }
  }
}

template <class T, bool kF8, int D, int kBatch>
int launch_batch(const AppendParams& p, int group, int items, void* stream) {
  cudaLaunchConfig_t cfg = {};
  const int share = kAppendThreads * kBatch;
  cfg.gridDim = dim3((unsigned)((p.tk.tokens + group - 1) / group), (unsigned)((group * items + share - 1) / share));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // ceil(2^32 / items): the upper half of its product with w is w / items while
  // w * items stays below 2^32 (with one token a block there is nothing to divide)
  const uint32_t inv_items = group == 1 ? 0u : (uint32_t)(((1ull << 32) + items - 1) / items);
  return (int)cudaLaunchKernelEx(&cfg, append_kernel<T, kF8, D, kBatch>, p, group, inv_items);
}

// Few tokens: one item a thread, over as many blocks as that gives. Many: 4
// items a thread and as many tokens a block as they make.
template <class T, bool kF8, int D>
int launch(const AppendParams& p, void* stream) {
  const int items = (2 * p.c.kv_heads + p.q_heads) * (D / 16);
  if ((long long)p.tk.tokens * items <= 1 << 17) return launch_batch<T, kF8, D, 1>(p, 1, items, stream);
  const int fit = 4 * kAppendThreads / items, group = fit < 1 ? 1 : fit > kMaxGroup ? kMaxGroup : fit;
  return launch_batch<T, kF8, D, 4>(p, group, items, stream);
}

template <class T, bool kF8>
int pick_dim(const AppendParams& p, int d, void* stream) {
  return d == 64    ? launch<T, kF8, 64>(p, stream)
         : d == 128 ? launch<T, kF8, 128>(p, stream)
                    : launch<T, kF8, 256>(p, stream);
}

}  // namespace

int launch_kv_append(const AppendParams& p, int dtype, int cache_dtype, int head_dim, void* stream) {
  const bool f8 = cache_dtype == DFLASH_E4M3;
  if (dtype == DFLASH_BF16)
    return f8 ? pick_dim<Bf16, true>(p, head_dim, stream) : pick_dim<Bf16, false>(p, head_dim, stream);
  return f8 ? pick_dim<F16, true>(p, head_dim, stream) : pick_dim<F16, false>(p, head_dim, stream);
}

}  // namespace dflash
