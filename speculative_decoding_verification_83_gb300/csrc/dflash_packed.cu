// dflash_packed.cu -- attention over packed sequences, row by row.
//
// out_i = sum_j e^(s q_i k_j) v_j / sum_j e^(s q_i k_j) over the keys j that row i
// sees, lse_i = log of that sum. Backward, with p_ij = e^(s q_i k_j - lse_i) and
// delta_i = sum over d of dout_id out_id:
//   dv_j = sum_i p_ij dout_i, ds_ij = p_ij (dout_i v_j - delta_i),
//   dq_i = s sum_j ds_ij k_j, dk_j = s sum_i ds_ij q_i,
// i over the rows, of all query heads that share the key's head, that see key j.
//
// One warp takes a row: 32 keys (queries) at a time, a score per lane, then
// D / 32 columns per lane. Pairs that do not see each other take no part,
// whatever they hold.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dflash_packed.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 8;
constexpr uint32_t kAll = 0xffffffffu;

template <class T>
__device__ __forceinline__ float value(const unsigned char* row, int d) {
  const uint32_t x = reinterpret_cast<const uint16_t*>(row)[d];
  return T::unpack(x).x;
}
// sum over d of a[d] b[d], a in shared memory
template <class T, int D>
__device__ __forceinline__ float dot(const float* a, const unsigned char* b) {
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 u = reinterpret_cast<const uint4*>(b)[c];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = T::unpack(w[e]);
      s0 = fmaf(a[8 * c + 2 * e], f.x, s0);
      s1 = fmaf(a[8 * c + 2 * e + 1], f.y, s1);
    }
  }
  return s0 + s1;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ unsigned char* row_of(const HeadRows& h, long long t, int head) {
  return h.p + 2 * (t * h.ts + (long long)head * h.hs);
}
template <class T>
__device__ __forceinline__ void put(unsigned char* row, int d, float v) {
  reinterpret_cast<uint16_t*>(row)[d] = (uint16_t)T::pack(v, 0.0f);
}
// whether a row of D values in memory holds one that is not finite
template <class T, int D>
__device__ __forceinline__ bool row_not_finite(const unsigned char* row) {
  bool found = false;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) found |= !(fabsf(value<T>(row, threadIdx.x % 32 + 32 * i)) < INFINITY);
  return __any_sync(kAll, found);
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) rows_forward_kernel(const PackedParams p, const uint32_t* redo) {
  __shared__ float q_row[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)p.q_tokens * p.q_heads;
  for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows; r += (long long)gridDim.x * kWarps) {
    const int t = (int)(r / p.q_heads), head = (int)(r - (long long)t * p.q_heads);
    unsigned char* out = row_of(p.o, t, head);
    const int b = sequence_of(p.q_start, p.B, t);
    int first = 0, n = 0, kv0 = 0, m = 0;
    bool bad = false;
    if (b >= 0) {
      extent(p.q_start, p.q_tokens, b, first, n, bad);
      extent(p.kv_start, p.kv_tokens, b, kv0, m, bad);
    }
    if (b < 0 || t < first || t >= first + n) {
      if (p.fill) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) put<T>(out, lane + 32 * i, 0.0f);
        if (p.low)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) p.low[r * D + lane + 32 * i] = 0;
        if (p.lse && lane == 0) p.lse[r] = -INFINITY;
      }
      continue;
    }
    const int kh = head / p.G, vis = seen_keys(p.causal, n, m, t - first);
    const unsigned char* q = row_of(p.q, t, head);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D / 32; ++i) q_row[warp][lane + 32 * i] = value<T>(q, lane + 32 * i);
    __syncwarp();
    float top = -INFINITY, sum = 0.0f, acc[D / 32] = {};
    uint32_t odd[D / 32] = {};  // values seen that are not finite: +inf (1), -inf (2), NaN (4)
    for (int j0 = 0; j0 < vis; j0 += 32) {
      const int j = j0 + lane, count = min(32, vis - j0);
      float x = -INFINITY;
      if (j < vis) x = dot<T, D>(q_row[warp], row_of(p.k, kv0 + j, kh)) * p.scale;
      const float m1 = warp_max_f32(fmaxf(x, top)), ref = m1 == -INFINITY ? 0.0f : m1;
      const float f = expf(top - ref), w = expf(x - ref);  // (a score that is NaN leaves NaN)
      sum = sum * f + warp_sum(w);
      top = m1;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] *= f;
      for (int k = 0; k < count; ++k) {
        const float wk = __shfl_sync(kAll, w, k);
        const unsigned char* v = row_of(p.v, kv0 + j0 + k, kh);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const float y = value<T>(v, lane + 32 * i);
          if (fabsf(y) < INFINITY)
            acc[i] = fmaf(wk, y, acc[i]);
          else
            odd[i] |= y > 0.0f ? 1u : y < 0.0f ? 2u : 4u;
        }
      }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      float y = acc[i] * inv;
      if (odd[i] && y == y) y = odd[i] == 1u ? INFINITY : odd[i] == 2u ? -INFINITY : NAN;
      const uint32_t hi = T::pack(y, 0.0f) & 0xffffu;
      reinterpret_cast<uint16_t*>(out)[lane + 32 * i] = (uint16_t)hi;
      if (p.low) p.low[r * D + lane + 32 * i] = low_bits(y, hi);
    }
    if (p.lse && lane == 0) p.lse[r] = sum == 0.0f ? -INFINITY : top + logf(sum);
  }
}

// sum over d of dout out, per row
template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) delta_kernel(const PackedParams p) {
  constexpr int kLanes = D / 8;  // 8 values each
  const int lane = threadIdx.x % kLanes;
  const long long rows = (long long)p.q_tokens * p.q_heads;
  const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
  float s = 0.0f;
  if (r < rows) {
    const int t = (int)(r / p.q_heads), head = (int)(r - (long long)t * p.q_heads);
    const uint4 a = reinterpret_cast<const uint4*>(row_of(p.o, t, head))[lane];
    const uint4 g = reinterpret_cast<const uint4*>(row_of(p.d_o, t, head))[lane];
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {g.x, g.y, g.z, g.w};
    uint2 l = make_uint2(0u, 0u);
    if (p.low) l = reinterpret_cast<const uint2*>(p.low + r * D)[lane];
    const uint32_t low[2] = {l.x, l.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = low[e >> 1] >> (16 * (e & 1));
      const float2 v = T::unpack(y[e]);
      s = fmaf(with_low(x[e] & 0xffffu, (int8_t)(b & 0xffu)), v.x,
               fmaf(with_low(x[e] >> 16, (int8_t)((b >> 8) & 0xffu)), v.y, s));
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if (r < rows && lane == 0) p.delta[r] = s;
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) rows_dq_kernel(const PackedParams p, const uint32_t* redo) {
  __shared__ float q_row[kWarps][D], g_row[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)p.q_tokens * p.q_heads;
  for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows; r += (long long)gridDim.x * kWarps) {
    const int t = (int)(r / p.q_heads), head = (int)(r - (long long)t * p.q_heads);
    unsigned char* out = row_of(p.dq, t, head);
    const int b = sequence_of(p.q_start, p.B, t);
    int first = 0, n = 0, kv0 = 0, m = 0;
    bool bad = false;
    if (b >= 0) {
      extent(p.q_start, p.q_tokens, b, first, n, bad);
      extent(p.kv_start, p.kv_tokens, b, kv0, m, bad);
    }
    if (b < 0 || t < first || t >= first + n) {
      if (p.fill)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) put<T>(out, lane + 32 * i, 0.0f);
      continue;
    }
    const int kh = head / p.G, vis = seen_keys(p.causal, n, m, t - first);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      q_row[warp][lane + 32 * i] = value<T>(row_of(p.q, t, head), lane + 32 * i);
      g_row[warp][lane + 32 * i] = value<T>(row_of(p.d_o, t, head), lane + 32 * i);
    }
    __syncwarp();
    const float lse = p.lse[r], delta = p.delta[r];
    float acc[D / 32] = {};
    for (int j0 = 0; j0 < vis; j0 += 32) {
      const int j = j0 + lane, count = min(32, vis - j0);
      float ds = 0.0f;
      if (j < vis) {
        const float x = dot<T, D>(q_row[warp], row_of(p.k, kv0 + j, kh)) * p.scale;
        ds = expf(x - lse) * (dot<T, D>(g_row[warp], row_of(p.v, kv0 + j, kh)) - delta) * p.scale;
      }
      for (int k = 0; k < count; ++k) {
        const float w = __shfl_sync(kAll, ds, k);
        const unsigned char* row = row_of(p.k, kv0 + j0 + k, kh);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(w, value<T>(row, lane + 32 * i), acc[i]);
      }
      bool lost = true;  // every column is NaN: nothing brings it back
#pragma unroll
      for (int i = 0; i < D / 32; ++i) lost &= acc[i] != acc[i];
      if (__all_sync(kAll, lost)) break;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) put<T>(out, lane + 32 * i, lse == -INFINITY ? 0.0f : acc[i]);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) rows_dkv_kernel(const PackedParams p, const uint32_t* redo) {
  __shared__ float k_row[kWarps][D], v_row[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)p.kv_tokens * p.kv_heads;
  for (long long r = (long long)blockIdx.x * kWarps + warp; r < rows; r += (long long)gridDim.x * kWarps) {
    const int t = (int)(r / p.kv_heads), kh = (int)(r - (long long)t * p.kv_heads);
    const int b = sequence_of(p.kv_start, p.B, t);
    int first = 0, n = 0, kv0 = 0, m = 0;
    bool bad = false;
    if (b >= 0) {
      extent(p.q_start, p.q_tokens, b, first, n, bad);
      extent(p.kv_start, p.kv_tokens, b, kv0, m, bad);
    }
    unsigned char *dk = row_of(p.dk, t, kh), *dv = row_of(p.dv, t, kh);
    if (b < 0 || t < kv0 || t >= kv0 + m) {
      if (p.fill)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          put<T>(dk, lane + 32 * i, 0.0f);
          put<T>(dv, lane + 32 * i, 0.0f);
        }
      continue;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      k_row[warp][lane + 32 * i] = value<T>(row_of(p.k, t, kh), lane + 32 * i);
      v_row[warp][lane + 32 * i] = value<T>(row_of(p.v, t, kh), lane + 32 * i);
    }
    __syncwarp();
    float ak[D / 32] = {}, av[D / 32] = {};
    const int i_first = first_query(p.causal, n, m, t - kv0);
    bool lost = false;
    for (int g = 0; g < p.G && !lost; ++g) {
      const int head = kh * p.G + g;
      for (int i0 = i_first; i0 < n && !lost; i0 += 32) {
        const int i = i0 + lane, count = min(32, n - i0);
        float w = 0.0f, ds = 0.0f;
        if (i < n) {
          const long long at = (long long)(first + i) * p.q_heads + head;
          const float x = dot<T, D>(k_row[warp], row_of(p.q, first + i, head)) * p.scale, lse = p.lse[at];
          w = lse == -INFINITY ? 0.0f : expf(x - lse);
          ds = w * (dot<T, D>(v_row[warp], row_of(p.d_o, first + i, head)) - p.delta[at]) * p.scale;
        }
        for (int k = 0; k < count; ++k) {
          const float wk = __shfl_sync(kAll, w, k), dsk = __shfl_sync(kAll, ds, k);
          const unsigned char *qr = row_of(p.q, first + i0 + k, head), *gr = row_of(p.d_o, first + i0 + k, head);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            av[e] = fmaf(wk, value<T>(gr, lane + 32 * e), av[e]);
            ak[e] = fmaf(dsk, value<T>(qr, lane + 32 * e), ak[e]);
          }
        }
        bool gone = true;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) gone &= av[e] != av[e] && ak[e] != ak[e];
        lost = __all_sync(kAll, gone);
      }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      put<T>(dk, lane + 32 * e, ak[e]);
      put<T>(dv, lane + 32 * e, av[e]);
    }
  }
}

// Offsets that leave the arrays or do not ascend are reported once.
__global__ void check_kernel(const PackedParams p) {
  bool bad = false;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    int first, n;
    extent(p.q_start, p.q_tokens, b, first, n, bad);
    extent(p.kv_start, p.kv_tokens, b, first, n, bad);
  }
  if (bad) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
}

unsigned blocks_for(long long rows) {
  const long long n = (rows + kWarps - 1) / kWarps;
  return (unsigned)(n < 152 * 64 ? n : 152 * 64);
}
template <class T>
int forward(const PackedParams& p, int d, const uint32_t* redo, cudaStream_t st) {
  const unsigned grid = blocks_for((long long)p.q_tokens * p.q_heads);
  if (!grid) return 0;
  if (d == 64)
    rows_forward_kernel<T, 64><<<grid, 32 * kWarps, 0, st>>>(p, redo);
  else
    rows_forward_kernel<T, 128><<<grid, 32 * kWarps, 0, st>>>(p, redo);
  return (int)cudaGetLastError();
}
template <int D>
int grad(const PackedParams& p, const uint32_t* redo_q, const uint32_t* redo_kv, cudaStream_t st) {
  const unsigned grid_q = blocks_for((long long)p.q_tokens * p.q_heads), grid_kv = blocks_for((long long)p.kv_tokens * p.kv_heads);
  if (grid_q) rows_dq_kernel<Bf16, D><<<grid_q, 32 * kWarps, 0, st>>>(p, redo_q);
  if (grid_kv) rows_dkv_kernel<Bf16, D><<<grid_kv, 32 * kWarps, 0, st>>>(p, redo_kv);
  return (int)cudaGetLastError();
}

}  // namespace

int launch_rows_forward(const PackedParams& p, int dtype, int head_dim, const uint32_t* redo, void* stream) {
  return dtype == DFLASH_BF16 ? forward<Bf16>(p, head_dim, redo, (cudaStream_t)stream)
                              : forward<F16>(p, head_dim, redo, (cudaStream_t)stream);
}
int launch_delta(const PackedParams& p, int head_dim, void* stream) {
  const long long threads = (long long)p.q_tokens * p.q_heads * (head_dim / 8);
  const unsigned grid = (unsigned)((threads + 32 * kWarps - 1) / (32 * kWarps));
  if (!grid) return 0;
  if (head_dim == 64)
    delta_kernel<Bf16, 64><<<grid, 32 * kWarps, 0, (cudaStream_t)stream>>>(p);
  else
    delta_kernel<Bf16, 128><<<grid, 32 * kWarps, 0, (cudaStream_t)stream>>>(p);
  return (int)cudaGetLastError();
}
int launch_rows_grad(const PackedParams& p, int head_dim, const uint32_t* redo_q, const uint32_t* redo_kv, void* stream) {
  return head_dim == 64 ? grad<64>(p, redo_q, redo_kv, (cudaStream_t)stream)
                        : grad<128>(p, redo_q, redo_kv, (cudaStream_t)stream);
}

size_t packed_workspace(int B, int q_tokens, int kv_tokens, int q_heads, int kv_heads, int head_dim, bool backward) {
  return backward ? ((size_t)q_tokens * q_heads * sizeof(float) + 255) / 256 * 256 + 256 : 256;
}
int launch_packed(const PackedParams& p, int dtype, int head_dim, int sms, void* stream) {
  check_kernel<<<1, 256, 0, (cudaStream_t)stream>>>(p);
  return launch_rows_forward(p, dtype, head_dim, nullptr, stream);
}
int launch_packed_grad(const PackedParams& p, int head_dim, int sms, void* stream) {
  PackedParams q = p;
  q.delta = reinterpret_cast<float*>(p.ws);
  const int e = launch_delta(q, head_dim, stream);
  return e ? e : launch_rows_grad(q, head_dim, nullptr, nullptr, stream);
}

}  // namespace dflash
