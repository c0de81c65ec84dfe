// dflash_norm.cu -- norms of queries and keys for each head, with the position
// rotation in the same pass, and their gradients.
//
// y = R(n) (x r w), r = 1 / sqrt(mean x^2 + eps) over a head's D values, R the
// rotation of pairs by the token's position n (as in dflash_kvappend.cu: the
// angle modulo a turn in 64-bit integers). Backward, with g = R(-n) dy:
//   dw = sum over tokens and heads of g x r,
//   dx = r (g w - x r mean(g w x r)).
// All in fp32, rounded once.
//
// What bounds both is reading and writing each value once. A head lies in D / 16
// lanes, two vectors of 8 values each, chosen so that both halves of a rotated
// pair meet in one lane; the same lane place holds the same values of every head
// that a thread goes through, so its sums of the weights' gradients stay in
// registers. A block takes tokens in turn: their angles
// go to shared memory while the first heads' values arrive. The weights'
// gradients are summed per thread, per block, and over blocks by a second kernel,
// always in the same order.
#include <cuda_runtime.h>

#include <cstdint>

#include "dflash_norm.cuh"
#include "dflash_train.h"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 4;  // tokens whose angles a block holds at a time

struct Place {
  int va, vb;   // the lane's two vectors
  bool split;   // its pairs lie between them
  bool turned;  // it has pairs
};
__device__ __forceinline__ Place place_of(const NormParams& p, int i) {
  const int rv = p.rot >> 4;
  Place l;
  l.turned = i < rv;
  l.split = !p.interleaved && l.turned;
  l.va = l.split ? i : 2 * i;
  l.vb = l.split ? i + rv : 2 * i + 1;
  return l;
}

// The angles of nt tokens from t0 on: pair 8 i + e at [token][e][i].
__device__ __forceinline__ void fill_turns(const NormParams& p, float2* turn, int t0, int nt) {
  const int half = p.rot >> 1, rv = p.rot >> 4;
  if (!half) return;
  for (int at = threadIdx.x; at < nt * half; at += kThreads) {
    const int ti = at / half, j = at - ti * half;
    turn[ti * half + (j & 7) * rv + (j >> 3)] = turn_at(p.phases[j], p.positions[t0 + ti]);
  }
}

// Weights for a lane place: 16 of one head in pieces of 4, a piece of all lanes side
// by side, so that reading them meets no bank twice.
template <class T, int D>
__device__ __forceinline__ void fill_weights(const NormParams& p, float4* w) {
  constexpr int kLanes = D / 16;
  for (int at = threadIdx.x; at < 2 * kLanes; at += kThreads) {
    const int part = at / kLanes, i = at - part * kLanes;
    const Place l = place_of(p, i);
    const void* from = part ? p.k_weight : p.q_weight;
    float a[8], b[8];
    weight8<T>(from, p.weight_f32, l.va, a);
    weight8<T>(from, p.weight_f32, l.vb, b);
    float4* to = w + part * 4 * kLanes + i;
    to[0] = make_float4(a[0], a[1], a[2], a[3]);
    to[kLanes] = make_float4(a[4], a[5], a[6], a[7]);
    to[2 * kLanes] = make_float4(b[0], b[1], b[2], b[3]);
    to[3 * kLanes] = make_float4(b[4], b[5], b[6], b[7]);
  }
}

// A row is one head of one token: queries, then keys. What bounds it: 302 MB of 8192
// tokens, 64 + 8 heads of 128 in bf16 take XXX us; with the weights in registers, two
// blocks an SM, they took 81.
template <class T, int D>
__global__ void __launch_bounds__(kThreads, 4) norm_kernel(const NormParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes, kBatch = 2;
  __shared__ float2 turn[kGroup * D / 2];
  __shared__ float4 weights[2 * 4 * kLanes];
  grid_dependency_sync();
  const int i = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
  const Place l = place_of(p, i);
  const int heads = p.q_heads + p.k_heads, t0 = blockIdx.x * kGroup, nt = min(kGroup, p.tokens - t0);
  const int rows = nt * heads, half = p.rot >> 1, rv = p.rot >> 4;
  bool ready = false;
  for (int r0 = first; r0 < rows || !ready; r0 += kBatch * kRows) {
    uint4 x[kBatch], y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kRows;
      if (r >= rows) continue;
      const int ti = r / heads, h = r - ti * heads;
      const HeadRows& s = h < p.q_heads ? p.q : p.k;
      const uint4* src = reinterpret_cast<const uint4*>(
          s.p + 2 * ((t0 + ti) * s.ts + (long long)(h < p.q_heads ? h : h - p.q_heads) * s.hs));
      x[k] = src[l.va];
      y[k] = src[l.vb];
    }
    if (!ready) {
      fill_weights<T, D>(p, weights);
      fill_turns(p, turn, t0, nt);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kRows;
      if (r >= rows) continue;
      const int ti = r / heads, h = r - ti * heads;
      const bool is_q = h < p.q_heads;
      float a[8], b[8];
      unpack8<T>(x[k], a);
      unpack8<T>(y[k], b);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += a[e] * a[e] + b[e] * b[e];
      const float inv = rsqrtf(head_sum<kLanes>(sum) * (1.0f / D) + p.eps);
      const float4* w = weights + (is_q ? 0 : 4 * kLanes) + i;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 u = w[e * kLanes], v = w[(2 + e) * kLanes];
        a[4 * e] *= inv * u.x, a[4 * e + 1] *= inv * u.y, a[4 * e + 2] *= inv * u.z, a[4 * e + 3] *= inv * u.w;
        b[4 * e] *= inv * v.x, b[4 * e + 1] *= inv * v.y, b[4 * e + 2] *= inv * v.z, b[4 * e + 3] *= inv * v.w;
      }
      if (l.turned) turn_pairs(a, b, turn + ti * half + i, rv, l.split, false);
      const HeadRows& o = is_q ? p.qo : p.ko;
      uint4* dst = reinterpret_cast<uint4*>(o.p + 2 * ((t0 + ti) * o.ts + (long long)(is_q ? h : h - p.q_heads) * o.hs));
      dst[l.va] = pack8<T>(a);
      dst[l.vb] = pack8<T>(b);
    }
  }
}

// Queries first, then keys: a thread's sums are those of one of them. The next row's
// values are asked for before this one's are worked on.
template <class T, int D>
__global__ void __launch_bounds__(kThreads, 2) norm_grad_kernel(const NormParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  __shared__ float2 turn[kGroup * D / 2];
  __shared__ float4 weights[2 * 4 * kLanes];
  __shared__ float sums[kThreads / 32][D];
  grid_dependency_sync();
  const int tid = threadIdx.x, i = tid % kLanes, first = tid / kLanes;
  const Place l = place_of(p, i);
  const int half = p.rot >> 1, rv = p.rot >> 4;
  fill_weights<T, D>(p, weights);
  __syncthreads();
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const HeadRows s = part ? p.k : p.q, d = part ? p.dk : p.dq, o = part ? p.ko : p.qo;
    const int hn = part ? p.k_heads : p.q_heads;
    float dw[16] = {};
    for (int t0 = blockIdx.x * kGroup; hn && t0 < p.tokens; t0 += gridDim.x * kGroup) {
      const int nt = min(kGroup, p.tokens - t0), rows = nt * hn;
      uint4 x0, x1, g0, g1;
      auto load = [&](int r) {
        const int ti = r / hn, h = r - ti * hn;
        const uint4* xs = reinterpret_cast<const uint4*>(s.p + 2 * ((t0 + ti) * s.ts + (long long)h * s.hs));
        const uint4* gs = reinterpret_cast<const uint4*>(d.p + 2 * ((t0 + ti) * d.ts + (long long)h * d.hs));
        x0 = xs[l.va], x1 = xs[l.vb], g0 = gs[l.va], g1 = gs[l.vb];
      };
      if (first < rows) load(first);
      if (half) {
        __syncthreads();
        fill_turns(p, turn, t0, nt);
        __syncthreads();
      }
      for (int r = first; r < rows; r += kRows) {
        const int ti = r / hn, h = r - ti * hn;
        float a[8], b[8], ga[8], gb[8];
        unpack8<T>(x0, a);
        unpack8<T>(x1, b);
        unpack8<T>(g0, ga);
        unpack8<T>(g1, gb);
        if (r + kRows < rows) load(r + kRows);
        if (l.turned) turn_pairs(ga, gb, turn + ti * half + i, rv, l.split, true);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += a[e] * a[e] + b[e] * b[e];
        const float inv = rsqrtf(head_sum<kLanes>(sum) * (1.0f / D) + p.eps);
        const float4* w = weights + part * 4 * kLanes + i;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[e] += ga[e] * (a[e] * inv);
          dw[8 + e] += gb[e] * (b[e] * inv);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 u = w[e * kLanes], v = w[(2 + e) * kLanes];
          ga[4 * e] *= u.x, ga[4 * e + 1] *= u.y, ga[4 * e + 2] *= u.z, ga[4 * e + 3] *= u.w;
          gb[4 * e] *= v.x, gb[4 * e + 1] *= v.y, gb[4 * e + 2] *= v.z, gb[4 * e + 3] *= v.w;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += a[e] * ga[e] + b[e] * gb[e];
        const float mean = head_sum<kLanes>(dot) * (1.0f / D) * inv * inv;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = inv * (ga[e] - a[e] * mean);
          b[e] = inv * (gb[e] - b[e] * mean);
        }
        uint4* dst = reinterpret_cast<uint4*>(o.p + 2 * ((t0 + ti) * o.ts + (long long)h * o.hs));
        dst[l.va] = pack8<T>(a);
        dst[l.vb] = pack8<T>(b);
      }
    }
    // the block's sums: over the heads inside a warp, then over the warps
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = dw[e];
#pragma unroll
      for (int m = 16; m >= kLanes; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if ((tid & 31) < kLanes) sums[tid >> 5][8 * (e < 8 ? l.va : l.vb) + (e & 7)] = v;
    }
    __syncthreads();
    for (int j = tid; j < D; j += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) v += sums[k][j];
      p.partial[((size_t)blockIdx.x * 2 + part) * D + j] = v;
    }
  }
}

// Sums the blocks' partial sums: 32 columns a block, 32 runs of blocks.
template <class T, int D>
__global__ void __launch_bounds__(1024) norm_weights_kernel(const NormParams p, int blocks) {
  __shared__ float sums[32][33];
  grid_dependency_sync();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;  // column of [2][D]
  float v = 0.0f;
  for (int b = run; b < blocks; b += 32) v += p.partial[(size_t)b * 2 * D + c];
  sums[run][threadIdx.x & 31] = v;
  __syncthreads();
  if (run) return;
  float s = 0.0f;
#pragma unroll
  for (int r = 0; r < 32; ++r) s += sums[r][threadIdx.x];
  const int part = c / D, j = c - part * D;
  void* out = part ? p.gk_weight : p.gq_weight;
  if (!out) return;
  if (p.weight_f32)
    static_cast<float*>(out)[j] = s;
  else
    static_cast<uint16_t*>(out)[j] = (uint16_t)T::pack(s, 0.0f);
}

template <class K, class... A>
int launch(K kernel, int grid, int threads, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int D>
int forward(const NormParams& p, void* stream) {
  return launch(norm_kernel<T, D>, (p.tokens + kGroup - 1) / kGroup, kThreads, stream, p);
}
template <class T, int D>
int backward(const NormParams& p, void* stream) {
  const int groups = (p.tokens + kGroup - 1) / kGroup, blocks = groups < kNormBlocks ? groups : kNormBlocks;
  const int e = launch(norm_grad_kernel<T, D>, blocks, kThreads, stream, p);
  if (e || !(p.gq_weight || p.gk_weight)) return e;
  return launch(norm_weights_kernel<T, D>, 2 * D / 32, 1024, stream, p, blocks);
}

}  // namespace

int launch_norm(const NormParams& p, int dtype, int d, void* stream) {
  if (dtype == DFLASH_BF16)
    return d == 64 ? forward<Bf16, 64>(p, stream) : d == 128 ? forward<Bf16, 128>(p, stream) : forward<Bf16, 256>(p, stream);
  return d == 64 ? forward<F16, 64>(p, stream) : d == 128 ? forward<F16, 128>(p, stream) : forward<F16, 256>(p, stream);
}
int launch_norm_grad(const NormParams& p, int dtype, int d, void* stream) {
  if (dtype == DFLASH_BF16)
    return d == 64    ? backward<Bf16, 64>(p, stream)
           : d == 128 ? backward<Bf16, 128>(p, stream)
                      : backward<Bf16, 256>(p, stream);
  return d == 64    ? backward<F16, 64>(p, stream)
         : d == 128 ? backward<F16, 128>(p, stream)
                    : backward<F16, 256>(p, stream);
}

}  // namespace dflash
