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
constexpr int kSms = 152;
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

__device__ __forceinline__ void ask16(uint4* to, const uint4* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void ask_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void ask_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The angles of kGroup tokens: pair 8 i + e at [token][e][i]. Positions are read while
// the group before is worked on.
template <int D>
struct Turns {
  static constexpr int kPer = (kGroup * D / 2 + kThreads - 1) / kThreads;
  int pos[kPer];
  __device__ __forceinline__ void ask(const NormParams& p, int t0) {
    const int half = p.rot >> 1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = threadIdx.x + k * kThreads, ti = half ? at / half : kGroup;
      pos[k] = ti < kGroup && t0 + ti < p.tokens ? p.positions[t0 + ti] : 0;
    }
  }
  __device__ __forceinline__ void put(const NormParams& p, float2* turn) const {
    const int half = p.rot >> 1, rv = p.rot >> 4;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = threadIdx.x + k * kThreads;
      if (at >= kGroup * half) continue;
      const int ti = at / half, j = at - ti * half;
      turn[ti * half + (j & 7) * rv + (j >> 3)] = turn_at(p.phases[j], pos[k]);
    }
  }
};

// A block's way through the rows (heads of tokens) of its groups of tokens, kRows at a time.
template <int kRows>
struct Walk {
  int t0, r;  // the group's first token, the first row of the step
  int heads;
  unsigned long long per;  // r / heads = r per / 2^48 while r heads < 2^48 (r < 2^23, heads < 2^21)
  __device__ __forceinline__ Walk(const NormParams& p, int heads_)
      : t0(heads_ ? blockIdx.x * kGroup : p.tokens), r(0), heads(heads_),
        per(heads_ ? (1ull << 48) / heads_ + 1 : 0) {}
  __device__ __forceinline__ int rows(int tokens) const { return min(kGroup, tokens - t0) * heads; }
  __device__ __forceinline__ int token(int row) const { return (int)((unsigned)row * per >> 48); }
  __device__ __forceinline__ int after() const { return t0 + gridDim.x * kGroup; }
  // true: on to the next group
  __device__ __forceinline__ bool next(int tokens) {
    r += kRows;
    if (r < rows(tokens)) return false;
    r = 0;
    t0 = after();
    return true;
  }
};

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
// tokens, 64 + 8 heads of 128 in bf16 take 52 us (5.8 TB/s), replayed from graphs 55. A
// thread's vectors are asked for three steps ahead and wait in shared memory: with loads
// into registers and a block for each group of tokens they took 61 replayed.
constexpr int kForwardSlots = 4, kForwardBlocks = 4;
template <class T, int D>
__global__ void __launch_bounds__(kThreads, kForwardBlocks) norm_kernel(const NormParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  extern __shared__ uint4 ring[];  // [slot][2][thread]
  __shared__ float2 turns[2][kGroup * D / 2];
  __shared__ float4 weights[2 * 4 * kLanes];
  grid_dependency_sync();
  const int i = threadIdx.x % kLanes, first = threadIdx.x / kLanes;
  const Place l = place_of(p, i);
  const int half = p.rot >> 1, rv = p.rot >> 4;
  Walk<kRows> at(p, p.q_heads + p.k_heads), to = at;  // where the work is, and the loads
  auto ask = [&](int slot) {
    if (to.t0 < p.tokens) {
      const int r = to.r + first;
      if (r < to.rows(p.tokens)) {
        const int ti = to.token(r), h = r - ti * to.heads;
        const HeadRows& s = h < p.q_heads ? p.q : p.k;
        const uint4* src = reinterpret_cast<const uint4*>(
            s.p + 2 * ((to.t0 + ti) * s.ts + (long long)(h < p.q_heads ? h : h - p.q_heads) * s.hs));
        ask16(ring + (2 * slot) * kThreads + threadIdx.x, src + l.va);
        ask16(ring + (2 * slot + 1) * kThreads + threadIdx.x, src + l.vb);
      }
      to.next(p.tokens);
    }
    ask_end();
  };
#pragma unroll
  for (int s = 0; s < kForwardSlots - 1; ++s) ask(s);
  Turns<D> ahead;
  ahead.ask(p, at.t0);
  fill_weights<T, D>(p, weights);
  ahead.put(p, turns[0]);
  ahead.ask(p, at.after());
  __syncthreads();
  int buf = 0;
  for (int slot = 0; at.t0 < p.tokens; slot = slot + 1 == kForwardSlots ? 0 : slot + 1) {
    ask_wait<kForwardSlots - 2>();
    const int t0 = at.t0, r = at.r + first;
    const bool mine = r < at.rows(p.tokens);
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (mine) x = ring[(2 * slot) * kThreads + threadIdx.x], y = ring[(2 * slot + 1) * kThreads + threadIdx.x];
    ask(slot ? slot - 1 : kForwardSlots - 1);  // the slot of the step before
    if (mine) {
      const int ti = at.token(r), h = r - ti * at.heads;
      const bool is_q = h < p.q_heads;
      float a[8], b[8];
      unpack8<T>(x, a);
      unpack8<T>(y, b);
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
      if (l.turned) turn_pairs(a, b, turns[buf] + ti * half + i, rv, l.split, false);
      const HeadRows& o = is_q ? p.qo : p.ko;
      uint4* dst = reinterpret_cast<uint4*>(o.p + 2 * ((t0 + ti) * o.ts + (long long)(is_q ? h : h - p.q_heads) * o.hs));
      dst[l.va] = pack8<T>(a);
      dst[l.vb] = pack8<T>(b);
    }
    if (at.next(p.tokens) && half) {
      buf ^= 1;
      ahead.put(p, turns[buf]);
      ahead.ask(p, at.after());
      __syncthreads();
    }
  }
}

// Queries first, then keys: a thread's sums are those of one of them. What bounds it:
// 503 MB of 16384 tokens, 32 + 8 heads of 128 in bf16 take 97 us (5.2 TB/s); with the next
// row in registers they took 111, and three slots of the ring take 104.
constexpr int kGradSlots = 4, kGradBlocks = 2;
template <class T, int D>
__global__ void __launch_bounds__(kThreads, kGradBlocks) norm_grad_kernel(const NormParams p) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;
  extern __shared__ uint4 ring[];  // [slot][4][thread]
  __shared__ float2 turns[2][kGroup * D / 2];
  __shared__ float4 weights[2 * 4 * kLanes];
  __shared__ float sums[kThreads / 32][D];
  grid_dependency_sync();
  const int tid = threadIdx.x, i = tid % kLanes, first = tid / kLanes;
  const Place l = place_of(p, i);
  const int half = p.rot >> 1, rv = p.rot >> 4;
  fill_weights<T, D>(p, weights);
  Turns<D> ahead;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const HeadRows s = part ? p.k : p.q, d = part ? p.dk : p.dq, o = part ? p.ko : p.qo;
    Walk<kRows> at(p, part ? p.k_heads : p.q_heads), to = at;
    auto ask = [&](int slot) {
      if (to.t0 < p.tokens) {
        const int r = to.r + first;
        if (r < to.rows(p.tokens)) {
          const int ti = to.token(r), h = r - ti * to.heads;
          const uint4* xs = reinterpret_cast<const uint4*>(s.p + 2 * ((to.t0 + ti) * s.ts + (long long)h * s.hs));
          const uint4* gs = reinterpret_cast<const uint4*>(d.p + 2 * ((to.t0 + ti) * d.ts + (long long)h * d.hs));
          uint4* r4 = ring + 4 * slot * kThreads + tid;
          ask16(r4, xs + l.va);
          ask16(r4 + kThreads, xs + l.vb);
          ask16(r4 + 2 * kThreads, gs + l.va);
          ask16(r4 + 3 * kThreads, gs + l.vb);
        }
        to.next(p.tokens);
      }
      ask_end();
    };
#pragma unroll
    for (int k = 0; k < kGradSlots - 1; ++k) ask(k);
    ahead.ask(p, at.t0);
    ahead.put(p, turns[0]);
    ahead.ask(p, at.after());
    __syncthreads();
    int buf = 0;
    float dw[16] = {};
    for (int slot = 0; at.t0 < p.tokens; slot = slot + 1 == kGradSlots ? 0 : slot + 1) {
      ask_wait<kGradSlots - 2>();
      const int t0 = at.t0, r = at.r + first;
      const bool mine = r < at.rows(p.tokens);
      ask(slot ? slot - 1 : kGradSlots - 1);  // the slot of the step before
      if (mine) {
        const uint4* r4 = ring + 4 * slot * kThreads + tid;
        const int ti = at.token(r), h = r - ti * at.heads;
        float a[8], b[8], ga[8], gb[8];
        unpack8<T>(r4[0], a);
        unpack8<T>(r4[kThreads], b);
        unpack8<T>(r4[2 * kThreads], ga);
        unpack8<T>(r4[3 * kThreads], gb);
        if (l.turned) turn_pairs(ga, gb, turns[buf] + ti * half + i, rv, l.split, true);
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
      if (at.next(p.tokens) && half) {
        buf ^= 1;
        ahead.put(p, turns[buf]);
        ahead.ask(p, at.after());
        __syncthreads();
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
int launch(K kernel, int grid, int threads, int smem, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Shared memory above 48 KB, once for each device.
template <class K>
int allow(K kernel, int smem, bool (&ready)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (ready[dev]) return 0;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  ready[dev] = e == cudaSuccess;
  return (int)e;
}

template <class T, int D>
int forward(const NormParams& p, void* stream) {
  static bool ready[64] = {};
  constexpr int kSmem = kForwardSlots * 2 * kThreads * 16, kBlocks = kForwardBlocks * kSms;
  const int e = allow(norm_kernel<T, D>, kSmem, ready);
  if (e) return e;
  const int groups = (p.tokens + kGroup - 1) / kGroup;
  return launch(norm_kernel<T, D>, groups < kBlocks ? groups : kBlocks, kThreads, kSmem, stream, p);
}
template <class T, int D>
int backward(const NormParams& p, void* stream) {
  static bool ready[64] = {};
  constexpr int kSmem = kGradSlots * 4 * kThreads * 16;
  int e = allow(norm_grad_kernel<T, D>, kSmem, ready);
  if (e) return e;
  const int groups = p.tokens ? (p.tokens + kGroup - 1) / kGroup : 1;  // (without tokens the weights' gradients are 0)
  const int blocks = groups < kNormBlocks ? groups : kNormBlocks;
  e = launch(norm_grad_kernel<T, D>, blocks, kThreads, kSmem, stream, p);
  if (e || !(p.gq_weight || p.gk_weight)) return e;
  return launch(norm_weights_kernel<T, D>, 2 * D / 32, 1024, 0, stream, p, blocks);
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
