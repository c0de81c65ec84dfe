// dflash_distill.cu -- distillation of a drafter from its target's top logits:
// loss and gradient.
//
// Row r holds the student's logits z over the whole vocabulary and the
// teacher's K largest logits t_j with their tokens v_j. With a temperature T,
//   p = softmax(t / T) over the row's K entries,  q = softmax(z / T) over V,
//   loss_r = w_r sum_j p_j (log p_j - log q_{v_j}),
//   dloss_r / dz_v = w_r (q_v - sum of p_j with v_j = v) / T.
// Entries with token -1 do not take part; a row left without any, or with
// w_r = 0, has loss 0 and gradient 0, and its logits are not read.
//
// The row's statistics are its maximum m and s = sum_v e^{(z_v - m)/T}, so
// q_v = e^{(z_v - m)/T} / s; all sums are fp32.
//
// What bounds it: reading the logits (and writing the gradient) once.
#include <cuda_runtime.h>

#include <cstdint>

#include "dflash_paged.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 512;
constexpr int kWarpsD = kThreads / 32;
constexpr float kLog2eD = 1.4426950408889634f;
constexpr float kLn2D = 0.6931471805599453f;

__device__ __forceinline__ float ex2d(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct B16 {  // bf16 logits: 8 to a vector
  static constexpr int kBytes = 2, kPer = 8;
  static __device__ __forceinline__ float load(const unsigned char* p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  }
  static __device__ __forceinline__ void store(unsigned char* p, float x) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)Bf16::pack(x, 0.0f);
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Bf16::unpack(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(Bf16::pack(x[0], x[1]), Bf16::pack(x[2], x[3]), Bf16::pack(x[4], x[5]), Bf16::pack(x[6], x[7]));
  }
};
struct F32 {
  static constexpr int kBytes = 4, kPer = 4;
  static __device__ __forceinline__ float load(const unsigned char* p) { return *reinterpret_cast<const float*>(p); }
  static __device__ __forceinline__ void store(unsigned char* p, float x) { *reinterpret_cast<float*>(p) = x; }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// Running maximum (of the raw logits) and sum of e^{(z - m) / T}.
struct Stat {
  float m, s;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  // a side that has seen nothing (-inf) carries its sum, 0 or NaN, as it is
  const float fa = a.m == r.m ? 1.0f : a.m == -INFINITY ? 0.0f : ex2d((a.m - r.m) * c);
  const float fb = b.m == r.m ? 1.0f : b.m == -INFINITY ? 0.0f : ex2d((b.m - r.m) * c);
  r.s = a.s * fa + b.s * fb;
  return r;
}

struct Teacher {
  int id[kMaxTeacher];     // -1: takes no part
  float p[kMaxTeacher];    // softmax(t / T)
  float logp[kMaxTeacher];
  float z[kMaxTeacher];    // the student's logit there
  float red[kWarpsD];
  float red2[kWarpsD];
  int any;
};

__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max_f32(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = red[0];
  for (int w = 1; w < kWarpsD; ++w) r = fmaxf(r, red[w]);
  __syncthreads();
  return r;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.0f;
  for (int w = 0; w < kWarpsD; ++w) r += red[w];
  __syncthreads();
  return r;
}

// The row's teacher distribution. Returns false when no entry takes part.
__device__ __forceinline__ bool teacher_row(const DistillParams& p, int r, Teacher& S) {
  float mx = -INFINITY;
  float t = 0.0f;
  const int j = threadIdx.x;  // K <= kMaxTeacher <= threads
  bool part = false, nan = false;
  if (j < p.K) {
    const int id = p.ids[(long long)r * p.K + j];
    t = p.teacher[(long long)r * p.K + j] * p.inv_t;
    part = id >= 0 && id < p.V;
    if (!part && id != -1) raise_status(p.status, DFLASH_STATUS_BAD_TOKEN);
    S.id[j] = part ? id : -1;
    nan = part && !(t == t);
    if (part) mx = t;
  }
  mx = block_max(mx, S.red);
  // one vote for "a NaN among them": it has to reach the loss
  const bool any_nan = __syncthreads_or(nan);
  if (mx == -INFINITY && !any_nan) return false;
  const float d = part ? (t - mx) * kLog2eD : -INFINITY;
  const float e = part ? ex2d(d) : 0.0f;
  const float sum = block_sum(e, S.red);
  if (j < p.K) {
    S.p[j] = part ? e / sum : 0.0f;
    S.logp[j] = (d - log2f(sum)) * kLn2D;
  }
  if (any_nan || mx == INFINITY)
    if (j == 0) raise_status(p.status, DFLASH_STATUS_BAD_ROW);
  __syncthreads();
  return true;
}

template <class T>
__device__ __forceinline__ Stat row_stat(const unsigned char* z, int V, float c) {
  Stat a = {-INFINITY, 0.0f};
  auto take = [&](float x) {
    const Stat b = {x, x == -INFINITY ? 0.0f : x == x ? 1.0f : x};
    a = join(a, b, c);
  };
  const int head = min(V, (int)(((16 - ((uintptr_t)z & 15)) & 15) / T::kBytes));
  if ((int)threadIdx.x < head) take(T::load(z + (size_t)threadIdx.x * T::kBytes));
  const unsigned char* body = z + (size_t)head * T::kBytes;
  const int nv = (V - head) / T::kPer;
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    float x[T::kPer];
    T::unpack(*(reinterpret_cast<const uint4*>(body) + i), x);
    float m = a.m;
#pragma unroll
    for (int e = 0; e < T::kPer; ++e) m = fmaxf(m, x[e]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = a.s * ex2d((a.m - ref) * c);
#pragma unroll
    for (int e = 0; e < T::kPer; ++e) s += ex2d((x[e] - ref) * c);
    a.m = m;
    a.s = s;
  }
  const int tail0 = head + nv * T::kPer;
  if (tail0 + (int)threadIdx.x < V) take(T::load(z + (size_t)(tail0 + threadIdx.x) * T::kBytes));
  return a;
}

template <class T, bool kLoss, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
  __shared__ Teacher S;
  __shared__ Stat stats[kWarpsD];
  grid_dependency_sync();
  const float c = p.inv_t * kLog2eD;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const unsigned char* z = p.z + (size_t)r * (size_t)p.z_stride * T::kBytes;
    unsigned char* g = kGrad ? p.grad + (size_t)r * (size_t)p.grad_stride * T::kBytes : nullptr;
    float w = p.weight ? p.weight[r] : 1.0f;
    if (p.upstream) w *= p.upstream[r];
    const bool active = (w != 0.0f) && teacher_row(p, r, S);
    if (!active) {
      if (kLoss && threadIdx.x == 0) {
        p.loss[r] = 0.0f;
        if (p.lse) p.lse[2 * (long long)r] = p.lse[2 * (long long)r + 1] = 0.0f;
      }
      if (kGrad)
        for (int i = threadIdx.x; i < p.V; i += kThreads) T::store(g + (size_t)i * T::kBytes, 0.0f);
      __syncthreads();
      continue;
    }
    const int j = threadIdx.x;
    if (j < p.K) S.z[j] = S.id[j] >= 0 ? T::load(z + (size_t)S.id[j] * T::kBytes) : 0.0f;
    Stat a;
    if (kLoss) {
      a = row_stat<T>(z, p.V, c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Stat b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)};
        a = join(a, b, c);
      }
      if ((threadIdx.x & 31) == 0) stats[threadIdx.x >> 5] = a;
      __syncthreads();
      a = stats[0];
      for (int i = 1; i < kWarpsD; ++i) a = join(a, stats[i], c);
      if (a.m == -INFINITY) a.s = NAN;  // no finite logit: the row has no distribution
      const float log_s = log2f(a.s) * kLn2D;
      float part = 0.0f;
      if (j < p.K && S.id[j] >= 0 && S.p[j] != 0.0f)
        part = S.p[j] * (S.logp[j] - ((S.z[j] - a.m) * p.inv_t - log_s));
      const float loss = block_sum(part, S.red);
      if (threadIdx.x == 0) {
        p.loss[r] = loss * w;
        if (p.lse) {
          p.lse[2 * (long long)r] = a.m;
          p.lse[2 * (long long)r + 1] = a.s;
        }
        if (!(a.s == a.s) || a.m == INFINITY) raise_status(p.status, DFLASH_STATUS_BAD_ROW);
      }
    } else {
      a.m = p.lse[2 * (long long)r];
      a.s = p.lse[2 * (long long)r + 1];
      __syncthreads();
    }
    if (kGrad) {
      const float coef = w * p.inv_t, f = coef / a.s;
      auto grad_of = [&](float x) { return ex2d((x - a.m) * c) * f; };
      const int head = min(p.V, (int)(((16 - ((uintptr_t)z & 15)) & 15) / T::kBytes));
      const bool same = (((uintptr_t)z ^ (uintptr_t)g) & 15) == 0;
      const int nv = same ? (p.V - head) / T::kPer : 0;
      const int edge = same ? head : 0;
      for (int i = threadIdx.x; i < edge; i += kThreads)
        T::store(g + (size_t)i * T::kBytes, grad_of(T::load(z + (size_t)i * T::kBytes)));
      for (int i = threadIdx.x; i < nv; i += kThreads) {
        float x[T::kPer];
        T::unpack(*(reinterpret_cast<const uint4*>(z + (size_t)head * T::kBytes) + i), x);
#pragma unroll
        for (int e = 0; e < T::kPer; ++e) x[e] = grad_of(x[e]);
        *(reinterpret_cast<uint4*>(g + (size_t)head * T::kBytes) + i) = T::pack(x);
      }
      for (int i = edge + nv * T::kPer + threadIdx.x; i < p.V; i += kThreads)
        T::store(g + (size_t)i * T::kBytes, grad_of(T::load(z + (size_t)i * T::kBytes)));
      __syncthreads();  // the row is written: the teacher's tokens go over it
      if (j < p.K && S.id[j] >= 0) {
        bool owner = true;
        float sum = 0.0f;
        for (int i = 0; i < p.K; ++i)
          if (S.id[i] == S.id[j]) {
            owner &= i >= j;
            sum += S.p[i];
          }
        if (owner) T::store(g + (size_t)S.id[j] * T::kBytes, grad_of(S.z[j]) - coef * sum);
      }
    }
    __syncthreads();
  }
}

template <class T, bool kLoss, bool kGrad>
int launch(const DistillParams& p, int sms, void* stream) {
  cudaLaunchConfig_t cfg = {};
  const int most = sms * (2048 / kThreads);
  cfg.gridDim = dim3((unsigned)(p.rows < most ? p.rows : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, distill_kernel<T, kLoss, kGrad>, p);
}

}  // namespace

int launch_distill_loss(const DistillParams& p, int dtype, int sms, void* stream) {
  return dtype == DFLASH_BF16 ? launch<B16, true, false>(p, sms, stream) : launch<F32, true, false>(p, sms, stream);
}
int launch_distill_grad(const DistillParams& p, int dtype, int sms, void* stream) {
  return dtype == DFLASH_BF16 ? launch<B16, false, true>(p, sms, stream) : launch<F32, false, true>(p, sms, stream);
}
int launch_distill_loss_grad(const DistillParams& p, int dtype, int sms, void* stream) {
  return dtype == DFLASH_BF16 ? launch<B16, true, true>(p, sms, stream) : launch<F32, true, true>(p, sms, stream);
}

}  // namespace dflash
