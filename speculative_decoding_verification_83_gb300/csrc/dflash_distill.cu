// dflash_distill.cu -- distillation of a drafter from its target's top logits:
// loss and gradient.
//
// Row r holds the student's logits z over the whole vocabulary and the
// teacher's K largest logits t_j with their tokens v_j. With a temperature T,
//   p = softmax(t / T) over the row's K entries,  q = softmax(z / T) over V,
//   loss_r = w_r sum_j p_j (log p_j - log q_{v_j}),
//   dloss_r / dz_v = w_r (q_v - sum of p_j with v_j = v) / T.
// Entries with token -1 do not take part; a row left without any, or with
// w_r = 0, has loss 0 and gradient 0, and its logits do not matter.
//
// Exponents are taken in base 2 with c = 1 / (T ln 2): the row's statistics
// are m = max z and s = sum_v 2^(c (z_v - m)), so that q_v = 2^(c (z_v - m)) / s
// and log q_v = (c (z_v - m) - log2 s) ln 2. The difference comes first: c z alone
// leaves fp32's range for logits near its ends (a row that is nothing but its
// type's lowest value), and is rounded to more than 1 from 2^24 on. All sums are
// fp32.
//
// What bounds it: reading the logits and writing the gradient, once each. A row
// is dealt out to a cluster of a few CTAs. Each moves the first 70 KB of its
// slice into shared memory by bulk copies, reduces the pieces as they land (a
// running maximum per thread), then the rest as it streams by; it sends its
// (m, s) to the other CTAs through distributed shared memory and writes the
// gradient, from shared memory and, for the rest, from L2, where the logits
// just read still are. Three CTAs share an SM, so that one's copies and stores
// fill the time of another's reductions and barriers: that counts for more
// than holding whole slices. Measured at 1920 x 248320 bf16, loss and
// gradient: clusters of 4 with 70 KB held 347 us (5.49 TB/s, 82% of a copy's
// measured rate), of 8 with whole slices held 406 us, of 2 453 us (more CTAs
// per row wait for their slowest, fewer read more again), of 4 with 110 KB and
// two CTAs an SM 583 us. The loss alone holds nothing back, and fewer CTAs per
// row are better: 158 us (6.0 TB/s) with 2, 182 us with 4. The teacher's K
// entries are one warp's work while the logits arrive. Per logit about 8
// instructions: maxima and multiply-adds work on pairs. The gradient alone
// (the backward call) is a plain stream: 306 us there (6.2 TB/s).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "dflash_paged.cuh"

namespace dflash {
namespace {

constexpr int kMaxSplit = 8;         // CTAs per row
constexpr int kPieces = 4;          // bulk copies of a slice
constexpr int kMaxHeld = 70 * 1024;  // bytes of a slice kept in shared memory: three fit an SM
constexpr float kMaxReference = 0x1p30f;  // of a row's statistics, in powers of 2: good to 2^5 of them
constexpr float kLog2eD = 1.4426950408889634f;
constexpr float kLn2D = 0.6931471805599453f;

__device__ __forceinline__ float ex2d(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// pairs of fp32 values in one register pair
__device__ __forceinline__ unsigned long long pair_of(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 floats_of(unsigned long long v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^(c (x - m)) of both values
__device__ __forceinline__ unsigned long long weights2(unsigned long long x, unsigned long long c2,
                                                       unsigned long long neg_m2) {
  const float2 a = floats_of(mul2(add2(x, neg_m2), c2));
  return pair_of(ex2d(a.x), ex2d(a.y));
}

struct B16 {  // bf16 logits: 8 to a vector
  static constexpr int kBytes = 2, kPer = 8;
  static __device__ __forceinline__ float load(const unsigned char* p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  }
  static __device__ __forceinline__ void store(unsigned char* p, float x) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)Bf16::pack(x, 0.0f);
  }
  static __device__ __forceinline__ void unpack(const uint4& u, unsigned long long (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair_of(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const unsigned long long (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = floats_of(x[i]);
      w[i] = Bf16::pack(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the largest of a vector's values (a NaN counts for nothing), on pairs
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float top(const uint4& a, const uint4& b) {
    const uint32_t m = max2(max2(max2(a.x, a.y), max2(a.z, a.w)), max2(max2(b.x, b.y), max2(b.z, b.w)));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
struct F32 {
  static constexpr int kBytes = 4, kPer = 4;
  static __device__ __forceinline__ float load(const unsigned char* p) { return *reinterpret_cast<const float*>(p); }
  static __device__ __forceinline__ void store(unsigned char* p, float x) { *reinterpret_cast<float*>(p) = x; }
  static __device__ __forceinline__ void unpack(const uint4& u, unsigned long long (&x)[2]) {
    x[0] = pair_of(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = pair_of(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const unsigned long long (&x)[2]) {
    const float2 a = floats_of(x[0]), b = floats_of(x[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
  static __device__ __forceinline__ float top(const uint4& a, const uint4& b) {
    return fmaxf(fmaxf(fmaxf(__uint_as_float(a.x), __uint_as_float(a.y)), fmaxf(__uint_as_float(a.z), __uint_as_float(a.w))),
                 fmaxf(fmaxf(__uint_as_float(b.x), __uint_as_float(b.y)), fmaxf(__uint_as_float(b.z), __uint_as_float(b.w))));
  }
};

// A part of a row: its largest logit m (-inf: no value above -inf yet) and s.
struct Stat {
  float ref, s;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
  Stat r;
  r.ref = fmaxf(a.ref, b.ref);
  // a side that has seen nothing carries its sum, 0 or NaN, as it is
  const float fa = a.ref == r.ref ? 1.0f : ex2d((a.ref - r.ref) * c),
              fb = b.ref == r.ref ? 1.0f : ex2d((b.ref - r.ref) * c);
  r.s = a.s * fa + b.s * fb;
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The join of the warp's 32 parts, in every lane.
__device__ __forceinline__ Stat warp_join(const Stat& a, float c) {
  Stat r;
  r.ref = warp_max_f32(a.ref);
  r.s = warp_sum(a.ref == r.ref ? a.s : a.s * ex2d((a.ref - r.ref) * c));
  return r;
}
// Two vectors into a running part: the reference moves up to their largest.
template <class T>
__device__ __forceinline__ void take(Stat& a, const uint4& u, const uint4& v, float c, unsigned long long c2) {
  const float m = T::top(u, v);
  if (m > a.ref) {
    a.s = a.ref == -INFINITY ? a.s : a.s * ex2d((a.ref - m) * c);
    a.ref = m;
  }
  const float neg = a.ref == -INFINITY ? 0.0f : -a.ref;
  const unsigned long long n2 = pair_of(neg, neg);
  unsigned long long x[T::kPer / 2], y[T::kPer / 2];
  T::unpack(u, x);
  T::unpack(v, y);
  unsigned long long s = add2(weights2(x[0], c2, n2), weights2(y[0], c2, n2));
#pragma unroll
  for (int i = 1; i < T::kPer / 2; ++i) s = add2(s, add2(weights2(x[i], c2, n2), weights2(y[i], c2, n2)));
  const float2 f = floats_of(s);
  a.s += f.x + f.y;
}
__device__ __forceinline__ void take_one(Stat& a, float x, float c) {
  a = join(a, Stat{x == x ? x : -INFINITY, x == -INFINITY ? 0.0f : x == x ? 1.0f : x}, c);
}

struct Teacher {
  int id[kMaxTeacher];     // -1: takes no part
  float p[kMaxTeacher];    // softmax(t / T)
  float log2p[kMaxTeacher];
  float z[kMaxTeacher];    // the student's logit there
  int empty;               // no entry takes part
};

// The row's teacher distribution, by one warp.
template <class T>
__device__ __forceinline__ void teacher_row(const DistillParams& p, long long r, const unsigned char* z, bool report,
                                            float c, Teacher& S) {
  const int lane = threadIdx.x & 31;
  float mx = -INFINITY;
  bool nan = false, outside = false;
  for (int j = lane; j < p.K; j += 32) {
    const int id = p.ids[r * p.K + j];
    const float t = p.teacher[r * p.K + j];
    const bool part = id >= 0 && id < p.V;
    outside |= !part && id != -1;
    S.id[j] = part ? id : -1;
    S.log2p[j] = t;
    S.z[j] = part ? T::load(z + (size_t)id * T::kBytes) : 0.0f;
    if (part) {
      nan |= !(t == t);
      mx = fmaxf(mx, t);
    }
  }
  mx = warp_max_f32(mx);
  nan = __any_sync(0xffffffffu, nan);
  float sum = 0.0f;
  for (int j = lane; j < p.K; j += 32) {
    const float d = (S.log2p[j] - mx) * c;
    const float e = S.id[j] >= 0 && S.log2p[j] != -INFINITY ? ex2d(d) : 0.0f;
    S.log2p[j] = d;
    S.p[j] = e;
    sum += e;
  }
  sum = warp_sum(sum);
  if (nan) sum = NAN;
  const float inv = 1.0f / sum, log2_sum = log2f(sum);
  for (int j = lane; j < p.K; j += 32) {
    S.p[j] = S.id[j] >= 0 ? S.p[j] * inv : 0.0f;
    S.log2p[j] -= log2_sum;
  }
  if (lane == 0) S.empty = mx == -INFINITY && !nan;
  if (report) {
    if (outside) raise_status(p.status, DFLASH_STATUS_BAD_TOKEN);
    if (lane == 0 && (nan || mx == INFINITY)) raise_status(p.status, DFLASH_STATUS_BAD_ROW);
  }
}

// The student's distribution: q = 2^(c (z - shift) + add) / s. For ordinary rows
// shift is 0 and add = -R, R = fl(c m), with s taken to it: one rounded
// multiply-add, the same in both gradients. Where R is rounded to too few bits
// for that, shift is the largest logit itself.
struct Student {
  float shift, add, s;
};
__device__ __forceinline__ Student student_of(const Stat& a, float c) {
  const float R = a.ref * c;
  if (fabsf(R) <= kMaxReference) return {0.0f, -R, a.s * ex2d(fmaf(a.ref, c, -R))};
  return {a.ref, 0.0f, a.s};
}

// The gradient at the teacher's tokens in [lo, hi), over what is written there.
template <class T>
__device__ __forceinline__ void teacher_gradient(const DistillParams& p, const Teacher& S, unsigned char* g, int lo,
                                                 int hi, float c, const Student& q, float coef) {
  for (int j = threadIdx.x; j < p.K; j += blockDim.x) {
    const int id = S.id[j];
    if (id < lo || id >= hi) continue;
    bool owner = true;  // of the entries with this token, the first writes their sum
    float sum = 0.0f;
    for (int i = 0; i < p.K; ++i)
      if (S.id[i] == id) {
        owner &= i >= j;
        sum += S.p[i];
      }
    if (owner) T::store(g + (size_t)id * T::kBytes, (ex2d(fmaf(S.z[j] - q.shift, c, q.add)) / q.s - sum) * coef);
  }
}

// A row's slice for one CTA, in vectors of the row's 16-byte-aligned body; the
// unaligned ends of the row belong to its first and last CTA.
template <class T>
struct Slice {
  int head, v0, v1, lo, hi, edge;
  __device__ __forceinline__ Slice(const unsigned char* z, int V, int rank, int split) {
    const int tid = threadIdx.x;
    head = min(V, (int)(((16 - ((uintptr_t)z & 15)) & 15) / T::kBytes));
    const int nv = (V - head) / T::kPer, per = (nv + split - 1) / split;
    v0 = min(nv, rank * per);
    v1 = min(nv, v0 + per);
    const int tail = head + nv * T::kPer;
    edge = -1;  // this thread's element of the ends
    if (rank == 0 && tid < head) edge = tid;
    if (rank == split - 1 && edge < 0 && tid >= 32 && tail + tid - 32 < V) edge = tail + tid - 32;
    lo = rank == 0 ? 0 : head + v0 * T::kPer;
    hi = rank == split - 1 ? V : head + v1 * T::kPer;
  }
};

// The gradient's vectors: 2^(c (z - shift) + add) f.
template <class T>
struct Writer {
  unsigned long long c2, n2, a2, f2;
  unsigned char* body;
  bool aligned;
  __device__ __forceinline__ Writer(const unsigned char* z, unsigned char* g, int head, float c, const Student& q, float f)
      : c2(pair_of(c, c)), n2(pair_of(-q.shift, -q.shift)), a2(pair_of(q.add, q.add)), f2(pair_of(f, f)), body(g + (size_t)head * T::kBytes),
        aligned((((uintptr_t)z ^ (uintptr_t)g) & 15) == 0) {}
  template <bool kShifted>
  __device__ __forceinline__ void put(int v, const uint4& u) const {
    unsigned long long x[T::kPer / 2];
    T::unpack(u, x);
#pragma unroll
    for (int i = 0; i < T::kPer / 2; ++i) {
      const float2 e = floats_of(fma2(kShifted ? add2(x[i], n2) : x[i], c2, a2));
      x[i] = mul2(pair_of(ex2d(e.x), ex2d(e.y)), f2);
    }
    if (aligned) {
      reinterpret_cast<uint4*>(body)[v] = T::pack(x);
    } else {
#pragma unroll
      for (int i = 0; i < T::kPer / 2; ++i) {
        const float2 f = floats_of(x[i]);
        T::store(body + ((size_t)v * T::kPer + 2 * i) * T::kBytes, f.x);
        T::store(body + ((size_t)v * T::kPer + 2 * i + 1) * T::kBytes, f.y);
      }
    }
  }
};

// The cluster's CTAs have started: one warp of each also publishes its barriers.
__device__ __forceinline__ void cluster_arrive(bool release) {
  if (release)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// a part into the same shared-memory place of the cluster's CTA number `rank`,
// then an arrival on the same barrier there
__device__ __forceinline__ void send_part(const Stat* at, const uint64_t* bar, uint32_t rank, const Stat& a) {
  uint32_t d, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_addr(at)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_addr(bar)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d), "f"(a.ref) : "memory");
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d + 4), "f"(a.s) : "memory");
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(b) : "memory");
}
// a bounded wait that also orders what the arriving CTAs stored
__device__ __forceinline__ bool wait_parts(uint64_t* bar) {
  unsigned long long t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar))
        : "memory");
    if (ok) return true;
    // longer than the pieces' limits together: no CTA leaves while another
    // may still send to it
    const unsigned long long t = global_timer_ns();
    if (t0 == 0)
      t0 = t;
    else if (t - t0 > (kPieces + 1) * kWaitLimitNs)
      return false;
  }
}
// barrier 1: the parts of the CTA's warps are in shared memory (warp 0 waits)
template <int kAll>
__device__ __forceinline__ void parts_ready(bool wait) {
  if (wait)
    asm volatile("bar.sync 1, %0;" ::"n"(kAll) : "memory");
  else
    asm volatile("bar.arrive 1, %0;" ::"n"(kAll) : "memory");
}

// ---- loss, and loss with gradient: CTA blockIdx.x % split of row blockIdx.x / split;
// a row's CTAs are one cluster. held: bytes of the slice kept in shared memory.
// kThreads threads work on the slice; one more warp takes the teacher's
// entries, whose two dependent loads would otherwise hold up a barrier.
template <class T, int kThreads, bool kGrad>
__global__ void __launch_bounds__(kThreads + 32, 1152 / (kThreads + 32))
    loss_kernel(const DistillParams p, int split, int held) {
  constexpr int kW = kThreads / 32;
  extern __shared__ __align__(128) unsigned char slice_mem[];
  __shared__ Teacher S;
  __shared__ uint64_t landed[kPieces];
  __shared__ Stat parts[kW];
  __shared__ __align__(8) Stat slices[kMaxSplit];  // every slice of the row
  __shared__ uint64_t exchanged;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) mbar_init(&landed[i], 1);
    mbar_init(&exchanged, (uint32_t)split);
    fence_barrier_init();
  }
  grid_dependency_sync();
  if (split > 1) {
    __syncwarp();
    cluster_arrive(warp == 0);
  }
  const long long r = blockIdx.x / (unsigned)split;
  const int rank = (int)(blockIdx.x - (unsigned)r * (unsigned)split);
  const float c = p.inv_t * kLog2eD;
  const unsigned long long c2 = pair_of(c, c);
  const unsigned char* z = p.z + (size_t)r * (size_t)p.z_stride * T::kBytes;
  unsigned char* g = kGrad ? p.grad + (size_t)r * (size_t)p.grad_stride * T::kBytes : nullptr;
  const Slice<T> L(z, p.V, rank, split);
  const uint4* body = reinterpret_cast<const uint4*>(z + (size_t)L.head * T::kBytes);
  const uint4* mine = reinterpret_cast<const uint4*>(slice_mem);
  const int n_held = min(L.v1 - L.v0, held / 16);
  // pieces in whole rounds of the CTA's vectors, two a thread
  const int piece = ((n_held + kPieces - 1) / kPieces + 2 * kThreads - 1) / (2 * kThreads) * (2 * kThreads);
  if (tid == 0)
    for (int i = 0; i < kPieces; ++i) {
      const int at = min(n_held, i * piece), n = min(n_held, at + piece) - at;
      if (n > 0) {
        mbar_arrive_expect_tx(&landed[i], (uint32_t)n * 16u);
        bulk_load(slice_mem + (size_t)at * 16, body + L.v0 + at, (uint32_t)n * 16u, &landed[i]);
      }
    }
  const float w = p.weight ? p.weight[r] : 1.0f;
  const float at_edge = L.edge >= 0 ? T::load(z + (size_t)L.edge * T::kBytes) : -INFINITY;
  __syncthreads();  // the barriers are initialised

  // ---- the slice's statistics
  Stat a = {-INFINITY, 0.0f};
  if (warp == kW) {
    teacher_row<T>(p, r, z, rank == 0 && w != 0.0f, c, S);
  } else {
    bool ok = true;
    const uint4 low = T::kBytes == 2 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                     : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);  // -inf
    for (int i = 0; i < kPieces; ++i) {
      const int at = min(n_held, i * piece), end = min(n_held, at + piece);
      if (end <= at) break;
      ok &= mbar_wait_landed(&landed[i], 0);
      for (int v = at + tid; v < end; v += 2 * kThreads)
        take<T>(a, mine[v], v + kThreads < end ? mine[v + kThreads] : low, c, c2);
    }
    for (int v = L.v0 + n_held + tid; v < L.v1; v += 2 * kThreads)
      take<T>(a, body[v], v + kThreads < L.v1 ? body[v + kThreads] : low, c, c2);
    if (L.edge >= 0) take_one(a, at_edge, c);
    if (!ok) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    a = warp_join(a, c);
    if (lane == 0) parts[warp] = a;
  }
  __syncwarp();
  parts_ready<kThreads + 32>(warp == 0 || split == 1);
  if (split > 1) {
    cluster_wait();  // every CTA of the row runs
    if (warp == 0) {
      a = warp_join(lane < kW ? parts[lane] : Stat{-INFINITY, 0.0f}, c);
      if (S.empty) a = Stat{0.0f, 0.0f};  // a row without entries: every CTA sends (0, 0)
      if (lane < split) send_part(&slices[rank], &exchanged, lane, a);
    }
    if (!wait_parts(&exchanged)) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    a = lane < split ? slices[lane] : Stat{-INFINITY, 0.0f};
  } else {
    a = S.empty ? Stat{0.0f, 0.0f} : lane < kW ? parts[lane] : Stat{-INFINITY, 0.0f};
  }
  __syncwarp();
  a = warp_join(a, c);  // the same bits in every warp of every CTA of the row
  const bool active = w != 0.0f && (a.s != 0.0f || a.ref == -INFINITY);
  if (fabsf(a.ref) == INFINITY) a.s = NAN;  // no logit above -inf, or +inf: the row has no distribution
  if (rank == 0 && warp == kW) {
    const float log2_s = log2f(a.s);
    float part = 0.0f;
    for (int j = lane; j < p.K; j += 32)
      if (S.id[j] >= 0 && S.p[j] != 0.0f) part += S.p[j] * (S.log2p[j] - ((S.z[j] - a.ref) * c - log2_s));
    part = warp_sum(part);
    if (lane == 0) {
      p.loss[r] = active ? part * kLn2D * w : 0.0f;
      if (p.lse) {
        const Student q = student_of(a, c);
        p.lse[2 * r] = !active ? 0.0f : q.shift == 0.0f ? -q.add : q.shift;
        p.lse[2 * r + 1] = !active ? 0.0f : q.shift == 0.0f ? q.s : -q.s;
      }
      if (active && !(a.s == a.s)) raise_status(p.status, DFLASH_STATUS_BAD_ROW);
    }
  }
  if (kGrad) {
    if (!active) {
      for (int i = L.lo + tid; i < L.hi; i += blockDim.x) T::store(g + (size_t)i * T::kBytes, 0.0f);
      return;
    }
    const Student q = student_of(a, c);
    const float coef = w * p.inv_t, f = coef / q.s;
    const Writer<T> out(z, g, L.head, c, q, f);
    auto write = [&](auto shifted) {
      for (int v = tid; v < n_held; v += kThreads) out.template put<decltype(shifted)::value>(L.v0 + v, mine[v]);
      for (int v = L.v0 + n_held + tid; v < L.v1; v += kThreads) out.template put<decltype(shifted)::value>(v, body[v]);
    };
    if (warp < kW) {
      if (__builtin_expect(q.shift != 0.0f, 0))
        write(std::true_type());
      else
        write(std::false_type());
    }
    if (L.edge >= 0) T::store(g + (size_t)L.edge * T::kBytes, ex2d(fmaf(at_edge - q.shift, c, q.add)) * f);
    __syncthreads();  // the slice is written
    teacher_gradient<T>(p, S, g, L.lo, L.hi, c, q, coef);
  }
}

// ---- the gradient alone, from the row's statistics: CTAs are independent.
constexpr int kGradThreads = 256;
constexpr int kGradHeld = 4;  // vectors a thread loads before it works on them
template <class T>
__global__ void __launch_bounds__(kGradThreads + 32) grad_kernel(const DistillParams p, int split) {
  __shared__ Teacher S;
  const int tid = threadIdx.x;
  grid_dependency_sync();
  const long long r = blockIdx.x / (unsigned)split;
  const int rank = (int)(blockIdx.x - (unsigned)r * (unsigned)split);
  const float c = p.inv_t * kLog2eD;
  const unsigned char* z = p.z + (size_t)r * (size_t)p.z_stride * T::kBytes;
  unsigned char* g = p.grad + (size_t)r * (size_t)p.grad_stride * T::kBytes;
  const Slice<T> L(z, p.V, rank, split);
  const uint4* body = reinterpret_cast<const uint4*>(z + (size_t)L.head * T::kBytes);
  uint4 u[kGradHeld];
#pragma unroll
  for (int i = 0; i < kGradHeld; ++i) {
    const int v = L.v0 + i * kGradThreads + tid;
    if (tid < kGradThreads && v < L.v1) u[i] = body[v];
  }
  const float at_edge = L.edge >= 0 ? T::load(z + (size_t)L.edge * T::kBytes) : 0.0f;
  const Stat a = {p.lse[2 * r], p.lse[2 * r + 1]};
  const Student q = a.s < 0.0f ? Student{a.ref, 0.0f, -a.s} : Student{0.0f, -a.ref, a.s};
  float w = p.weight ? p.weight[r] : 1.0f;
  if (p.upstream) w *= p.upstream[r * p.upstream_stride];
  if (w == 0.0f || a.s == 0.0f) {  // the statistics of a row that has no part are (0, 0)
    for (int i = L.lo + tid; i < L.hi; i += blockDim.x) T::store(g + (size_t)i * T::kBytes, 0.0f);
    return;
  }
  if (tid >= kGradThreads) teacher_row<T>(p, r, z, false, c, S);
  if (g == z) __syncthreads();  // in place: the teacher's logits are read before they are written over
  const float coef = w * p.inv_t, f = coef / q.s;
  const Writer<T> out(z, g, L.head, c, q, f);
  auto write = [&](auto shifted) {
    for (int v = L.v0 + tid; v < L.v1 && tid < kGradThreads; v += kGradHeld * kGradThreads) {
#pragma unroll
      for (int i = 0; i < kGradHeld; ++i)
        if (v + i * kGradThreads < L.v1) out.template put<decltype(shifted)::value>(v + i * kGradThreads, u[i]);
#pragma unroll
      for (int i = 0; i < kGradHeld; ++i) {
        const int n = v + (kGradHeld + i) * kGradThreads;
        if (n < L.v1) u[i] = body[n];
      }
    }
  };
  if (__builtin_expect(q.shift != 0.0f, 0))
    write(std::true_type());
  else
    write(std::false_type());
  if (L.edge >= 0) T::store(g + (size_t)L.edge * T::kBytes, ex2d(fmaf(at_edge - q.shift, c, q.add)) * f);
  __syncthreads();  // the slice is written
  teacher_gradient<T>(p, S, g, L.lo, L.hi, c, q, coef);
}

int launch_cfg(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, long long grid, int threads, size_t smem,
               int cluster, void* stream) {
  cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return 0;
}

template <class T, int kThreads, bool kGrad>
int launch_split(const DistillParams& p, int split, int held, void* stream) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(loss_kernel<T, kThreads, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxHeld);
    if (e != cudaSuccess) return (int)e;
    ready[dev] = true;
  }
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_cfg(cfg, attr, (long long)p.rows * split, kThreads + 32, (size_t)held, split, stream);
  return (int)cudaLaunchKernelEx(&cfg, loss_kernel<T, kThreads, kGrad>, p, split, held);
}

// CTAs per row: slices of at most 128 KB (256 KB for the loss alone), and,
// where the rows alone would leave SMs idle, up to 8 CTAs with at least 8 KB
// each. Slices of up to 16 KB take 128 threads, of which 9 CTAs fit an SM.
template <class T, bool kGrad>
int launch_loss(const DistillParams& p, int sms, void* stream) {
  const long long bytes = (long long)p.V * T::kBytes;
  int split = 1;
  while (split < kMaxSplit && bytes > split * (kGrad ? 131072LL : 262144LL)) split *= 2;
  while (split < kMaxSplit && (long long)p.rows * split < 2LL * sms && bytes / (2 * split) >= 8192) split *= 2;
  const long long slice = ((bytes + split - 1) / split + 31) / 16 * 16;
  const int held = slice < kMaxHeld ? (int)slice : kMaxHeld;
  return slice <= 16384 ? launch_split<T, 96, kGrad>(p, split, held, stream)
                        : launch_split<T, 352, kGrad>(p, split, held, stream);
}

template <class T>
int launch_grad(const DistillParams& p, void* stream) {
  // slices of 32 KB
  const long long bytes = (long long)p.V * T::kBytes;
  long long split = (bytes + 32767) / 32768;
  const long long most = 0x7fffffffLL / p.rows;
  if (split > most) split = most;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  launch_cfg(cfg, attr, (long long)p.rows * split, kGradThreads + 32, 0, 1, stream);
  return (int)cudaLaunchKernelEx(&cfg, grad_kernel<T>, p, (int)split);
}

}  // namespace

int launch_distill_loss(const DistillParams& p, int dtype, int sms, void* stream) {
  return dtype == DFLASH_BF16 ? launch_loss<B16, false>(p, sms, stream) : launch_loss<F32, false>(p, sms, stream);
}
int launch_distill_grad(const DistillParams& p, int dtype, void* stream) {
  return dtype == DFLASH_BF16 ? launch_grad<B16>(p, stream) : launch_grad<F32>(p, stream);
}
int launch_distill_loss_grad(const DistillParams& p, int dtype, int sms, void* stream) {
  return dtype == DFLASH_BF16 ? launch_loss<B16, true>(p, sms, stream) : launch_loss<F32, true>(p, sms, stream);
}

}  // namespace dflash
