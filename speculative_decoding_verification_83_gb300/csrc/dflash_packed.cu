// dflash_packed.cu -- attention over packed sequences: the formulas, the lists of
// work, and the rows that are gone through one by one.
//
// out_i = sum_j e^(s q_i k_j) v_j / sum_j e^(s q_i k_j) over the keys j that row i
// sees, lse_i = log of that sum. Backward, with p_ij = e^(s q_i k_j - lse_i) and
// delta_i = sum over d of dout_id out_id:
//   dv_j = sum_i p_ij dout_i, ds_ij = p_ij (dout_i v_j - delta_i),
//   dq_i = s sum_j ds_ij k_j, dk_j = s sum_i ds_ij q_i,
// i over the rows, of all query heads that share the key's head, that see key j.
//
// The products run on the tensor cores (dflash_packed_fwd.cu, dflash_packed_bwd.cu),
// where a masked pair counts as a weight of 0, and 0 times a value that is not
// finite is NaN. So they flag what came out not finite, and here one warp takes
// each such row: 32 keys (queries) at a time, a score per lane, then D / 32 columns
// per lane; pairs that do not see each other take no part, whatever they hold.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

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

// Row t of the outputs: query i of n over m keys from kv0 on. One warp; D / 8 lanes read a
// key, 32 of which are scored at a time, and a lane ends with the score of its own.
template <class T, int D>
__device__ void attend_row(const PackedParams& p, int t, int head, int i, int n, int kv0, int m) {
  constexpr int kLanes = D / 8, kWords = D / 64, kAtOnce = 8;  // of a key; a lane's columns of V, in pairs; keys in flight
  constexpr uint32_t kExponents = std::is_same<T, F16>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t kCarry = std::is_same<T, F16>::value ? 0x04000400u : 0x00800080u;
  const int lane = threadIdx.x & 31, part = lane % kLanes, kh = head / p.G, vis = seen_keys(p.causal, n, m, i);
  const long long r = (long long)t * p.q_heads + head;
  unsigned char* out = row_of(p.o, t, head);
  float2 q[4];
  {
    const uint4 u = reinterpret_cast<const uint4*>(row_of(p.q, t, head))[part];
    q[0] = T::unpack(u.x), q[1] = T::unpack(u.y), q[2] = T::unpack(u.z), q[3] = T::unpack(u.w);
  }
  float top = -INFINITY, sum = 0.0f, acc[D / 32] = {};
  uint32_t odd[D / 32] = {};  // values seen that are not finite: +inf (1), -inf (2), NaN (4)
  for (int j0 = 0; j0 < vis; j0 += 32) {
    const int count = min(32, vis - j0);
    float s[kLanes];
#pragma unroll
    for (int k0 = 0; k0 < kLanes; k0 += kAtOnce) {
      uint4 u[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        u[k] = reinterpret_cast<const uint4*>(row_of(p.k, kv0 + j0 + min(k0 + k + lane - part, count - 1), kh))[part];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float2 a = T::unpack(u[k].x), b = T::unpack(u[k].y), c = T::unpack(u[k].z), d = T::unpack(u[k].w);
        s[k0 + k] = fmaf(q[0].x, a.x, fmaf(q[0].y, a.y, fmaf(q[1].x, b.x, q[1].y * b.y))) +
                    fmaf(q[2].x, c.x, fmaf(q[2].y, c.y, fmaf(q[3].x, d.x, q[3].y * d.y)));
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < o; ++k) {
        const bool hi = lane & o;
        s[k] = (hi ? s[k + o] : s[k]) + __shfl_xor_sync(kAll, hi ? s[k] : s[k + o], o);
      }
    const float x = lane < count ? s[0] * p.scale : -INFINITY;
    const float m1 = warp_max_f32(fmaxf(x, top)), ref = m1 == -INFINITY ? 0.0f : m1;
    const float f = expf(top - ref), w = expf(x - ref);  // (a score that is NaN leaves NaN)
    sum = sum * f + warp_sum(w);
    top = m1;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] *= f;
    for (int k0 = 0; k0 < count; k0 += kAtOnce) {
      uint32_t v[kAtOnce][kWords];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const unsigned char* from = row_of(p.v, kv0 + j0 + min(k0 + k, count - 1), kh) + 4 * kWords * lane;
#pragma unroll
        for (int e = 0; e < kWords; ++e) v[k][e] = reinterpret_cast<const uint32_t*>(from)[e];
      }
      uint32_t special = 0;  // a pair's exponent of all ones carries into its top bits
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
        for (int e = 0; e < kWords; ++e) special |= (v[k][e] & kExponents) + kCarry;
      if (!__any_sync(kAll, special & 0x80008000u)) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const float wk = __shfl_sync(kAll, w, (k0 + k) & 31);  // (0 from `count` on: no lane sees those keys)
#pragma unroll
          for (int e = 0; e < kWords; ++e) {
            const float2 y = T::unpack(v[k][e]);
            acc[2 * e] = fmaf(wk, y.x, acc[2 * e]);
            acc[2 * e + 1] = fmaf(wk, y.y, acc[2 * e + 1]);
          }
        }
        continue;
      }
      for (int k = k0; k < min(count, k0 + kAtOnce); ++k) {
        const float wk = __shfl_sync(kAll, w, k);
        const unsigned char* row = row_of(p.v, kv0 + j0 + k, kh);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const float y = value<T>(row, lane * (D / 32) + c);
          if (fabsf(y) < INFINITY)
            acc[c] = fmaf(wk, y, acc[c]);
          else
            odd[c] |= y > 0.0f ? 1u : y < 0.0f ? 2u : 4u;
        }
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const int d = lane * (D / 32) + c;
    float y = acc[c] * inv;
    if (odd[c] && y == y) y = odd[c] == 1u ? INFINITY : odd[c] == 2u ? -INFINITY : NAN;
    const uint32_t hi = T::pack(y, 0.0f) & 0xffffu;
    reinterpret_cast<uint16_t*>(out)[d] = (uint16_t)hi;
    if (p.low) p.low[r * D + d] = low_bits(y, hi);
  }
  if (p.lse && lane == 0) p.lse[r] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

// Goes through the flags; row(t, head, i, unit) is called by one warp for every row
// of a flagged 32, for any of its kSame flags.
template <int kPer, int kSame, class F>
__device__ __forceinline__ void each_flagged(const PackedList& list, const uint8_t* flags, int heads, F row) {
  const long long total = (long long)*list.count * heads * kPer;
  const int warp = threadIdx.x >> 5;
  for (long long base = (long long)blockIdx.x * blockDim.x; base < total; base += (long long)gridDim.x * blockDim.x) {
    const long long at = base + threadIdx.x;
    if (!__syncthreads_or(at < total && flags[at])) continue;
    for (long long f = base; f < min(total, base + blockDim.x); ++f) {
      if (!flags[f]) continue;
      const int part = (int)(f % kPer) / kSame, head = (int)(f / kPer % heads);
      const PackedUnit u = list.units[f / kPer / heads];
      for (int r = 32 * part + warp; r < min(u.rows, 32 * part + 32); r += kWarps) row(u.row0 + r, head, u.i0 + r, u);
    }
  }
}
// Rows of no sequence: pieces of 8 values set to 0.
template <int D, class F>
__device__ __forceinline__ void each_spare(const int32_t* start, int B, int tokens, int heads, F piece) {
  const int lo = min(max(start[0], 0), tokens), hi = max(lo, min(max(start[B], 0), tokens));
  const long long n = (long long)(lo + tokens - hi) * heads * (D / 8);
  for (long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x; at < n; at += (long long)gridDim.x * blockDim.x) {
    const int c = (int)(at % (D / 8)), head = (int)(at / (D / 8) % heads), r = (int)(at / (D / 8) / heads);
    piece(r < lo ? r : hi + r - lo, head, c);
  }
}
__device__ __forceinline__ void clear8(const HeadRows& h, int t, int head, int c) {
  reinterpret_cast<uint4*>(row_of(h, t, head))[c] = make_uint4(0u, 0u, 0u, 0u);
}

template <int D>
__device__ __forceinline__ void clear_spare(const PackedParams& p) {
  each_spare<D>(p.q_start, p.B, p.q_tokens, p.q_heads, [&](int t, int head, int c) {
    clear8(p.o, t, head, c);
    const long long r = (long long)t * p.q_heads + head;
    if (p.low) reinterpret_cast<uint2*>(p.low + r * D)[c] = make_uint2(0u, 0u);
    if (p.lse && c == 0) p.lse[r] = -INFINITY;
  });
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps)
    redo_forward_kernel(const PackedParams p, const PackedList list, const uint8_t* flags) {
  grid_dependency_sync();
  each_flagged<kForwardFlags, 2>(list, flags, p.q_heads, [&](int t, int head, int i, const PackedUnit& u) {
    if (row_not_finite<T, D>(row_of(p.o, t, head))) attend_row<T, D>(p, t, head, i, u.n, u.other0, u.m);
  });
  if (p.fill) clear_spare<D>(p);
}

// Prompts of few words: a warp a row, in one launch where the tensor cores' way takes
// three. Latency bounds both. Replayed, 32 + 8 heads of 128: one prompt of 7 tokens 6.2
// against 14.3 us, of 32 tokens 12.3 against 14.4, of 64 tokens 18.4 against 14.5 (but 23
// against 27 called directly); 16 prompts of 4 tokens 10.2 against 28.6. A batch's offsets
// are on the GPU, so the rule goes by what all its keys, in one sequence, would take.
constexpr int kFewKeys = 64, kFewRows = 4096, kFewWarps = 2;
constexpr int kFewBatch = 32 * kFewWarps - 1;  // (a thread an offset)
template <class T, int D>
__global__ void __launch_bounds__(32 * kFewWarps) few_rows_kernel(const PackedParams p) {
  __shared__ int starts[2][kFewBatch + 1];
  grid_dependency_sync();
  if (threadIdx.x <= p.B) {
    starts[0][threadIdx.x] = p.q_start[threadIdx.x];
    starts[1][threadIdx.x] = p.kv_start[threadIdx.x];
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, warps = gridDim.x * kFewWarps;
  int next = blockIdx.x * kFewWarps + warp;  // this warp's next row, counted from the sequence's first
  bool bad = false;
  for (int b = 0; b < p.B; ++b) {
    int q0, n, k0, m;
    extent(starts[0], p.q_tokens, b, q0, n, bad);
    extent(starts[1], p.kv_tokens, b, k0, m, bad);
    for (; next < n * p.q_heads; next += warps) {
      const int i = next / p.q_heads;
      attend_row<T, D>(p, q0 + i, next - i * p.q_heads, i, n, k0, m);
    }
    next -= n * p.q_heads;
  }
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
  if (p.fill) clear_spare<D>(p);
}

// Row t of the queries' gradients.
template <class T, int D>
__device__ void dq_row(const PackedParams& p, int t, int head, int i, int n, int kv0, int m, float* q_row, float* g_row) {
  const int lane = threadIdx.x & 31, kh = head / p.G, vis = seen_keys(p.causal, n, m, i);
  const long long r = (long long)t * p.q_heads + head;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    q_row[lane + 32 * c] = value<T>(row_of(p.q, t, head), lane + 32 * c);
    g_row[lane + 32 * c] = value<T>(row_of(p.d_o, t, head), lane + 32 * c);
  }
  __syncwarp();
  const float lse = p.lse[r], delta = -p.row_stats[((size_t)head * 2 + 1) * p.stat_pitch + t];
  float acc[D / 32] = {};
  for (int j0 = 0; j0 < vis; j0 += 32) {
    const int j = j0 + lane, count = min(32, vis - j0);
    float ds = 0.0f;
    if (j < vis) {
      const float x = dot<T, D>(q_row, row_of(p.k, kv0 + j, kh)) * p.scale;
      ds = expf(x - lse) * (dot<T, D>(g_row, row_of(p.v, kv0 + j, kh)) - delta) * p.scale;
    }
    for (int k = 0; k < count; ++k) {
      const float w = __shfl_sync(kAll, ds, k);
      const unsigned char* row = row_of(p.k, kv0 + j0 + k, kh);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(w, value<T>(row, lane + 32 * c), acc[c]);
    }
    bool lost = true;  // every column is NaN: nothing brings it back
#pragma unroll
    for (int c = 0; c < D / 32; ++c) lost &= acc[c] != acc[c];
    if (__all_sync(kAll, lost)) break;
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) put<T>(row_of(p.dq, t, head), lane + 32 * c, lse == -INFINITY ? 0.0f : acc[c]);
}

// Row t of the keys' and values' gradients: key j of m, n queries from q0 on.
template <class T, int D>
__device__ void dkv_row(const PackedParams& p, int t, int kh, int j, int m, int q0, int n, float* k_row, float* v_row) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    k_row[lane + 32 * c] = value<T>(row_of(p.k, t, kh), lane + 32 * c);
    v_row[lane + 32 * c] = value<T>(row_of(p.v, t, kh), lane + 32 * c);
  }
  __syncwarp();
  float ak[D / 32] = {}, av[D / 32] = {};
  const int i_first = first_query(p.causal, n, m, j);
  bool lost = false;
  for (int g = 0; g < p.G && !lost; ++g) {
    const int head = kh * p.G + g;
    for (int i0 = i_first; i0 < n && !lost; i0 += 32) {
      const int i = i0 + lane, count = min(32, n - i0);
      float w = 0.0f, ds = 0.0f;
      if (i < n) {
        const long long at = (long long)(q0 + i) * p.q_heads + head;
        const float x = dot<T, D>(k_row, row_of(p.q, q0 + i, head)) * p.scale, lse = p.lse[at];
        w = lse == -INFINITY ? 0.0f : expf(x - lse);
        ds = w * (dot<T, D>(v_row, row_of(p.d_o, q0 + i, head)) + p.row_stats[((size_t)head * 2 + 1) * p.stat_pitch + q0 + i]) * p.scale;
      }
      for (int k = 0; k < count; ++k) {
        const float wk = __shfl_sync(kAll, w, k), dsk = __shfl_sync(kAll, ds, k);
        const unsigned char *qr = row_of(p.q, q0 + i0 + k, head), *gr = row_of(p.d_o, q0 + i0 + k, head);
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
    put<T>(row_of(p.dk, t, kh), lane + 32 * e, ak[e]);
    put<T>(row_of(p.dv, t, kh), lane + 32 * e, av[e]);
  }
}

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps)
    redo_grad_kernel(const PackedParams p, const PackedList queries, const uint8_t* q_flags, const PackedList keys,
                     const uint8_t* kv_flags) {
  __shared__ float rows[kWarps][2][D];
  grid_dependency_sync();
  const int warp = threadIdx.x >> 5;
  each_flagged<kGradFlags, 4>(queries, q_flags, p.q_heads, [&](int t, int head, int i, const PackedUnit& u) {
    if (!row_not_finite<T, D>(row_of(p.dq, t, head))) return;
    dq_row<T, D>(p, t, head, i, u.n, u.other0, u.m, rows[warp][0], rows[warp][1]);
  });
  each_flagged<kGradFlags, 4>(keys, kv_flags, p.kv_heads, [&](int t, int head, int j, const PackedUnit& u) {
    if (!row_not_finite<T, D>(row_of(p.dk, t, head)) && !row_not_finite<T, D>(row_of(p.dv, t, head))) return;
    dkv_row<T, D>(p, t, head, j, u.n, u.other0, u.m, rows[warp][0], rows[warp][1]);
  });
  if (!p.fill) return;
  each_spare<D>(p.q_start, p.B, p.q_tokens, p.q_heads, [&](int t, int head, int c) { clear8(p.dq, t, head, c); });
  each_spare<D>(p.kv_start, p.B, p.kv_tokens, p.kv_heads, [&](int t, int head, int c) {
    clear8(p.dk, t, head, c);
    clear8(p.dv, t, head, c);
  });
}

// The list of units: counted and sorted by one block. Work goes by how many of the
// other array's rows the unit's last (queries) or first (keys) row meets; units of equal work keep
// no order among themselves, which no result depends on.
constexpr int kListThreads = 1024, kPrepareThreads = 512, kBuckets = 1024;
template <int kN>  // threads
__device__ __noinline__ void build_list(const PackedParams& p, bool keys, int rows, const PackedList& list) {
  __shared__ int before[kMaxBatch], warp_sum_[kN / 32], bucket[kBuckets];
  const int32_t *sa = keys ? p.kv_start : p.q_start, *sb = keys ? p.q_start : p.kv_start;
  const int ta = keys ? p.kv_tokens : p.q_tokens, tb = keys ? p.q_tokens : p.kv_tokens;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  // units before each sequence (2^28 at most, where offsets name every row in every sequence)
  int done = 0;
  for (int b0 = 0; b0 < p.B; b0 += kN) {
    const int b = b0 + tid;
    int mine = 0;
    if (b < p.B) {
      int first, n;
      extent(sb, tb, b, first, n, bad);
      extent(sa, ta, b, first, n, bad);
      mine = (n + rows - 1) / rows;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum_[warp] = incl;
    __syncthreads();
    int pre = 0, all = 0;
    for (int w = 0; w < kN / 32; ++w) {
      if (w < warp) pre += warp_sum_[w];
      all += warp_sum_[w];
    }
    if (b < p.B) before[b] = done + pre + incl - mine;
    done += all;
    __syncthreads();
  }
  // offsets that do not ascend may name more units than the list holds
  const int total = min(done, most_units(ta, p.B, rows));
  if (tid == 0) *list.count = total;
  for (int i = tid; i < kBuckets; i += kN) bucket[i] = 0;
  __syncthreads();
  auto unit_at = [&](int k, int& work) {
    int lo = 0, hi = p.B;  // the last b with before[b] <= k
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= k)
        lo = mid;
      else
        hi = mid;
    }
    PackedUnit u = {};
    int first, fb;
    extent(sa, ta, lo, first, u.n, bad);
    extent(sb, tb, lo, fb, u.m, bad);
    u.i0 = (k - before[lo]) * rows;
    u.row0 = first + u.i0;
    u.rows = min(rows, u.n - u.i0);
    u.other0 = fb;
    const int meets = keys ? u.m - first_query(p.causal, u.m, u.n, u.i0) : seen_keys(p.causal, u.n, u.m, u.i0 + u.rows - 1);
    work = kBuckets - 1 - min(kBuckets - 1, (max(0, meets) + 127) / 128);  // most work: bucket 0
    return u;
  };
  for (int k = tid; k < total; k += kN) {
    int work;
    unit_at(k, work);
    atomicAdd(&bucket[work], 1);
  }
  __syncthreads();
  {
    constexpr int kPer = kBuckets / kN;  // buckets of a thread, side by side
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) mine += bucket[tid * kPer + k];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum_[warp] = incl;
    __syncthreads();
    int pre = incl - mine;
    for (int w = 0; w < warp; ++w) pre += warp_sum_[w];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int n = bucket[tid * kPer + k];
      bucket[tid * kPer + k] = pre;
      pre += n;
    }
  }
  __syncthreads();
  for (int k = tid; k < total; k += kN) {
    int work;
    const PackedUnit u = unit_at(k, work);
    list.units[atomicAdd(&bucket[work], 1)] = u;
  }
  if (bad) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
}

__global__ void __launch_bounds__(kListThreads) list_kernel(const PackedParams p, const PackedList list) {
  grid_dependency_sync();
  build_list<kListThreads>(p, false, kForwardRows, list);
}

// What the gradients' kernels read: both lists (the first two blocks), and the rows'
// statistics: delta, the sum over d of dout out, and lse, their signs reversed; behind
// the last row a tile's worth of zeros. D / 8 lanes take four tokens of a head at a time,
// whose loads are in flight together and whose statistics lie side by side (8192 tokens,
// 32 heads of 128, 168 MB: 38 us, one token at a time 47, 1024 threads a block 40).
template <class T, int D>
__global__ void __launch_bounds__(kPrepareThreads, 2)
    grad_prepare_kernel(const PackedParams p, const PackedList queries, const PackedList keys) {
  constexpr unsigned kLanes = D / 8;  // 8 values each
  grid_dependency_sync();
  if (blockIdx.x < 2) {
    build_list<kPrepareThreads>(p, blockIdx.x == 1, kGradRows, blockIdx.x ? keys : queries);
    return;
  }
  const long long id = (long long)(blockIdx.x - 2) * kPrepareThreads + threadIdx.x;
  const unsigned lane = threadIdx.x % kLanes;
  const unsigned unit = (unsigned)(id / kLanes), head = unit % (unsigned)p.q_heads;  // (as many as rows / 4: below 2^32)
  const long long t0 = unit / (unsigned)p.q_heads * 4ll;
  const int spare = p.stat_pitch - p.q_tokens, left = (int)(p.q_tokens - t0 < 4 ? p.q_tokens - t0 : 4);
  for (long long at = id; at < spare * 2ll * p.q_heads; at += (long long)(gridDim.x - 2) * kPrepareThreads)
    p.row_stats[at / spare * p.stat_pitch + p.q_tokens + at % spare] = 0.0f;
  uint4 a[4], g[4];
  uint2 l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    a[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
    l[k] = make_uint2(0u, 0u);
    if (k >= left) continue;
    a[k] = reinterpret_cast<const uint4*>(row_of(p.o, (int)t0 + k, (int)head))[lane];
    g[k] = reinterpret_cast<const uint4*>(row_of(p.d_o, (int)t0 + k, (int)head))[lane];
    if (p.low) l[k] = reinterpret_cast<const uint2*>(p.low + ((t0 + k) * p.q_heads + head) * D)[lane];
  }
  float s[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, y[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
    const uint32_t low[2] = {l[k].x, l[k].y};
    s[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = low[e >> 1] >> (16 * (e & 1));
      const float2 v = T::unpack(y[e]);
      s[k] = fmaf(with_low(x[e] & 0xffffu, (int8_t)(b & 0xffu)), v.x,
                  fmaf(with_low(x[e] >> 16, (int8_t)((b >> 8) & 0xffu)), v.y, s[k]));
    }
  }
  // lane k of each four ends with token k's sum
  const bool odd = lane & 1u, high = lane & 2u;
  const float s01 = (odd ? s[1] : s[0]) + __shfl_xor_sync(kAll, odd ? s[0] : s[1], 1);
  const float s23 = (odd ? s[3] : s[2]) + __shfl_xor_sync(kAll, odd ? s[2] : s[3], 1);
  float sum = (high ? s23 : s01) + __shfl_xor_sync(kAll, high ? s01 : s23, 2);
#pragma unroll
  for (unsigned o = 4; o < kLanes; o <<= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if ((int)lane < left) {  // (no more than 4)
    const long long t = t0 + lane;
    const float lse = p.lse[t * p.q_heads + head];
    float* st = p.row_stats + (size_t)head * 2 * p.stat_pitch;
    st[t] = lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f;
    st[p.stat_pitch + t] = -sum;
  }
}

template <class... A>
int launch(void (*kernel)(A...), unsigned grid, unsigned threads, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}
// Blocks for the flags' kernels: a thread a flag, which in sound data is all they do.
unsigned redo_blocks(long long flags) {
  const long long n = (flags + 32 * kWarps - 1) / (32 * kWarps);
  return (unsigned)(n < 1 ? 1 : n < 304 ? n : 304);
}

}  // namespace

int launch_redo_forward(const PackedParams& p, int dtype, int d, const PackedList& list, const uint8_t* flags,
                        void* stream) {
  const unsigned grid = redo_blocks((long long)most_units(p.q_tokens, p.B, kForwardRows) * p.q_heads * kForwardFlags);
  if (dtype == DFLASH_BF16)
    return d == 64 ? launch(redo_forward_kernel<Bf16, 64>, grid, 32u * kWarps, stream, p, list, flags)
                   : launch(redo_forward_kernel<Bf16, 128>, grid, 32u * kWarps, stream, p, list, flags);
  return d == 64 ? launch(redo_forward_kernel<F16, 64>, grid, 32u * kWarps, stream, p, list, flags)
                 : launch(redo_forward_kernel<F16, 128>, grid, 32u * kWarps, stream, p, list, flags);
}
// ---- workspaces
// Forward: the list of queries, their flags. Backward: delta, both lists, both sets of flags.
namespace {
size_t up(size_t n) { return (n + 255) / 256 * 256; }
size_t flag_bytes(int tokens, int B, int rows, int heads) {
  return up((size_t)most_units(tokens, B, rows) * heads * (rows == kForwardRows ? kForwardFlags : kGradFlags));
}
// Rows of a head's statistics: a multiple of 4, and room behind the last row for a whole tile.
int stat_pitch(int tokens) { return (tokens + 131) / 4 * 4; }
}  // namespace

size_t packed_workspace(int B, int q_tokens, int kv_tokens, int q_heads, int kv_heads, int head_dim, bool backward) {
  if (!backward) return list_bytes(q_tokens, B, kForwardRows) + flag_bytes(q_tokens, B, kForwardRows, q_heads);
  return up((size_t)stat_pitch(q_tokens) * q_heads * 2 * sizeof(float)) + list_bytes(q_tokens, B, kGradRows) +
         flag_bytes(q_tokens, B, kGradRows, q_heads) + list_bytes(kv_tokens, B, kGradRows) +
         flag_bytes(kv_tokens, B, kGradRows, kv_heads);
}

int launch_packed(const PackedParams& p, int dtype, int head_dim, int sms, void* stream) {
  if (!p.low && p.kv_tokens <= kFewKeys && p.B <= kFewBatch && (long long)p.q_tokens * p.q_heads <= kFewRows) {
    const int rows = p.q_tokens * p.q_heads;
    const unsigned grid = (unsigned)(rows < kFewWarps ? 1 : (rows + kFewWarps - 1) / kFewWarps);
    if (dtype == DFLASH_BF16)
      return head_dim == 64 ? launch(few_rows_kernel<Bf16, 64>, grid, 32u * kFewWarps, stream, p)
                            : launch(few_rows_kernel<Bf16, 128>, grid, 32u * kFewWarps, stream, p);
    return head_dim == 64 ? launch(few_rows_kernel<F16, 64>, grid, 32u * kFewWarps, stream, p)
                          : launch(few_rows_kernel<F16, 128>, grid, 32u * kFewWarps, stream, p);
  }
  const PackedList list = list_at(p.ws);
  uint8_t* flags = p.ws + list_bytes(p.q_tokens, p.B, kForwardRows);
  int e = launch(list_kernel, 1u, (unsigned)kListThreads, stream, p, list);
  if (!e) e = launch_forward_tc(p, dtype, head_dim, list, flags, sms, stream);
  return e ? e : launch_redo_forward(p, dtype, head_dim, list, flags, stream);
}

int launch_packed_grad(const PackedParams& p0, int head_dim, int sms, void* stream) {
  PackedParams p = p0;
  unsigned char* ws = p.ws;
  p.row_stats = reinterpret_cast<float*>(ws);
  p.stat_pitch = stat_pitch(p.q_tokens);
  ws += up((size_t)p.stat_pitch * p.q_heads * 2 * sizeof(float));
  const PackedList queries = list_at(ws);
  ws += list_bytes(p.q_tokens, p.B, kGradRows);
  uint8_t* q_flags = ws;
  ws += flag_bytes(p.q_tokens, p.B, kGradRows, p.q_heads);
  const PackedList keys = list_at(ws);
  ws += list_bytes(p.kv_tokens, p.B, kGradRows);
  uint8_t* kv_flags = ws;
  const long long lanes = (p.q_tokens + 3ll) / 4 * p.q_heads * (head_dim / 8);
  const unsigned blocks = 2u + (unsigned)((lanes + kPrepareThreads - 1) / kPrepareThreads);
  int e = head_dim == 64 ? launch(grad_prepare_kernel<Bf16, 64>, blocks, (unsigned)kPrepareThreads, stream, p, queries, keys)
                         : launch(grad_prepare_kernel<Bf16, 128>, blocks, (unsigned)kPrepareThreads, stream, p, queries, keys);
  if (!e && p.q_tokens) e = launch_dq_tc(p, head_dim, queries, q_flags, sms, stream);
  if (!e && p.kv_tokens) e = launch_dkv_tc(p, head_dim, keys, kv_flags, p.q_tokens > 0, sms, stream);
  if (e) return e;
  const unsigned redo = redo_blocks((long long)most_units(p.q_tokens, p.B, kGradRows) * p.q_heads * kGradFlags +
                                    (long long)most_units(p.kv_tokens, p.B, kGradRows) * p.kv_heads * kGradFlags);
  e = head_dim == 64 ? launch(redo_grad_kernel<Bf16, 64>, redo, 32u * kWarps, stream, p, queries,
                              (const uint8_t*)q_flags, keys, (const uint8_t*)kv_flags)
                     : launch(redo_grad_kernel<Bf16, 128>, redo, 32u * kWarps, stream, p, queries,
                              (const uint8_t*)q_flags, keys, (const uint8_t*)kv_flags);
  return e;
}

}  // namespace dflash
