// dflash_attention.cu -- attention of a few new tokens per request over a paged
// key/value cache: one token each in plain decoding, the block of drafts in
// verification.
//
// For query row r (new token i of request b, query head h G + g of key/value
// head h): x_j = scale q_r . k_j over the keys j the row sees (all L of the
// request, or the first L - n + i + 1 with n new tokens and a causal mask),
// out = sum_j e^{x_j} v_j / sum_j e^{x_j}, lse = log sum_j e^{x_j}. A row that
// sees no key gives 0 and -inf.
//
// What bounds it: every key and value is read once for the n G rows that
// share its head, 2 n G flops per byte of a 16-bit cache, so the reads of the
// cache bound it until n G nears 100 rows. Design:
//  * Work is a list of units (request, head, 16 query rows), each a run of
//    64-key tiles (128 where a row of the cache has 128 bytes or less); the list's
//    tiles are dealt out in equal contiguous runs, one per CTA, whatever the
//    requests' lengths. A unit that spans CTAs
//    leaves unnormalised partial results (fp32 sum, maximum, sum of weights)
//    in the workspace, which a second kernel joins in a fixed order: the
//    results do not depend on timing.
//  * In a CTA each of four warps takes its own 16 (or 32) keys of every tile, with a
//    ring of its own in shared memory filled by asynchronous 16-byte copies,
//    which address any page size, stride and order; no barrier of the CTA is
//    needed until the unit ends, where the warps' results are joined through
//    shared memory. The ring runs on into the next unit.
//  * S = Q K^T and O += P V by m16n8k16 tensor instructions with fp32
//    accumulators; P leaves the S registers as the second product's operand.
//    The running maximum rescales O only in steps where a maximum moved.
//  * e4m3 caches are widened in registers, exactly, to f16. q is then scaled
//    per row by a power of two into f16's range (exact but for values
//    below 2^-31 of the row's largest), undone in the scores.
// Measured on one GB300 (bytes of keys and values over time): 64 requests of up
// to 8192 positions, 64 query and 8 key/value heads of 128, bf16: 199 us, 6.2
// TB/s, 92% of a copy's rate; three CTAs an SM with two ring stages each beat
// two with three (206 us). A step's overhead (page indexes, maxima, the rescaling
// vote) is per warp, so rows of 128 bytes take 32 keys a step: head_dim 64 (twice
// the positions) 196 against 274 us with 16, e4m3 at head_dim 128 (two requests of
// 200001 positions) 145 us, 5.6 TB/s, against 164 us. There, and more so for e4m3
// at head_dim 64 (131 us for 92 us of bytes), the warps' chain of widening,
// products and softmax bounds it. At head_dim 256 O alone takes 128 registers a
// thread, which leaves 4 warps an SM (e4m3: 8): 264 us for 181 us of bytes (64
// requests of up to 4096 positions), e4m3 285 us for 192 (8192). Copies of K and V in groups of their own, each
// reissued as its half of the stage is read, were slower (217 us): twice the waits
// and shuffles.
// Rounding: P is rounded to the operands' type (half a step of its own
// relative to each weight; f16: down to 2^-29 of a row's largest); all sums,
// maxima and exponents are fp32.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_attention.cuh"

namespace dflash {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kRows = 16;                  // query rows per unit
// f16 holds normal numbers from 2^-14 to below 2^16: a row's reference lies this
// many powers of 2 below its largest score, so that weights are rounded by half a
// step of their own down to 2^-29 of the largest. (bf16 has the range of fp32.)
constexpr float kTopF16 = 15.0f;
constexpr int kMaxCtas = 640;              // CTAs whose partial results the workspace holds

__host__ __device__ inline AttnGeometry warp_geometry(int tile) { return {kRows, tile, kMaxCtas}; }

struct Unit {
  int b, h, rb, L, first, n, tiles;
  long long start;  // index of its first tile in the whole list
};

// The unit that tile t of the list belongs to (pre: tiles before each request).
template <int kTile>
__device__ __forceinline__ Unit locate(const AttnParams& p, const long long* pre, long long t) {
  Unit u;
  int lo = 0, hi = p.tk.B;  // largest b with pre[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  u.b = lo;
  bool bad = false;
  request_tokens(p.tk, lo, u.first, u.n, bad);
  u.L = clamped_len(p, lo, bad);
  u.tiles = tiles_of<kTile>(u.L);
  const int rbs = row_blocks<kRows>(u.n, p.G);
  const long long k = (t - pre[lo]) / u.tiles;
  u.h = (int)(k / rbs);
  u.rb = (int)(k - (long long)u.h * rbs);
  u.start = pre[lo] + k * u.tiles;
  return u;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  const int n = take ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <bool kF8, int D>
struct Shape {
  static constexpr int kRowBytes = kF8 ? D : 2 * D;
  static constexpr int kWarpKeys = kRowBytes <= 128 ? 32 : 16;  // keys of a warp's step: 4 to 16 KB of keys and values
  static constexpr int kTile = kWarps * kWarpKeys;              // keys per tile
  static constexpr int kHalfStage = kWarpKeys * kRowBytes;  // K or V of one warp's step
  static constexpr int kStageBytes = 2 * kHalfStage * kWarps;
  // CTAs per SM, and a ring that fills the SM's shared memory with them
  static constexpr int kPerSm = D < 256 ? 3 : kF8 ? 2 : 1;  // as registers allow: O alone takes D / 2 a thread
  static constexpr int kRing = kPerSm == 3 ? 65536 : kPerSm == 2 ? 98304 : 196608;
  static constexpr int kStages = kRing / kStageBytes;
  static constexpr int kCols = 32;  // columns of O joined at a time
  static constexpr size_t kMerge = (size_t)kWarps * kRows * (kCols + 1) * sizeof(float);
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kMerge + 2 * kWarps * kRows * sizeof(float);
};

// Shared-memory place of 16-byte piece c of row r: pieces of a row are
// exchanged so that the 8 rows of one matrix load fall in different banks.
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return kRowBytes >= 128 ? r * kRowBytes + ((c ^ (r & 7)) << 4) : r * kRowBytes + ((c ^ ((r >> 1) & 3)) << 4);
}

template <class T, bool kF8, int D>
__global__ void __launch_bounds__(kAttnThreads, Shape<kF8, D>::kPerSm) attention_kernel(const AttnParams p) {
  using S = Shape<kF8, D>;
  using M = typename std::conditional<kF8, F16, T>::type;  // the products' type
  constexpr int kWarpKeys = S::kWarpKeys, kTile = S::kTile;
  constexpr uint32_t kAllKeys = kWarpKeys == 32 ? 0xffffffffu : 0xffffu;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem;
  float* merge = reinterpret_cast<float*>(smem + (size_t)S::kStages * S::kStageBytes);
  float* merge_ml = merge + S::kMerge / sizeof(float);
  long long* pre = reinterpret_cast<long long*>(merge_ml + 2 * kWarps * kRows);
  __shared__ long long warp_sum[kWarps];
  __shared__ int replaced;  // values of the unit that are not finite have been replaced
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_dependency_sync();

  // ---- the list: tiles before each request
  bool bad = false;
  {
    const int chunk = (p.tk.B + kAttnThreads - 1) / kAttnThreads;
    const int lo = min(p.tk.B, tid * chunk), hi = min(p.tk.B, lo + chunk);
    long long mine = 0;
    for (int b = lo; b < hi; ++b) {
      int first, n;
      request_tokens(p.tk, b, first, n, bad);
      pre[b] = mine;
      mine += (long long)row_blocks<kRows>(n, p.G) * p.c.kv_heads * tiles_of<kTile>(clamped_len(p, b, bad));
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int b = lo; b < hi; ++b) pre[b] += before;
    if (tid == 0) {
      pre[p.tk.B] = warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
      replaced = 0;
    }
    __syncthreads();
  }
  if (bad && blockIdx.x == 0) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
  const long long total = pre[p.tk.B];
  const long long run = max((long long)kMinRun, (total + gridDim.x - 1) / gridDim.x);
  if (blockIdx.x == 0 && tid == 0) *reinterpret_cast<long long*>(p.ws) = run;
  const long long t_begin = (long long)blockIdx.x * run, t_end = min(total, t_begin + run);
  if (tid == 0) {
    SplitUnit s = {0, 0, 0, 0, 0, 0, 0};
    if (t_begin < t_end) {
      const Unit u = locate<kTile>(p, pre, t_end - 1);
      if (u.start >= t_begin && u.start + u.tiles > t_end) s = {u.start, u.tiles, u.h, u.rb, u.first, u.n, 0};
    }
    split_units(p)[blockIdx.x] = s;
  }
  if (t_begin >= t_end) return;

  // ---- this warp's ring: one step = this warp's kWarpKeys keys of a tile
  const uint32_t my_ring = smem_addr(ring) + warp * 2 * S::kHalfStage;
  __shared__ uint32_t step_mask[kWarps][8];  // per stage: the keys that exist and have a page

  Unit lu = locate<kTile>(p, pre, t_begin);  // the unit being loaded
  long long lt = t_begin;
  int l_stage = 0;
  uint32_t next_off = 0;
  bool next_ok = false, bad_page = false;
  auto look_up = [&]() {  // lane l: the row of key l of step lt
    const int key = (int)(lt - lu.start) * kTile + warp * kWarpKeys + (lane & (kWarpKeys - 1));
    next_ok = key < lu.L;
    int page = 0, slot = 0, id = 0;
    if (next_ok) {
      split_position(p.c, key, page, slot);
      id = p.c.table[(long long)lu.b * p.c.table_stride + page];
      if (id < 0 || id >= p.c.num_pages) {
        bad_page = true;
        next_ok = false;
        id = 0;
      }
    }
    next_off = next_ok ? row_offset(p.c, id, lu.h, slot) : 0u;
  };
  look_up();
  constexpr int kPieces = S::kRowBytes / 16;        // pieces per row
  constexpr int kLoads = kWarpKeys * kPieces / 32;  // per lane, for K and for V each
  auto load_step = [&]() {
    if (lt < t_end) {
      const uint32_t ok = __ballot_sync(0xffffffffu, next_ok);
      const uint32_t base = my_ring + l_stage * S::kStageBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = i * 32 + lane, r = at / kPieces, c = at % kPieces;
        const uint32_t off = __shfl_sync(0xffffffffu, next_off, r);
        const bool take = (ok >> r) & 1u;
        const size_t o = ((size_t)off + c) * 16u;
        const uint32_t d = base + piece_at<S::kRowBytes>(r, c);
        cp_async16(d, p.c.k + o, take);
        cp_async16(d + S::kHalfStage, p.c.v + o, take);
      }
      if (lane == 0) step_mask[warp][l_stage] = ok;
      ++lt;
      if (lt < t_end) {
        if (lt >= lu.start + lu.tiles) lu = locate<kTile>(p, pre, lt);
        look_up();
      }
    }
    cp_commit();
    l_stage = l_stage + 1 == S::kStages ? 0 : l_stage + 1;
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) load_step();

  const int qr = lane >> 2, qc = lane & 3;
  // ldmatrix source rows: K, lanes 0-15 address the keys 0-7 (two 16-byte
  // column pieces), lanes 16-31 the keys 8-15
  int stage = 0;
  long long t = t_begin;
  while (t < t_end) {
    const Unit u = locate<kTile>(p, pre, t);
    const long long u_end = min(t_end, u.start + u.tiles);
    // ---- this thread's two query rows
    int row_tok[2], row_head[2], vis[2];
    float unit_scale[2];
    bool row_ok[2];
    uint32_t q[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = u.rb * kRows + qr + 8 * e;
      const int i = r / p.G;
      row_ok[e] = r < u.n * p.G;
      row_tok[e] = u.first + i;
      row_head[e] = u.h * p.G + (r - i * p.G);
      vis[e] = !row_ok[e] ? 0 : p.causal ? min(u.L, max(0, u.L - u.n + i + 1)) : u.L;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + 2 * ((long long)row_tok[e] * p.q_ts + (long long)row_head[e] * p.q_hs));
      float mult = 1.0f;
      if (!kF8) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          q[ks][e] = row_ok[e] ? src[8 * ks + qc] : 0u;
          q[ks][2 + e] = row_ok[e] ? src[8 * ks + 4 + qc] : 0u;
        }
      } else {
        // an 8-bit matrix load gives a thread four neighbouring values of a
        // key: values 4 qc .. 4 qc + 3 of 16 stand for the product's inner
        // indexes 2 qc, 2 qc + 1, 2 qc + 8, 2 qc + 9
        float big = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          q[ks][e] = row_ok[e] ? src[8 * ks + 2 * qc] : 0u;
          q[ks][2 + e] = row_ok[e] ? src[8 * ks + 2 * qc + 1] : 0u;
          const float2 f = T::unpack(q[ks][e]), g = T::unpack(q[ks][2 + e]);
          big = fmaxf(fmaxf(fmaxf(big, fabsf(f.x)), fabsf(f.y)), fmaxf(fabsf(g.x), fabsf(g.y)));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // the row's largest value into [2^14, 2^15): the exponent alone,
        // limited so that both factors stay normal numbers
        const int ex = min(max((int)(__float_as_uint(big) >> 23) - 141, -120), 120);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        mult = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const float2 f = T::unpack(q[ks][e]), g = T::unpack(q[ks][2 + e]);
          q[ks][e] = F16::pack(f.x * down, f.y * down);
          q[ks][2 + e] = F16::pack(g.x * down, g.y * down);
        }
      }
      unit_scale[e] = p.scale * mult;
      if (kF8 && p.c.k_scale) unit_scale[e] *= p.c.k_scale[u.h];
      unit_scale[e] *= kLog2e;
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};

    for (; t < u_end; ++t) {
      cp_wait<S::kStages - 2>();
      __syncwarp();
      load_step();  // into the stage whose step every lane has finished
      const uint32_t kb = my_ring + stage * S::kStageBytes, vb = kb + S::kHalfStage;
      const uint32_t ok = step_mask[warp][stage] & kAllKeys;
      // ---- S = Q K^T
      float s[kWarpKeys / 8][4];
#pragma unroll
      for (int i = 0; i < kWarpKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
      if (!kF8) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int g = 0; g < kWarpKeys / 16; ++g) {
            uint32_t k4[4];  // keys 0-7: inner 0-7, 8-15; keys 8-15: the same
            ldsm4(k4, kb + piece_at<S::kRowBytes>(16 * g + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
            M::mma(s[2 * g], q[ks], k4[0], k4[1]);
            M::mma(s[2 * g + 1], q[ks], k4[2], k4[3]);
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += 2)
#pragma unroll
          for (int g = 0; g < kWarpKeys / 16; ++g) {
            uint32_t k4[4];  // keys 0-7: values 0-15, 16-31; keys 8-15: the same
            ldsm4(k4, kb + piece_at<S::kRowBytes>(16 * g + (lane & 7) + ((lane >> 4) << 3), ks + ((lane >> 3) & 1)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t lo, hi;
              widen4(k4[j], lo, hi);
              M::mma(s[2 * g], q[ks + j], lo, hi);
              widen4(k4[2 + j], lo, hi);
              M::mma(s[2 * g + 1], q[ks + j], lo, hi);
            }
          }
      }
      // ---- scale, mask, running maximum
      const int key0 = (int)(t - u.start) * kTile + warp * kWarpKeys;
      const bool masked = ok != kAllKeys || key0 + kWarpKeys > u.L - (p.causal ? u.n : 0);
      float mx[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int nb = 0; nb < kWarpKeys / 8; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[nb][e] * unit_scale[e >> 1];
          if (masked) {
            const int kk = 8 * nb + 2 * qc + (e & 1);
            if (!((ok >> kk) & 1u) || key0 + kk >= vis[e >> 1]) x = kNegInf;
          }
          s[nb][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      float keep[2];
      bool moved = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        if (std::is_same<M, F16>::value) mx[e] -= kTopF16;
        const float m_new = fmaxf(m[e], mx[e]);
        moved |= m_new > m[e];
        // no key seen yet: any finite reference will do
        const float ref = m_new == kNegInf ? 0.0f : m_new;
        keep[e] = ex2(m[e] - ref);
        m[e] = m_new;
        float sum = 0.0f;
#pragma unroll
        for (int nb = 0; nb < kWarpKeys / 8; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float w = ex2(s[nb][2 * e + j] - ref);
            s[nb][2 * e + j] = w;
            sum += w;
          }
        l[e] = l[e] * keep[e] + sum;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= keep[0];
          o[i][1] *= keep[0];
          o[i][2] *= keep[1];
          o[i][3] *= keep[1];
        }
      }
      // ---- O += P V
      // Under a causal mask a step may hold values that only some rows see:
      // those that are not finite are replaced by 0.
      if (masked && p.causal && u.n > 1) {
        uint4* own = reinterpret_cast<uint4*>(ring + (vb - smem_addr(ring))) + lane;
        bool found = false;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          uint4 w = own[i * 32];
          found |= drop_not_finite<T, kF8>(w.x) | drop_not_finite<T, kF8>(w.y) | drop_not_finite<T, kF8>(w.z) |
                   drop_not_finite<T, kF8>(w.w);
        }
        if (__builtin_expect(__any_sync(0xffffffffu, found), 0)) {
#pragma unroll 1
          for (int i = 0; i < kLoads; ++i) {
            uint4 w = own[i * 32];
            drop_not_finite<T, kF8>(w.x);
            drop_not_finite<T, kF8>(w.y);
            drop_not_finite<T, kF8>(w.z);
            drop_not_finite<T, kF8>(w.w);
            own[i * 32] = w;
          }
          if (lane == 0) replaced = 1;
          __syncwarp();
        }
      }
#pragma unroll
      for (int g = 0; g < kWarpKeys / 16; ++g) {
        const float(&a)[4] = s[2 * g], (&b)[4] = s[2 * g + 1];
        const uint32_t pa[4] = {M::pack(a[0], a[1]), M::pack(a[2], a[3]), M::pack(b[0], b[1]), M::pack(b[2], b[3])};
        const int vr = 16 * g + (lane & 7) + (((lane >> 3) & 1) << 3);
        if (!kF8) {
#pragma unroll
          for (int ds = 0; ds < D / 16; ++ds) {
            uint32_t v4[4];  // values 0-7: keys 0-7, 8-15; values 8-15: the same
            ldsm4t(v4, vb + piece_at<S::kRowBytes>(vr, 2 * ds + (lane >> 4)));
            M::mma(o[2 * ds], pa, v4[0], v4[1]);
            M::mma(o[2 * ds + 1], pa, v4[2], v4[3]);
          }
        } else {
          // a transposed load of byte pairs: even values in bytes 0 and 2, odd
          // ones in 1 and 3, of two neighbouring keys
#pragma unroll
          for (int ds = 0; ds < D / 16; ds += 2) {
            uint32_t v4[4];  // values 0-15: keys 0-7, 8-15; values 16-31: the same
            ldsm4t(v4, vb + piece_at<S::kRowBytes>(vr, ds + (lane >> 4)));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t even0, odd0, even1, odd1;
              widen4(__byte_perm(v4[2 * j], 0, 0x3120), even0, odd0);
              widen4(__byte_perm(v4[2 * j + 1], 0, 0x3120), even1, odd1);
              M::mma(o[2 * (ds + j)], pa, even0, even1);
              M::mma(o[2 * (ds + j) + 1], pa, odd0, odd1);
            }
          }
        }
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }

    // ---- the unit (or this CTA's run of it) ends: join the warps
    const long long seg_begin = max(t_begin, u.start);
    const bool whole = seg_begin == u.start && u_end == u.start + u.tiles;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (qc == 0) {
        merge_ml[2 * (warp * kRows + qr + 8 * e)] = m[e];
        merge_ml[2 * (warp * kRows + qr + 8 * e) + 1] = l[e];
      }
    }
    __syncthreads();
    float mine[2];  // this warp's factor for its two rows
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = kNegInf;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, merge_ml[2 * (w * kRows + qr + 8 * e)]);
      mine[e] = m[e] == kNegInf ? 0.0f : ex2(m[e] - top);
    }
    // each thread then owns row jr and columns jc .. jc + 3 of each run of 32
    const int jr = tid >> 3, jc = (tid & 7) * 4;
    float top = kNegInf, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, merge_ml[2 * (w * kRows + jr)]);
    for (int w = 0; w < kWarps; ++w) {
      const float mw = merge_ml[2 * (w * kRows + jr)], lw = merge_ml[2 * (w * kRows + jr) + 1];
      sum += mw != kNegInf ? lw * ex2(mw - top) : lw == lw ? 0.0f : lw;  // a NaN sum stays one
    }
    const int jrow = u.rb * kRows + jr, ji = jrow / p.G;
    const bool jok = jrow < u.n * p.G;
    const long long jtok = u.first + ji, jhead = u.h * p.G + (jrow - ji * p.G);
    const long long slot = 2LL * blockIdx.x + (seg_begin == t_begin ? 0 : 1);
    float* part_o = reinterpret_cast<float*>(p.ws + warp_geometry(kTile).o()) + (slot * kRows + jr) * D;
    float factor = reciprocal_or_zero(sum);
    if (kF8 && p.c.v_scale) factor *= p.c.v_scale[u.h];
    if ((tid & 7) == 0 && jok) {
      if (whole) {
        if (p.lse) p.lse[jtok * ((long long)p.G * p.c.kv_heads) + jhead] = (top + log2f(sum)) * kLn2;
      } else {
        reinterpret_cast<Part*>(p.ws + warp_geometry(kTile).ml())[slot * kRows + jr] = {top, sum};
      }
    }
    bool odd = replaced;  // or a result is not finite
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += S::kCols) {
      __syncthreads();
#pragma unroll
      for (int nb = 0; nb < S::kCols / 8; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // columns of the accumulators: two neighbours per 8, or (8-bit) the
          // even values of 16 in one block and the odd ones in the next
          const int col = kF8 ? 16 * (nb >> 1) + 2 * (2 * qc + (e & 1)) + (nb & 1) : 8 * nb + 2 * qc + (e & 1);
          merge[(warp * kRows + qr + 8 * (e >> 1)) * (S::kCols + 1) + col] = o[c0 / 8 + nb][e] * mine[e >> 1];
        }
      __syncthreads();
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] += merge[(w * kRows + jr) * (S::kCols + 1) + jc + j];
      // (a row whose sum of weights is not finite has NaN everywhere)
      odd |= jok && sum < INFINITY && (x[0] * 0.0f + x[1] * 0.0f) + (x[2] * 0.0f + x[3] * 0.0f) != 0.0f;
      if (jok) {
        if (whole) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + 2 * (jtok * p.o_ts + jhead * p.o_hs + c0 + jc));
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(T::pack(x[0] * factor, x[1] * factor), T::pack(x[2] * factor, x[3] * factor));
        } else {
          *reinterpret_cast<float4*>(part_o + c0 + jc) = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
    }
    if (__builtin_expect(__syncthreads_or(odd), 0)) {  // (merge and merge_ml are written again)
      // results that values which are not finite decide
      int* first = reinterpret_cast<int*>(merge);
      for (int i = tid; i < 3 * D; i += kAttnThreads) first[i] = kNever;
      replaced = 0;
      __syncthreads();
      find_not_finite<T, kF8, D>(p, u.b, u.h, (int)(seg_begin - u.start) * kTile,
                                 (int)min((long long)u.L, (u_end - u.start) * kTile), first, tid, kAttnThreads);
      __syncthreads();
      if (jok && sum < INFINITY) {
        const int jvis = p.causal ? min(u.L, max(0, u.L - u.n + ji + 1)) : u.L;
        for (int d = tid & 7; d < D; d += 8) {
          const float v = not_finite_value<D>(first, d, jvis);
          if (v == 0.0f) continue;
          if (whole)
            reinterpret_cast<uint16_t*>(p.out + 2 * (jtok * p.o_ts + jhead * p.o_hs))[d] = (uint16_t)T::pack(v, 0.0f);
          else
            part_o[d] = v;
        }
      }
      __syncthreads();
    }
  }
  if (bad_page) raise_status(p.status, DFLASH_STATUS_BAD_PAGE);
  cp_wait<0>();
}

// ---- joining the partial results of units that span CTAs -------------------------------
// CTA (c, z): 16 rows of the unit that begins in CTA c's run, one warp each. The
// segments' maxima give their factors, then the segments are summed in list
// order. A chain of three loads bounds it, so every row has its warp and a warp
// 16 segments in flight.
constexpr int kJoinWarps = 16;
// A column of a unit whose segments' sum x is not finite: the sum of the partial
// results that are not, whatever their segments weigh (x where all are finite).
__device__ __forceinline__ float not_finite_sum(const float* first, const float* rest, long long step, int n, float x) {
  float s = fabsf(*first) < INFINITY ? 0.0f : *first;
  for (int c = 0; c < n; ++c) {
    const float y = rest[c * step];
    if (!(fabsf(y) < INFINITY)) s += y;
  }
  return s != 0.0f ? s : x;
}
template <class T, bool kF8, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const AttnParams p, const AttnGeometry geo) {
  constexpr int kPer = D / 32;  // columns of a lane
  grid_dependency_sync();
  const int lane = threadIdx.x & 31, c0 = blockIdx.x, jr = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const SplitUnit u = split_units(p)[c0];
  const long long run = *reinterpret_cast<const long long*>(p.ws);
  if (u.tiles == 0 || jr >= min(geo.rows, u.n * p.G - u.rb * geo.rows)) return;
  const int c1 = (int)((u.start + u.tiles - 1) / run);
  const Part* parts = reinterpret_cast<const Part*>(p.ws + geo.ml());
  const float* os = reinterpret_cast<const float*>(p.ws + geo.o());
  const long long slot0 = 2LL * c0 + (u.start == (long long)c0 * run ? 0 : 1);
  auto slot_row = [&](int c) { return (c == c0 ? slot0 : 2LL * c) * geo.rows + jr; };
  Part mine = {kNegInf, 0.0f};  // this lane's segment of the first 32
  if (c0 + lane <= c1) mine = parts[slot_row(c0 + lane)];
  float top = mine.m;
  for (int c = c0 + 32 + lane; c <= c1; c += 32) top = fmaxf(top, parts[slot_row(c)].m);
  top = warp_max_f32(top);
  float x[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
  float sum = 0.0f;
  for (int cb = c0; cb <= c1; cb += 32) {
    if (cb > c0) mine = cb + lane <= c1 ? parts[slot_row(cb + lane)] : Part{kNegInf, 0.0f};
    const float w = mine.m == kNegInf ? 0.0f : ex2(mine.m - top), l = part_sum(mine, top);
    const int cnt = min(32, c1 - cb + 1);
#pragma unroll 16
    for (int j = 0; j < cnt; ++j) {
      const float* src = os + slot_row(cb + j) * D + lane * kPer;
      float y[kPer];
#pragma unroll
      for (int e = 0; e < kPer; e += 2) *reinterpret_cast<float2*>(y + e) = *reinterpret_cast<const float2*>(src + e);
      const float wj = __shfl_sync(0xffffffffu, w, j);
      sum += __shfl_sync(0xffffffffu, l, j);
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] = fmaf(y[e], wj, x[e]);
    }
  }
  // a partial result that is not finite counts whatever its segment weighs
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (__builtin_expect(!(fabsf(x[e]) < INFINITY), 0))
      x[e] = not_finite_sum(os + slot_row(c0) * D + lane * kPer + e, os + slot_row(c0 + 1) * D + lane * kPer + e, 2LL * geo.rows * D, c1 - c0, x[e]);
  float factor = reciprocal_or_zero(sum);
  if (kF8 && p.c.v_scale) factor *= p.c.v_scale[u.h];
  const int g = u.rb * geo.rows + jr, ti = g / p.G;
  const long long tok = u.first + ti, head = u.h * p.G + g - ti * p.G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + 2 * (tok * p.o_ts + head * p.o_hs)) + lane * (kPer / 2);
#pragma unroll
  for (int e = 0; e < kPer; e += 2) dst[e / 2] = T::pack(x[e] * factor, x[e + 1] * factor);
  if (lane == 0 && p.lse) p.lse[tok * ((long long)p.G * p.c.kv_heads) + head] = (top + log2f(sum)) * kLn2;
}

template <class T, bool kF8, int D>
int launch(const AttnParams& p, int sms, void* stream) {
  using S = Shape<kF8, D>;
  const size_t smem = S::kSmem + (size_t)(p.tk.B + 1) * sizeof(long long);
  static int ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attention_kernel<T, kF8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(S::kSmem + (kOpsMaxB + 1) * sizeof(long long)));
    if (e != cudaSuccess) return (int)e;
    ready[dev] = 1;
  }
  int grid = sms * S::kPerSm;
  if (grid > kMaxCtas) grid = kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, attention_kernel<T, kF8, D>, p);
  if (e != cudaSuccess) return (int)e;
  return launch_join(p, warp_geometry(S::kTile), grid, std::is_same<T, Bf16>::value ? DFLASH_BF16 : DFLASH_F16, kF8, D, stream);
}

template <class T, bool kF8>
int pick_dim(const AttnParams& p, int d, int sms, void* stream) {
  return d == 64    ? launch<T, kF8, 64>(p, sms, stream)
         : d == 128 ? launch<T, kF8, 128>(p, sms, stream)
                    : launch<T, kF8, 256>(p, sms, stream);
}

template <class T, bool kF8, int D>
int launch_join_dim(const AttnParams& p, const AttnGeometry& g, int grid, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((g.rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  return (int)cudaLaunchKernelEx(&cfg, join_kernel<T, kF8, D>, p, g);
}
template <class T, bool kF8>
int launch_join_type(const AttnParams& p, const AttnGeometry& g, int grid, int d, void* stream) {
  return d == 64    ? launch_join_dim<T, kF8, 64>(p, g, grid, stream)
         : d == 128 ? launch_join_dim<T, kF8, 128>(p, g, grid, stream)
                    : launch_join_dim<T, kF8, 256>(p, g, grid, stream);
}

}  // namespace

int launch_join(const AttnParams& p, const AttnGeometry& g, int grid, int dtype, bool f8, int head_dim, void* stream) {
  if (dtype == DFLASH_BF16)
    return f8 ? launch_join_type<Bf16, true>(p, g, grid, head_dim, stream)
              : launch_join_type<Bf16, false>(p, g, grid, head_dim, stream);
  return f8 ? launch_join_type<F16, true>(p, g, grid, head_dim, stream)
            : launch_join_type<F16, false>(p, g, grid, head_dim, stream);
}

size_t attention_workspace(int head_dim) {
  const size_t a = warp_geometry(0).bytes(head_dim), b = tc_geometry(128, head_dim).bytes(head_dim);
  return a > b ? a : b;
}

// By the query rows that share a key/value head, per request on average. Up to
// 16 rows go to the warps' own products, which read the cache once for them
// (64 single tokens, 8 rows: 198 us; the tensor-memory kernel 207 us). From 17 on
// they would read it again for every 16 rows: at 32 requests of up to 16384
// positions and 8 key/value heads of 128, 32 rows take 422 us against 197 us, 64
// rows 704 against 218 us. 8-bit caches have half the bytes to read again and the
// widening to pay: 32 rows 204 against 252 us, 64 rows 386 against 296 us, so
// they change over after 32; at head_dim 256 they stay with the warps.
int launch_attention(const AttnParams& p, int dtype, int cache_dtype, int head_dim, int sms, void* stream) {
  const bool f8 = cache_dtype == DFLASH_E4M3;
  const long long rows = (((long long)p.tk.tokens + p.tk.B - 1) / p.tk.B) * p.G;
  if (f8 ? rows > 32 && head_dim != 256 : rows > 16)
    return launch_attention_tc(p, rows <= 32 ? 32 : rows <= 64 ? 64 : 128, dtype, f8, head_dim, sms, stream);
  if (dtype == DFLASH_BF16)
    return f8 ? pick_dim<Bf16, true>(p, head_dim, sms, stream) : pick_dim<Bf16, false>(p, head_dim, sms, stream);
  return f8 ? pick_dim<F16, true>(p, head_dim, sms, stream) : pick_dim<F16, false>(p, head_dim, sms, stream);
}

}  // namespace dflash
