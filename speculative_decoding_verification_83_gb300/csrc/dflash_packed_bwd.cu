// dflash_packed_bwd.cu -- the gradients of attention over packed sequences on the
// 5th-generation tensor cores (bf16).
//
// Scores are computed again, P = 2^(s q k log2 e - lse log2 e), and
// dS = P (dP - delta) with dP = dO V^T. Two kernels, so that every sum has one place
// and one order (no atomics), at 7 products per pair of tiles instead of 5:
//  * keys: a unit is 128 keys of one head, for all queries of the heads that share it.
//    The products are laid out transposed, keys as rows: S^T = K Q^T, dP^T = V dO^T, and
//    P^T, dS^T take the scores' place in tensor memory, where dV += P^T dO and
//    dK += dS^T Q read them. All of tensor memory is in use (4 x 128 columns).
//  * queries: a unit is 128 queries of one head: S = Q K^T, dP = dO V^T, dQ += dS K, with
//    two buffers of scores.
// What bounds both: the products. They are issued in an order that leaves each
// exchange with the threads in the shadow of two products: dV(j), S(j + 1) run while
// dS(j) is made, dK(j), dP(j + 1) while P(j + 1) is. 8 warps make P and dS, two for each quarter
// of the lanes, half of the columns each; since the results take the scores' place, the
// two meet once they have read (`met`). The rows' lse and delta lie as pairs by head,
// made with delta ahead of the kernels; for the keys' kernel 128 of them come with each
// tile of dO. Masks select P = 0 and dS = 0 in tiles at a border only. Rows with a result that is not
// finite are flagged (see dflash_packed.cuh). Every wait is bounded; a CTA that gives up
// raises DFLASH_STATUS_TIMEOUT.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_packed_mma.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 320, kMmaWarp = 8, kLoadWarp = 9, kWorkWarps = 8;
constexpr int kTileRows = 128;
constexpr uint32_t kStatBytes = 1040;  // 130 pairs: 128 from an even place on, or from the one after it

template <int D>
struct GradShape {
  static constexpr uint32_t kTile = 128u * D * 2u;
  // keys: K, V; tiles of Q and of dO. queries: Q, dO; tiles of K and of V.
  static constexpr int kFirst = D == 128 ? 3 : 5, kSecond = D == 128 ? 2 : 4;
  static constexpr uint32_t kRing1 = 2 * kTile, kRing2 = kRing1 + kFirst * kTile, kStats = kRing2 + kSecond * kTile;
  static constexpr uint32_t kBars = (kStats + kSecond * kStatBytes + 15u) / 16u * 16u;
};
struct GradShared {
  uint64_t own_full, own_empty;       // the unit's own two tiles
  uint64_t full1[5], empty1[5], full2[4], empty2[4];
  uint64_t s_full[2], dp_full, p_full, ds_full, acc_full, drained;
  uint64_t met[4];
  uint32_t tmem;
  volatile int failed;
};
template <int D>
constexpr size_t kGradSmem = GradShape<D>::kBars + sizeof(GradShared);
static_assert(kGradSmem<128> <= 232448, "one CTA's shared memory (227 KB)");

__device__ __forceinline__ const float2* stats_of(const PackedParams& p, int head) {
  return p.row_stats + (size_t)head * p.stat_pitch;
}

// What all roles of both kernels begin with: barriers, tensor memory.
template <int D>
__device__ __forceinline__ uint32_t begin(GradShared& S, int warp, uint32_t second_readers) {
  using W = GradShape<D>;
  if (threadIdx.x == 0) {
    mbar_init(&S.own_full, 1);
    mbar_init(&S.own_empty, 1);
    for (int i = 0; i < W::kFirst; ++i) {
      mbar_init(&S.full1[i], 1);
      mbar_init(&S.empty1[i], 1);
    }
    for (int i = 0; i < W::kSecond; ++i) {
      mbar_init(&S.full2[i], 1);
      mbar_init(&S.empty2[i], second_readers);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&S.s_full[i], 1);
    mbar_init(&S.dp_full, 1);
    mbar_init(&S.p_full, kWorkWarps);
    mbar_init(&S.ds_full, kWorkWarps);
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.drained, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&S.met[i], 2);
    S.failed = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc::alloc(&S.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = S.tmem;
  grid_dependency_sync();
  return tmem;
}
__device__ __forceinline__ void end(const PackedParams& p, GradShared& S, uint32_t tmem, int warp) {
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, 512);
  if (threadIdx.x == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

// Tiles of 128 rows of one head, all D values.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int row, uint64_t* bar) {
#pragma unroll
  for (int d = 0; d < D; d += 64) tc::load_3d(dst + (uint32_t)d * 256u, map, d, head, row, bar);
}
// D (+)= A B^T over D inner values, both tiles as they lie
template <int D>
__device__ __forceinline__ void mma_inner(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t id = tc::idesc<Bf16>(128, 128, false, false);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    tc::mma_ss(d, tc::operand(a + (uint32_t)((k >> 2) * 16384 + (k & 3) * 32)),
               tc::operand(b + (uint32_t)((k >> 2) * 16384 + (k & 3) * 32)), id, k > 0);
}
// D (+)= A B over 128 rows of B; A in tensor memory
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool add) {
  constexpr uint32_t id = tc::idesc<Bf16>(128, D, false, true);
#pragma unroll
  for (int k = 0; k < 8; ++k) tc::mma_ts(d, a + 8 * k, tc::operand(b + k * 2048u, 16384u), id, add || k > 0);
}

// The two warps of a lane quarter have both read; bounded like every wait.
__device__ __forceinline__ bool meet(GradShared& S, int quarter, uint32_t& phase) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&S.met[quarter]);
  const bool ok = bounded_warp_wait(&S.met[quarter], phase & 1u, &S.failed);
  ++phase;
  return ok;
}

// 32 sums of this thread's row times `factor` to memory as bf16; whether all are finite
__device__ __forceinline__ bool store32(uint32_t taddr, float factor, bool zero, bool there, unsigned char* dst) {
  uint32_t y[32], w[16];
  tc::ld32(taddr, y);
  tc::wait_ld32(y);
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    // (a row that sees nothing is 0, whatever the products left there)
    const float a = zero ? 0.0f : __uint_as_float(y[2 * i]) * factor, b = zero ? 0.0f : __uint_as_float(y[2 * i + 1]) * factor;
    w[i] = Bf16::pack(a, b);
    fine &= fabsf(a) < INFINITY && fabsf(b) < INFINITY;
  }
  if (there)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  return fine;
}
__device__ __forceinline__ void clear32(bool there, unsigned char* dst) {
  if (there)
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// ---- keys and values
// A unit's queries: from i0 on, `tiles` tiles for each of the heads that share the key.
struct QuerySpan {
  int i0, tiles;
};
__device__ __forceinline__ QuerySpan query_span(const PackedUnit& u, int causal) {
  const int i0 = first_query(causal, u.m, u.n, u.i0);  // (u.m queries, u.n keys)
  return {i0, max(0, (u.m - i0 + kTileRows - 1) / kTileRows)};
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const PackedParams p,
               const PackedList list, uint8_t* flags) {
  using W = GradShape<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t base = smem_addr(raw);
  if (base & 1023u) {  // (the dynamic part begins on such a boundary)
    if (threadIdx.x == 0) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    return;
  }
  GradShared& S = *reinterpret_cast<GradShared*>(raw + W::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = begin<D>(S, warp, 1 + kWorkWarps);
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + D;
  const uint32_t k_mem = base, v_mem = base + W::kTile;
  const long long work = (long long)*list.count * p.kv_heads;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      long long it = 0;
      int units = 0;
      bool ok = true;
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.kv_heads];
        const int kh = (int)(w % p.kv_heads);
        const QuerySpan q = query_span(u, p.causal);
        if (!q.tiles) continue;
        if (units > 0 && !(ok = bounded_wait(&S.own_empty, (uint32_t)(units - 1) & 1u, &S.failed))) break;
        ++units;
        mbar_arrive_expect_tx(&S.own_full, 2 * W::kTile);
        load_tile<D>(k_mem, &map_k, kh, u.row0, &S.own_full);
        load_tile<D>(v_mem, &map_v, kh, u.row0, &S.own_full);
        for (int t = 0; t < p.G * q.tiles && ok; ++t, ++it) {
          const int head = kh * p.G + t / q.tiles, row = u.other0 + q.i0 + (t % q.tiles) * kTileRows;
          const int s1 = (int)(it % W::kFirst), s2 = (int)(it % W::kSecond);
          const uint32_t r1 = (uint32_t)(it / W::kFirst), r2 = (uint32_t)(it / W::kSecond);
          if (r1 > 0 && !(ok = bounded_wait(&S.empty1[s1], (r1 - 1) & 1u, &S.failed))) break;
          mbar_arrive_expect_tx(&S.full1[s1], W::kTile);
          load_tile<D>(base + W::kRing1 + s1 * W::kTile, &map_q, head, row, &S.full1[s1]);
          if (r2 > 0 && !(ok = bounded_wait(&S.empty2[s2], (r2 - 1) & 1u, &S.failed))) {
            (void)mbar_wait_landed(&S.full1[s1], r1 & 1u);
            break;
          }
          mbar_arrive_expect_tx(&S.full2[s2], W::kTile + kStatBytes);
          load_tile<D>(base + W::kRing2 + s2 * W::kTile, &map_do, head, row, &S.full2[s2]);
          bulk_load(raw + W::kStats + s2 * kStatBytes, stats_of(p, head) + (row & ~1), kStatBytes, &S.full2[s2]);
        }
      }
      // every copy has landed before the CTA may end
      if (units) (void)mbar_wait_landed(&S.own_full, (uint32_t)(units - 1) & 1u);
      for (long long i = it > W::kFirst ? it - W::kFirst : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst) & 1u);
      for (long long i = it > W::kSecond ? it - W::kSecond : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      long long it = 0;  // tiles so far
      int units = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (!bounded_wait(bar, phase & 1u, &S.failed)) return false;
        tc::fence_after();
        return true;
      };
      auto q_mem = [&](long long i) { return base + W::kRing1 + (uint32_t)(i % W::kFirst) * W::kTile; };
      auto do_mem = [&](long long i) { return base + W::kRing2 + (uint32_t)(i % W::kSecond) * W::kTile; };
      auto scores = [&](long long i) {
        if (!wait(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst))) return false;
        mma_inner<D>(t_s, k_mem, q_mem(i));
        tc::commit(&S.s_full[0]);
        return true;
      };
      auto products = [&](long long i) {
        if (!wait(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond))) return false;
        mma_inner<D>(t_dp, v_mem, do_mem(i));
        tc::commit(&S.dp_full);
        return true;
      };
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.kv_heads];
        const QuerySpan q = query_span(u, p.causal);
        const int n = p.G * q.tiles;
        if (!n) continue;
        if (!(ok = wait(&S.own_full, (uint32_t)units))) break;
        ++units;
        if (!(ok = scores(it)) || !(ok = products(it))) break;
        if (n == 1) tc::commit(&S.own_empty);
        for (int j = 0; j < n; ++j) {
          const long long i = it + j;
          if (!(ok = wait(&S.p_full, (uint32_t)i))) break;
          mma_rows<D>(t_dv, t_s, do_mem(i), j > 0);
          tc::commit(&S.empty2[i % W::kSecond]);
          if (j + 1 < n && !(ok = scores(i + 1))) break;
          if (!(ok = wait(&S.ds_full, (uint32_t)i))) break;
          mma_rows<D>(t_dk, t_dp, q_mem(i), j > 0);
          tc::commit(&S.empty1[i % W::kFirst]);
          if (j + 1 < n && !(ok = products(i + 1))) break;
          if (j + 2 == n) tc::commit(&S.own_empty);
        }
        if (!ok) break;
        tc::commit(&S.acc_full);
        it += n;
      }
      tc::commit(&S.drained);  // nothing is left in flight when the tensor memory is freed
      (void)mbar_wait_landed(&S.drained, 0);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float c = p.scale * kLog2e;
    long long it = 0;
    int units = 0;
    uint32_t meets = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
      const PackedUnit u = list.units[w / p.kv_heads];
      const int kh = (int)(w % p.kv_heads);
      const QuerySpan q = query_span(u, p.causal);
      const int n = p.G * q.tiles;
      const bool there = row < u.rows;
      const int mine = first_query(p.causal, u.m, u.n, u.i0 + row);          // this key's first query
      const int last = first_query(p.causal, u.m, u.n, u.i0 + kTileRows - 1);  // the unit's last key's
      for (int j = 0; j < n; ++j, ++it) {
        const int i0 = q.i0 + (j % q.tiles) * kTileRows, s2 = (int)(it % W::kSecond);
        const int first_row = u.other0 + i0;
        const bool border = i0 < last || i0 + kTileRows > u.m;
        const int lo = mine - i0 - half * 64, hi = u.m - i0 - half * 64;  // of the half's columns
        const float2* st = reinterpret_cast<const float2*>(raw + W::kStats + s2 * kStatBytes) + (first_row & 1) + half * 64;
        if (!(ok = bounded_warp_wait(&S.full2[s2], (uint32_t)(it / W::kSecond) & 1u, &S.failed))) break;
        if (!(ok = bounded_warp_wait(&S.s_full[0], (uint32_t)it & 1u, &S.failed))) break;
        tc::fence_after();
        uint32_t x[64];
        tc::ld32(t_s + lanes + half * 64, x);
        tc::ld32(t_s + lanes + half * 64 + 32, x + 32);
        tc::wait_ld32(x);
        tc::wait_ld32(x + 32);
        if (!(ok = meet(S, quarter, meets))) break;
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = ex2_approx(fmaf(__uint_as_float(x[k + e]), c, -st[k + e].x));
            const float b = ex2_approx(fmaf(__uint_as_float(x[k + e + 1]), c, -st[k + e + 1].x));
            x[k + e] = __float_as_uint(a);
            x[k + e + 1] = __float_as_uint(b);
          }
          if (border) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k + e < lo || k + e >= hi) x[k + e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = Bf16::pack(__uint_as_float(x[k + 2 * e]), __uint_as_float(x[k + 2 * e + 1]));
          tc::st16(t_s + lanes + half * 32 + k / 2, pk);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full);

        if (!(ok = bounded_warp_wait(&S.dp_full, (uint32_t)it & 1u, &S.failed))) break;
        tc::fence_after();
        uint32_t y[64];
        tc::ld32(t_dp + lanes + half * 64, y);
        tc::ld32(t_dp + lanes + half * 64 + 32, y + 32);
        tc::wait_ld32(y);
        tc::wait_ld32(y + 32);
        if (!(ok = meet(S, quarter, meets))) break;
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            y[k + e] = __float_as_uint(__uint_as_float(x[k + e]) * (__uint_as_float(y[k + e]) - st[k + e].y));
          if (border) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k + e < lo || k + e >= hi) y[k + e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = Bf16::pack(__uint_as_float(y[k + 2 * e]), __uint_as_float(y[k + 2 * e + 1]));
          tc::st16(t_dp + lanes + half * 32 + k / 2, pk);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.ds_full);
          mbar_arrive(&S.empty2[s2]);  // the statistics are read
        }
      }
      if (!ok) break;

      // ---- the keys' ends: half of the columns each
      unsigned char* dk = p.dk.p + 2 * ((long long)(u.row0 + row) * p.dk.ts + (long long)kh * p.dk.hs);
      unsigned char* dv = p.dv.p + 2 * ((long long)(u.row0 + row) * p.dv.ts + (long long)kh * p.dv.hs);
      bool fine = true;
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.acc_full, (uint32_t)units & 1u, &S.failed))) break;
        ++units;
        tc::fence_after();
      }
#pragma unroll 1
      for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
        if (n > 0) {
          fine &= store32(t_dv + lanes + d, 1.0f, false, there, dv + 2 * d);
          fine &= store32(t_dk + lanes + d, p.scale, false, there, dk + 2 * d);
        } else {
          clear32(there, dv + 2 * d);
          clear32(there, dk + 2 * d);
        }
      }
      const bool odd = __any_sync(0xffffffffu, there && !fine);
      if (lane == 0) flags[w * kGradFlags + 2 * quarter + half] = odd;
      tc::fence_before();
    }
  }
  end(p, S, tmem, warp);
}

// ---- queries
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const PackedParams p,
              const PackedList list, uint8_t* flags) {
  using W = GradShape<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t base = smem_addr(raw);
  if (base & 1023u) {
    if (threadIdx.x == 0) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    return;
  }
  GradShared& S = *reinterpret_cast<GradShared*>(raw + W::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = begin<D>(S, warp, 1);
  const uint32_t t_s = tmem, t_dp = tmem + 256, t_dq = tmem + 384;
  const uint32_t q_mem = base, do_mem = base + W::kTile;
  const long long work = (long long)*list.count * p.q_heads;
  auto tiles_of = [&](const PackedUnit& u) {
    return (seen_keys(p.causal, u.n, u.m, u.i0 + u.rows - 1) + kTileRows - 1) / kTileRows;
  };

  if (warp == kLoadWarp) {
    if (lane == 0) {
      long long it = 0;
      int units = 0;
      bool ok = true;
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.q_heads];
        const int head = (int)(w % p.q_heads), kh = head / p.G, n = tiles_of(u);
        if (!n) continue;
        if (units > 0 && !(ok = bounded_wait(&S.own_empty, (uint32_t)(units - 1) & 1u, &S.failed))) break;
        ++units;
        mbar_arrive_expect_tx(&S.own_full, 2 * W::kTile);
        load_tile<D>(q_mem, &map_q, head, u.row0, &S.own_full);
        load_tile<D>(do_mem, &map_do, head, u.row0, &S.own_full);
        for (int t = 0; t < n && ok; ++t, ++it) {
          const int row = u.other0 + t * kTileRows;
          const int s1 = (int)(it % W::kFirst), s2 = (int)(it % W::kSecond);
          const uint32_t r1 = (uint32_t)(it / W::kFirst), r2 = (uint32_t)(it / W::kSecond);
          if (r1 > 0 && !(ok = bounded_wait(&S.empty1[s1], (r1 - 1) & 1u, &S.failed))) break;
          mbar_arrive_expect_tx(&S.full1[s1], W::kTile);
          load_tile<D>(base + W::kRing1 + s1 * W::kTile, &map_k, kh, row, &S.full1[s1]);
          if (r2 > 0 && !(ok = bounded_wait(&S.empty2[s2], (r2 - 1) & 1u, &S.failed))) {
            (void)mbar_wait_landed(&S.full1[s1], r1 & 1u);
            break;
          }
          mbar_arrive_expect_tx(&S.full2[s2], W::kTile);
          load_tile<D>(base + W::kRing2 + s2 * W::kTile, &map_v, kh, row, &S.full2[s2]);
        }
      }
      if (units) (void)mbar_wait_landed(&S.own_full, (uint32_t)(units - 1) & 1u);
      for (long long i = it > W::kFirst ? it - W::kFirst : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst) & 1u);
      for (long long i = it > W::kSecond ? it - W::kSecond : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      long long it = 0;
      int units = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (!bounded_wait(bar, phase & 1u, &S.failed)) return false;
        tc::fence_after();
        return true;
      };
      auto k_mem = [&](long long i) { return base + W::kRing1 + (uint32_t)(i % W::kFirst) * W::kTile; };
      // scores and products of the ring's tile i, which takes buffer i % 2
      auto scores = [&](long long i) {
        if (!wait(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst))) return false;
        mma_inner<D>(t_s + (uint32_t)(i & 1) * 128u, q_mem, k_mem(i));
        tc::commit(&S.s_full[i & 1]);
        return true;
      };
      auto products = [&](long long i) {
        if (!wait(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond))) return false;
        mma_inner<D>(t_dp, do_mem, base + W::kRing2 + (uint32_t)(i % W::kSecond) * W::kTile);
        tc::commit(&S.dp_full);
        tc::commit(&S.empty2[i % W::kSecond]);
        return true;
      };
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.q_heads];
        const int n = tiles_of(u);
        if (!n) continue;
        if (!(ok = wait(&S.own_full, (uint32_t)units))) break;
        ++units;
        if (!(ok = scores(it)) || !(ok = products(it))) break;
        if (n == 1) tc::commit(&S.own_empty);
        int issued = 1;  // scores
        if (n > 1) {
          if (!(ok = scores(it + 1))) break;
          issued = 2;
        }
        for (int j = 0; j < n; ++j) {
          const long long i = it + j;
          if (!(ok = wait(&S.ds_full, (uint32_t)i))) break;
          if (j + 1 < n) {
            if (issued == j + 1) {  // these scores could not go ahead of the product before
              if (!(ok = scores(i + 1))) break;
              ++issued;
            }
            if (!(ok = products(i + 1))) break;
            if (j + 2 == n) tc::commit(&S.own_empty);
          }
          mma_rows<D>(t_dq, t_s + (uint32_t)(i & 1) * 128u, k_mem(i), j > 0);
          tc::commit(&S.empty1[i % W::kFirst]);
          if (j + 2 < n && mbar_test_wait(&S.full1[(i + 2) % W::kFirst], (uint32_t)((i + 2) / W::kFirst) & 1u)) {
            if (!(ok = scores(i + 2))) break;
            issued = j + 3;
          }
        }
        if (!ok) break;
        tc::commit(&S.acc_full);
        it += n;
      }
      tc::commit(&S.drained);
      (void)mbar_wait_landed(&S.drained, 0);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float c = p.scale * kLog2e;
    long long it = 0;
    int units = 0;
    uint32_t meets = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
      const PackedUnit u = list.units[w / p.q_heads];
      const int head = (int)(w % p.q_heads), n = tiles_of(u);
      const bool there = row < u.rows;
      const int vis = there ? seen_keys(p.causal, u.n, u.m, u.i0 + row) : 0, vis0 = seen_keys(p.causal, u.n, u.m, u.i0);
      const float2 st = there ? stats_of(p, head)[u.row0 + row] : make_float2(INFINITY, 0.0f);
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t buf = t_s + (uint32_t)(it & 1) * 128u + lanes;
        const int left = (j + 1) * kTileRows > vis0 ? vis - j * kTileRows - half * 64 : 64;
        if (!(ok = bounded_warp_wait(&S.s_full[it & 1], (uint32_t)(it >> 1) & 1u, &S.failed))) break;
        tc::fence_after();
        uint32_t x[64];
        tc::ld32(buf + half * 64, x);
        tc::ld32(buf + half * 64 + 32, x + 32);
        tc::wait_ld32(x);
        tc::wait_ld32(x + 32);
#pragma unroll
        for (int e = 0; e < 64; ++e) x[e] = __float_as_uint(ex2_approx(fmaf(__uint_as_float(x[e]), c, -st.x)));
        if (!(ok = bounded_warp_wait(&S.dp_full, (uint32_t)it & 1u, &S.failed))) break;
        tc::fence_after();
        if (!(ok = meet(S, quarter, meets))) break;
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
          uint32_t y[32], pk[16];
          tc::ld32(t_dp + lanes + half * 64 + k, y);
          tc::wait_ld32(y);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            y[e] = __float_as_uint(__uint_as_float(x[k + e]) * (__uint_as_float(y[e]) - st.y));
          if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (k + e >= left) y[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = Bf16::pack(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1]));
          tc::st16(buf + half * 32 + k / 2, pk);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.ds_full);
      }
      if (!ok) break;

      unsigned char* dq = p.dq.p + 2 * ((long long)(u.row0 + row) * p.dq.ts + (long long)head * p.dq.hs);
      bool fine = true;
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.acc_full, (uint32_t)units & 1u, &S.failed))) break;
        ++units;
        tc::fence_after();
      }
#pragma unroll 1
      for (int d = half * (D / 2); d < (half + 1) * (D / 2); d += 32) {
        if (n > 0)
          fine &= store32(t_dq + lanes + d, p.scale, vis <= 0, there, dq + 2 * d);
        else
          clear32(there, dq + 2 * d);
      }
      const bool odd = __any_sync(0xffffffffu, there && !fine);
      if (lane == 0) flags[w * kGradFlags + 2 * quarter + half] = odd;
      tc::fence_before();
    }
  }
  end(p, S, tmem, warp);
}

template <class K>
int launch(K kernel, const PackedParams& p, int D, size_t smem, long long most, const PackedList& list, uint8_t* flags, int sms,
           bool* ready, void* stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return (int)e;
    ready[dev] = true;
  }
  CUtensorMap q, k, v, d_o;
  // (an array without rows is never loaded)
  const HeadRows &some = p.q_tokens ? p.q : p.k;
  const int tokens = p.q_tokens ? p.q_tokens : p.kv_tokens, heads = p.q_tokens ? p.q_heads : p.kv_heads;
  if (!map_heads(&q, true, some, tokens, heads, D, kTileRows)) return (int)cudaErrorInvalidValue;
  k = v = d_o = q;
  if ((p.q_tokens && !map_heads(&d_o, true, p.d_o, p.q_tokens, p.q_heads, D, kTileRows)) ||
      (p.kv_tokens && (!map_heads(&k, true, p.k, p.kv_tokens, p.kv_heads, D, kTileRows) ||
                       !map_heads(&v, true, p.v, p.kv_tokens, p.kv_heads, D, kTileRows))))
    return (int)cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  return (int)cudaLaunchKernelEx(&cfg, kernel, q, k, v, d_o, p, list, flags);
}
template <int D>
int launch_dq(const PackedParams& p, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  static bool ready[64] = {};
  return launch(dq_kernel<D>, p, D, kGradSmem<D>, (long long)most_units(p.q_tokens, p.B, kGradRows) * p.q_heads, list, flags,
                sms, ready, stream);
}
template <int D>
int launch_dkv(const PackedParams& p, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  static bool ready[64] = {};
  return launch(dkv_kernel<D>, p, D, kGradSmem<D>, (long long)most_units(p.kv_tokens, p.B, kGradRows) * p.kv_heads, list,
                flags, sms, ready, stream);
}

}  // namespace

int launch_dq_tc(const PackedParams& p, int d, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  return d == 64 ? launch_dq<64>(p, list, flags, sms, stream) : launch_dq<128>(p, list, flags, sms, stream);
}
int launch_dkv_tc(const PackedParams& p, int d, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  return d == 64 ? launch_dkv<64>(p, list, flags, sms, stream) : launch_dkv<128>(p, list, flags, sms, stream);
}

}  // namespace dflash
