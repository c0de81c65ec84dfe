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
// dS(j) is made, dK(j), dP(j + 1) while P(j + 1) is. 16 warps make P and dS, four for each
// quarter of the lanes, 32 of the columns each. Their results take the place of scores:
// a warp's 32 columns, packed, lie in the first 16 of the 32 that it has read itself, so no
// warp writes over what another still reads (mma_rows steps over the parts so). A row's
// lse and delta, made ahead of the kernels, lie by head, all of lse and then all of delta; for the
// keys' kernel 128 of lse come with each tile of Q and 128 of delta with each tile of dO.
// Masks select P = 0 in tiles at a border only (dS is then 0 times something, which is 0 or
// mended with the rest). 8 x 1024 queries over 8 x 4096 keys, 32 heads of 128 over 8: keys
// 654 us (1.68 PFLOP/s), queries 465 us (1.77 PFLOP/s); over 1024 keys, 187 and 139 us, the
// units' beginnings and ends weigh more. Rows with a result that is not
// finite are flagged (see dflash_packed.cuh). Every wait is bounded; a CTA that gives up
// raises DFLASH_STATUS_TIMEOUT.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_packed_mma.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 576, kMmaWarp = 16, kLoadWarp = 17, kWorkWarps = 16;
constexpr int kParts = kWorkWarps / 4;   // warps that share rows
constexpr int kCols = 128 / kParts;      // columns of a tile for each
constexpr int kTileRows = 128;
constexpr uint32_t kStatBytes = 512;  // of a tile of queries: lse comes with Q, delta with dO

template <int D>
struct GradShape {
  static constexpr uint32_t kTile = 128u * D * 2u;
  // keys: K, V; tiles of Q and of dO. queries: Q, dO; tiles of K and of V.
  static constexpr int kFirst = D == 128 ? 3 : 5, kSecond = D == 128 ? 2 : 4;
  static constexpr uint32_t kRing1 = 2 * kTile, kRing2 = kRing1 + kFirst * kTile, kLse = kRing2 + kSecond * kTile;
  static constexpr uint32_t kDelta = kLse + kFirst * kStatBytes, kBars = kDelta + kSecond * kStatBytes;
};
struct GradShared {
  uint64_t own_full, own_empty;       // the unit's own two tiles
  uint64_t full1[5], empty1[5], full2[4], empty2[4];
  uint64_t s_full[2], dp_full, p_full, ds_full, acc_full, drained;
  uint32_t tmem;
  volatile int failed;
};
template <int D>
constexpr size_t kGradSmem = GradShape<D>::kBars + sizeof(GradShared);
static_assert(kGradSmem<128> <= 232448, "one CTA's shared memory (227 KB)");

// A head's statistics, their signs reversed: lse, then (stat_pitch further on) delta
__device__ __forceinline__ const float* stats_of(const PackedParams& p, int head) {
  return p.row_stats + (size_t)head * 2 * p.stat_pitch;
}

// What all roles of both kernels begin with: barriers, tensor memory (all of it, so it
// begins at 0).
template <int D>
__device__ __forceinline__ void begin(GradShared& S, int warp, uint32_t second_readers, bool wait) {
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
    S.failed = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc::alloc(&S.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (wait)
    grid_dependency_sync();
  else
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void end(const PackedParams& p, GradShared& S, int warp) {
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(0, 512);
  if (threadIdx.x == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

// Tiles of 128 rows of one head, all D values.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int row, uint64_t* bar) {
#pragma unroll
  for (int d = 0; d < D; d += 64) tc::load_3d(dst + (uint32_t)d * 256u, map, d, head, row, bar);
}
// D (+)= A B^T over D inner values, both tiles as they lie (addresses count in 16 bytes)
template <int D>
__device__ __forceinline__ void mma_inner(uint32_t d, uint32_t a, uint32_t b, uint32_t lead) {
  constexpr uint32_t id = tc::idesc<Bf16>(128, 128, false, false);
  const uint64_t ad = tc::operand(a), bd = tc::operand(b);
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    tc::mma_ss(d, ad + (uint64_t)((k >> 2) * 1024 + (k & 3) * 2), bd + (uint64_t)((k >> 2) * 1024 + (k & 3) * 2), id, k > 0,
               lead);
}
// D (+)= A B over 128 rows of B; A in tensor memory, each part of its columns in the first
// half of that part of the scores, which the warp that wrote it had read
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool add, uint32_t lead) {
  constexpr uint32_t id = tc::idesc<Bf16>(128, D, false, true);
  const uint64_t bd = tc::operand(b, 16384u);
#pragma unroll
  for (int k = 0; k < 8; ++k) tc::mma_ts(d, a + (k >> 1) * 32 + (k & 1) * 8, bd + (uint64_t)(k * 128), id, add || k > 0, lead);
}
// A tile of a ring of kSlots: its place, and the parity of its round
template <int kSlots>
struct RingAt {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

__device__ __forceinline__ float2 pair(const uint32_t* x, int e) {
  return make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
}

// A part of a warp's 32 rows of sums times `factor` to memory as bf16 (rows where `zero`
// holds: 0, whatever the products left there); whether this lane's are finite
template <int D>
__device__ __forceinline__ bool store_part(uint32_t taddr, float factor, bool zero, unsigned char* dst, long long stride,
                                           int rows, int lane) {
  constexpr int kMine = D / kParts, kPieces = kMine / 8;
  uint32_t y[kMine], w[4 * kPieces];
  if constexpr (kMine == 32) {
    tc::ld32(taddr, y);
    tc::wait_ld32(y);
  } else {
    tc::ld16(taddr, y);
    tc::wait_ld16(y);
  }
  float2 probe = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kMine / 2; ++i) {
    float2 f = mul2(make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), make_float2(factor, factor));
    if (zero) f = make_float2(0.0f, 0.0f);
    w[i] = Bf16::pack(f.x, f.y);
    probe = fma2(f, make_float2(0.0f, 0.0f), probe);
  }
  store_rows<kPieces>(w, dst, stride, rows, lane);
  return probe.x + probe.y == 0.0f;
}
template <int D>
__device__ __forceinline__ void clear_part(unsigned char* dst, long long stride, int rows, int lane) {
  constexpr int kPieces = D / kParts / 8;
  uint32_t w[4 * kPieces] = {};
  store_rows<kPieces>(w, dst, stride, rows, lane);
}

// ---- keys and values
// A unit's queries: from i0 on, `tiles` tiles for each of the heads that share the
// key. The first row is a multiple of 4, so that four statistics are one load; up to 3
// queries in front of the first (or rows of the sequence before) count as masked.
struct QuerySpan {
  int i0, tiles;
};
__device__ __forceinline__ QuerySpan query_span(const PackedUnit& u, int causal) {
  const int i0 = first_query(causal, u.m, u.n, u.i0);  // (u.m queries, u.n keys)
  if (i0 >= u.m) return {0, 0};
  const int at = i0 - ((u.other0 + i0) & 3);
  return {at, (u.m - at + kTileRows - 1) / kTileRows};
}

// behind_dq: the kernel ahead in the stream is the queries', whose CTAs have waited for
// what this one reads. So its CTAs begin as SMs become free, and wait only at their ends,
// for the kernels behind.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do, const PackedParams p,
               const PackedList list, uint8_t* flags, const bool behind_dq) {
  using W = GradShape<D>;
  extern __shared__ __align__(1024) unsigned char raw[];
  const uint32_t base = smem_addr(raw);
  if (base & 1023u) {  // (the dynamic part begins on such a boundary)
    if (threadIdx.x == 0) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    return;
  }
  GradShared& S = *reinterpret_cast<GradShared*>(raw + W::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  begin<D>(S, warp, 1 + kWorkWarps, !behind_dq);
  constexpr uint32_t t_s = 0, t_dp = 128, t_dv = 256, t_dk = 256 + D;
  const uint32_t k_mem = base, v_mem = base + W::kTile;
  const int work = *list.count * p.kv_heads;  // (below 2^28)

  if (warp == kLoadWarp) {
    if (lane == 0) {
      RingAt<W::kFirst> r1;
      RingAt<W::kSecond> r2;
      int units = 0, it = 0;
      bool ok = true;
      for (int round = 0; ok; ++round) {
        const int w = unit_of(round);
        if (w >= work) break;
        const PackedUnit u = list.units[w / p.kv_heads];
        const int kh = w % p.kv_heads;
        const QuerySpan q = query_span(u, p.causal);
        if (!q.tiles) continue;
        if (units > 0 && !(ok = bounded_wait(&S.own_empty, (uint32_t)(units - 1) & 1u, &S.failed))) break;
        ++units;
        mbar_arrive_expect_tx(&S.own_full, 2 * W::kTile);
        load_tile<D>(k_mem, &map_k, kh, u.row0, &S.own_full);
        load_tile<D>(v_mem, &map_v, kh, u.row0, &S.own_full);
        for (int head = kh * p.G; head < (kh + 1) * p.G && ok; ++head)
          for (int t = 0; t < q.tiles && ok; ++t, ++it) {
            const int row = u.other0 + q.i0 + t * kTileRows;
            const float* st = stats_of(p, head) + row;
            if (it >= W::kFirst && !(ok = bounded_wait(&S.empty1[r1.slot], r1.phase ^ 1u, &S.failed))) break;
            mbar_arrive_expect_tx(&S.full1[r1.slot], W::kTile + kStatBytes);
            load_tile<D>(base + W::kRing1 + r1.slot * W::kTile, &map_q, head, row, &S.full1[r1.slot]);
            bulk_load(raw + W::kLse + r1.slot * kStatBytes, st, kStatBytes, &S.full1[r1.slot]);
            if (it >= W::kSecond && !(ok = bounded_wait(&S.empty2[r2.slot], r2.phase ^ 1u, &S.failed))) {
              (void)mbar_wait_landed(&S.full1[r1.slot], r1.phase);
              break;
            }
            mbar_arrive_expect_tx(&S.full2[r2.slot], W::kTile + kStatBytes);
            load_tile<D>(base + W::kRing2 + r2.slot * W::kTile, &map_do, head, row, &S.full2[r2.slot]);
            bulk_load(raw + W::kDelta + r2.slot * kStatBytes, st + p.stat_pitch, kStatBytes, &S.full2[r2.slot]);
            r1.advance();
            r2.advance();
          }
      }
      // every copy has landed before the CTA may end
      if (units) (void)mbar_wait_landed(&S.own_full, (uint32_t)(units - 1) & 1u);
      for (int i = it > W::kFirst ? it - W::kFirst : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst) & 1u);
      for (int i = it > W::kSecond ? it - W::kSecond : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t lead = tc::elect();
    RingAt<W::kFirst> q1, q2;     // the tiles of Q of the next scores, and of the next dK
    RingAt<W::kSecond> d1, d2;    // the tiles of dO of the next products with V, and of the next dV
    uint32_t units = 0, it = 0;   // units and tiles so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool done = bounded_warp_wait(bar, parity & 1u, &S.failed);
      tc::fence_after();
      return done;
    };
    auto q_mem = [&](int slot) { return base + W::kRing1 + (uint32_t)slot * W::kTile; };
    auto do_mem = [&](int slot) { return base + W::kRing2 + (uint32_t)slot * W::kTile; };
    auto scores = [&] {
      mma_inner<D>(t_s, k_mem, q_mem(q1.slot), lead);
      tc::commit(&S.s_full[0], lead);
      q1.advance();
    };
    auto products = [&] {
      mma_inner<D>(t_dp, v_mem, do_mem(d1.slot), lead);
      tc::commit(&S.dp_full, lead);
      d1.advance();
    };
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.kv_heads];
      const int n = tc::uniform(p.G * query_span(u, p.causal).tiles);
      if (!n) continue;
      if (!(ok = wait(&S.own_full, units)) || !(ok = wait(&S.full1[q1.slot], q1.phase))) break;
      ++units;
      scores();
      if (!(ok = wait(&S.full2[d1.slot], d1.phase))) break;
      products();
      if (n == 1) tc::commit(&S.own_empty, lead);
      for (int j = 0; j < n; ++j, ++it) {
        // (operands are waited for ahead of what the threads make)
        const bool more = j + 1 < n;
        if (more && !(ok = wait(&S.full1[q1.slot], q1.phase))) break;
        if (!(ok = wait(&S.p_full, it))) break;
        mma_rows<D>(t_dv, t_s, do_mem(d2.slot), j > 0, lead);
        tc::commit(&S.empty2[d2.slot], lead);
        d2.advance();
        if (more) scores();
        if (more && !(ok = wait(&S.full2[d1.slot], d1.phase))) break;
        if (!(ok = wait(&S.ds_full, it))) break;
        mma_rows<D>(t_dk, t_dp, q_mem(q2.slot), j > 0, lead);
        tc::commit(&S.empty1[q2.slot], lead);
        q2.advance();
        if (more) products();
        if (j + 2 == n) tc::commit(&S.own_empty, lead);
      }
      if (!ok) break;
      tc::commit(&S.acc_full, lead);
    }
    tc::commit(&S.drained, lead);  // nothing is left in flight when the tensor memory is freed
    (void)mbar_wait_landed(&S.drained, 0);
    __syncwarp();
  } else {
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
    const uint32_t mine = ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kCols);
    const float c = p.scale * kLog2e;
    uint32_t it = 0, units = 0;  // tiles and units so far
    RingAt<W::kFirst> r1;
    RingAt<W::kSecond> r2;
    bool ok = true;
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.kv_heads];
      const int kh = w % p.kv_heads;
      const QuerySpan q = query_span(u, p.causal);
      const int n = p.G * q.tiles;
      const bool there = row < u.rows;
      const int first = first_query(p.causal, u.m, u.n, u.i0 + row);          // that sees this key
      const int last = first_query(p.causal, u.m, u.n, u.i0 + kTileRows - 1);  // ... the unit's last
      int i0 = q.i0, t = 0;  // this tile's first query and its number
      for (int j = 0; j < n; ++j, ++it) {
        const bool from_front = i0 < max(last, 0), at_end = i0 + kTileRows > u.m;  // some keys are not seen by all
        const int lo = first - i0 - part * kCols, hi = u.m - i0 - part * kCols;    // of this part's columns
        const float4* lse4 = reinterpret_cast<const float4*>(raw + W::kLse + r1.slot * kStatBytes) + part * (kCols / 4);
        const float4* delta4 = reinterpret_cast<const float4*>(raw + W::kDelta + r2.slot * kStatBytes) + part * (kCols / 4);
        i0 += kTileRows;
        if (++t == q.tiles) {
          t = 0;
          i0 = q.i0;
        }
        if (!(ok = bounded_warp_wait2(&S.s_full[0], it & 1u, &S.full1[r1.slot], r1.phase, &S.failed))) break;
        tc::fence_after();
        uint32_t x[kCols], pk[kCols / 2];
        tc::ld32(t_s + mine, x);
        tc::wait_ld32(x);
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          const float4 s4 = lse4[e / 4];
          const float2 a = fma2(pair(x, e), make_float2(c, c), make_float2(s4.x, s4.y));
          const float2 b = fma2(pair(x, e + 2), make_float2(c, c), make_float2(s4.z, s4.w));
          x[e] = __float_as_uint(ex2_approx(a.x));
          x[e + 1] = __float_as_uint(ex2_approx(a.y));
          x[e + 2] = __float_as_uint(ex2_approx(b.x));
          x[e + 3] = __float_as_uint(ex2_approx(b.y));
        }
        if (from_front) {
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e < lo) x[e] = 0u;
        }
        if (at_end) {
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= hi) x[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < kCols / 2; ++e) pk[e] = Bf16::pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
        tc::st16(t_s + mine, pk);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full);

        if (!(ok = bounded_warp_wait2(&S.dp_full, it & 1u, &S.full2[r2.slot], r2.phase, &S.failed))) break;
        tc::fence_after();
        uint32_t y[kCols];
        tc::ld32(t_dp + mine, y);
        tc::wait_ld32(y);
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          const float4 s4 = delta4[e / 4];
          const float2 a = mul2(pair(x, e), add2(pair(y, e), make_float2(s4.x, s4.y)));
          const float2 b = mul2(pair(x, e + 2), add2(pair(y, e + 2), make_float2(s4.z, s4.w)));
          pk[e / 2] = Bf16::pack(a.x, a.y);
          pk[e / 2 + 1] = Bf16::pack(b.x, b.y);
        }
        tc::st16(t_dp + mine, pk);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.ds_full);
          mbar_arrive(&S.empty2[r2.slot]);  // delta is read
        }
        r1.advance();
        r2.advance();
      }
      if (!ok) break;

      // ---- the keys' ends: a part of the columns each
      const int rows = u.rows - quarter * 32;  // of this warp's 32
      const long long tok0 = u.row0 + quarter * 32;
      constexpr int kMine = D / kParts;
      unsigned char* dk = p.dk.p + 2 * (tok0 * p.dk.ts + (long long)kh * p.dk.hs + part * kMine);
      unsigned char* dv = p.dv.p + 2 * (tok0 * p.dv.ts + (long long)kh * p.dv.hs + part * kMine);
      const uint32_t sums = ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kMine);
      bool fine = true;
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.acc_full, units & 1u, &S.failed))) break;
        ++units;
        tc::fence_after();
        fine &= store_part<D>(t_dv + sums, 1.0f, false, dv, 2 * p.dv.ts, rows, lane);
        fine &= store_part<D>(t_dk + sums, p.scale, false, dk, 2 * p.dk.ts, rows, lane);
      } else {
        clear_part<D>(dv, 2 * p.dv.ts, rows, lane);
        clear_part<D>(dk, 2 * p.dk.ts, rows, lane);
      }
      const bool odd = __any_sync(0xffffffffu, there && !fine);
      if (lane == 0) flags[(size_t)w * kGradFlags + kParts * quarter + part] = odd;
      tc::fence_before();
    }
  }
  end(p, S, warp);
  if (behind_dq) asm volatile("griddepcontrol.wait;" ::: "memory");
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
  begin<D>(S, warp, 1, true);
  constexpr uint32_t t_s = 0, t_dp = 256, t_dq = 384;
  const uint32_t q_mem = base, do_mem = base + W::kTile;
  const int work = *list.count * p.q_heads;  // (below 2^28)
  auto tiles_of = [&](const PackedUnit& u) {
    return (seen_keys(p.causal, u.n, u.m, u.i0 + u.rows - 1) + kTileRows - 1) / kTileRows;
  };

  if (warp == kLoadWarp) {
    if (lane == 0) {
      RingAt<W::kFirst> r1;
      RingAt<W::kSecond> r2;
      int units = 0, it = 0;
      bool ok = true;
      for (int round = 0; ok; ++round) {
        const int w = unit_of(round);
        if (w >= work) break;
        const PackedUnit u = list.units[w / p.q_heads];
        const int head = w % p.q_heads, kh = head / p.G, n = tiles_of(u);
        if (!n) continue;
        if (units > 0 && !(ok = bounded_wait(&S.own_empty, (uint32_t)(units - 1) & 1u, &S.failed))) break;
        ++units;
        mbar_arrive_expect_tx(&S.own_full, 2 * W::kTile);
        load_tile<D>(q_mem, &map_q, head, u.row0, &S.own_full);
        load_tile<D>(do_mem, &map_do, head, u.row0, &S.own_full);
        for (int t = 0; t < n && ok; ++t, ++it) {
          const int row = u.other0 + t * kTileRows;
          if (it >= W::kFirst && !(ok = bounded_wait(&S.empty1[r1.slot], r1.phase ^ 1u, &S.failed))) break;
          mbar_arrive_expect_tx(&S.full1[r1.slot], W::kTile);
          load_tile<D>(base + W::kRing1 + r1.slot * W::kTile, &map_k, kh, row, &S.full1[r1.slot]);
          if (it >= W::kSecond && !(ok = bounded_wait(&S.empty2[r2.slot], r2.phase ^ 1u, &S.failed))) {
            (void)mbar_wait_landed(&S.full1[r1.slot], r1.phase);
            break;
          }
          mbar_arrive_expect_tx(&S.full2[r2.slot], W::kTile);
          load_tile<D>(base + W::kRing2 + r2.slot * W::kTile, &map_v, kh, row, &S.full2[r2.slot]);
          r1.advance();
          r2.advance();
        }
      }
      if (units) (void)mbar_wait_landed(&S.own_full, (uint32_t)(units - 1) & 1u);
      for (int i = it > W::kFirst ? it - W::kFirst : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full1[i % W::kFirst], (uint32_t)(i / W::kFirst) & 1u);
      for (int i = it > W::kSecond ? it - W::kSecond : 0; i < it; ++i)
        (void)mbar_wait_landed(&S.full2[i % W::kSecond], (uint32_t)(i / W::kSecond) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t lead = tc::elect();
    RingAt<W::kFirst> k1, k2;   // the tiles of K of the next scores, and of the next dQ
    RingAt<W::kSecond> v1;
    uint32_t units = 0, it = 0, ahead = 0;  // units, tiles and tiles of scores so far (scores take buffer ahead % 2)
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool done = bounded_warp_wait(bar, parity & 1u, &S.failed);
      tc::fence_after();
      return done;
    };
    auto k_mem = [&](int slot) { return base + W::kRing1 + (uint32_t)slot * W::kTile; };
    auto scores = [&] {
      mma_inner<D>(t_s + (ahead & 1u) * 128u, q_mem, k_mem(k1.slot), lead);
      tc::commit(&S.s_full[ahead & 1u], lead);
      k1.advance();
      ++ahead;
    };
    auto products = [&] {
      mma_inner<D>(t_dp, do_mem, base + W::kRing2 + (uint32_t)v1.slot * W::kTile, lead);
      tc::commit(&S.dp_full, lead);
      tc::commit(&S.empty2[v1.slot], lead);
      v1.advance();
    };
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.q_heads];
      const int n = tc::uniform(tiles_of(u));
      if (!n) continue;
      if (!(ok = wait(&S.own_full, units)) || !(ok = wait(&S.full1[k1.slot], k1.phase))) break;
      ++units;
      scores();
      if (!(ok = wait(&S.full2[v1.slot], v1.phase))) break;
      products();
      if (n == 1) tc::commit(&S.own_empty, lead);
      for (int j = 0; j < n; ++j, ++it) {
        if (j + 1 < n) {
          // (operands are waited for ahead of what the threads make)
          if (ahead == it + 1) {
            if (!(ok = wait(&S.full1[k1.slot], k1.phase))) break;
            scores();
          }
          if (!(ok = wait(&S.full2[v1.slot], v1.phase))) break;
        }
        if (!(ok = wait(&S.ds_full, it))) break;
        if (j + 1 < n) products();
        if (j + 2 == n) tc::commit(&S.own_empty, lead);
        mma_rows<D>(t_dq, t_s + (it & 1u) * 128u, k_mem(k2.slot), j > 0, lead);
        tc::commit(&S.empty1[k2.slot], lead);
        k2.advance();
        if (j + 2 < n && __all_sync(0xffffffffu, mbar_test_wait(&S.full1[k1.slot], k1.phase))) {
          tc::fence_after();
          scores();
        }
      }
      if (!ok) break;
      tc::commit(&S.acc_full, lead);
    }
    tc::commit(&S.drained, lead);
    (void)mbar_wait_landed(&S.drained, 0);
    __syncwarp();
  } else {
    const int quarter = warp & 3, part = warp >> 2, row = quarter * 32 + lane;
    const uint32_t mine = ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kCols);
    const float c = p.scale * kLog2e;
    uint32_t it = 0, units = 0;  // tiles and units so far
    bool ok = true;
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.q_heads];
      const int head = w % p.q_heads, n = tiles_of(u);
      const bool there = row < u.rows;
      const int vis = there ? seen_keys(p.causal, u.n, u.m, u.i0 + row) : 0, vis0 = seen_keys(p.causal, u.n, u.m, u.i0);
      const float lse = there ? stats_of(p, head)[u.row0 + row] : -INFINITY;
      const float delta = there ? stats_of(p, head)[p.stat_pitch + u.row0 + row] : 0.0f;
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t buf = t_s + (it & 1u) * 128u + mine;
        if (!(ok = bounded_warp_wait(&S.s_full[it & 1u], (it >> 1) & 1u, &S.failed))) break;
        tc::fence_after();
        uint32_t x[kCols], y[kCols], pk[kCols / 2];
        tc::ld32(buf, x);
        tc::wait_ld32(x);
#pragma unroll
        for (int e = 0; e < kCols; e += 2) {
          const float2 a = fma2(pair(x, e), make_float2(c, c), make_float2(lse, lse));
          x[e] = __float_as_uint(ex2_approx(a.x));
          x[e + 1] = __float_as_uint(ex2_approx(a.y));
        }
        if ((j + 1) * kTileRows > vis0) {  // some row does not see all of the tile
          const int left = vis - j * kTileRows - part * kCols;
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= left) x[e] = 0u;
        }
        if (!(ok = bounded_warp_wait(&S.dp_full, it & 1u, &S.failed))) break;
        tc::fence_after();
        tc::ld32(t_dp + mine, y);
        tc::wait_ld32(y);
#pragma unroll
        for (int e = 0; e < kCols / 2; ++e) {
          const float2 a = mul2(pair(x, 2 * e), add2(pair(y, 2 * e), make_float2(delta, delta)));
          pk[e] = Bf16::pack(a.x, a.y);
        }
        tc::st16(buf, pk);
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.ds_full);
      }
      if (!ok) break;

      const int rows = u.rows - quarter * 32;
      const long long tok0 = u.row0 + quarter * 32;
      constexpr int kMine = D / kParts;
      unsigned char* dq = p.dq.p + 2 * (tok0 * p.dq.ts + (long long)head * p.dq.hs + part * kMine);
      bool fine = true;
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.acc_full, units & 1u, &S.failed))) break;
        ++units;
        tc::fence_after();
        fine = store_part<D>(t_dq + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kMine), p.scale, vis <= 0, dq,
                             2 * p.dq.ts, rows, lane);
      } else {
        clear_part<D>(dq, 2 * p.dq.ts, rows, lane);
      }
      const bool odd = __any_sync(0xffffffffu, there && !fine);
      if (lane == 0) flags[(size_t)w * kGradFlags + kParts * quarter + part] = odd;
      tc::fence_before();
    }
  }
  end(p, S, warp);
}

template <class K, class... A>
int launch(K kernel, const PackedParams& p, int D, size_t smem, long long most, const PackedList& list, uint8_t* flags, int sms,
           bool* ready, void* stream, A... more) {
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
  return (int)cudaLaunchKernelEx(&cfg, kernel, q, k, v, d_o, p, list, flags, more...);
}
template <int D>
int launch_dq(const PackedParams& p, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  static bool ready[64] = {};
  return launch(dq_kernel<D>, p, D, kGradSmem<D>, (long long)most_units(p.q_tokens, p.B, kGradRows) * p.q_heads, list, flags,
                sms, ready, stream);
}
template <int D>
int launch_dkv(const PackedParams& p, const PackedList& list, uint8_t* flags, bool behind_dq, int sms, void* stream) {
  static bool ready[64] = {};
  return launch(dkv_kernel<D>, p, D, kGradSmem<D>, (long long)most_units(p.kv_tokens, p.B, kGradRows) * p.kv_heads, list,
                flags, sms, ready, stream, behind_dq);
}

}  // namespace

int launch_dq_tc(const PackedParams& p, int d, const PackedList& list, uint8_t* flags, int sms, void* stream) {
  return d == 64 ? launch_dq<64>(p, list, flags, sms, stream) : launch_dq<128>(p, list, flags, sms, stream);
}
int launch_dkv_tc(const PackedParams& p, int d, const PackedList& list, uint8_t* flags, bool behind_dq, int sms,
                  void* stream) {
  return d == 64 ? launch_dkv<64>(p, list, flags, behind_dq, sms, stream)
                 : launch_dkv<128>(p, list, flags, behind_dq, sms, stream);
}

}  // namespace dflash
