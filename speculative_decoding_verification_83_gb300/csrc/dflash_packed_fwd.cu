// dflash_packed_fwd.cu -- attention over packed sequences on the 5th-generation
// tensor cores.
//
// One pass over the keys with a running maximum and sum per row. A unit is 256
// queries of one sequence and head, two tiles of 128 rows that share every tile of
// 128 keys; persistent CTAs, one per SM, take units of a list that begins
// with the largest, from either end of each round in turn (unit_of).
//
// What bounds it: the products, 2 x 128 x 128 x D multiply-adds per tile of keys
// and of queries, against 128 x 128 exponentials. So the two tiles alternate: while
// the tensor cores work on one, the other's scores are turned into weights by 8 warps,
// two for each quarter of the lanes, half of the columns each (with one thread a
// row the chain of load, maximum, exponentials and store took longer than the products
// of both tiles: 8192 tokens, 32 heads of 128, causal took 492 us, and 421 with two and the
// products issued from uniform control flow). The two exchange a
// row's maximum through shared memory; 2^(x - m) goes back to tensor memory as 16-bit
// pairs (over the thread's own scores, or beside them), from where the product with V
// reads them, beginning with the first half that is there. m may lag behind by kSlack
// powers of 2, so that the sums in tensor memory are rarely rescaled.
//  * warp 17: loads. Queries, and the tiles of keys and values in a ring, by TMA; tiles
//    that reach past a sequence's end hold the next one's rows, which count as masked.
//  * warp 16: products. For each tile of keys and each tile of queries: O += P V, then
//    the next S = Q K^T over the scores that P has replaced.
//  * warps 0-7 and 8-15: the weights of the first and the second tile, and the rows'
//    ends.
// A unit takes 4.5 us and 1.49 us for each tile of keys (head_dim 128): 4 x 4096 tokens,
// 16 heads, all keys 375 us (1.47 PFLOP/s), 8192 tokens, 32 heads, causal 385 us.
// Rows with a result that is not finite are flagged (see dflash_packed.cuh). Every
// wait is bounded; a CTA that gives up raises DFLASH_STATUS_TIMEOUT.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_packed_mma.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 576, kMmaWarp = 16, kLoadWarp = 17;
constexpr int kKeys = 128;
constexpr float kSlack = 8.0f;
// Where the reference lies below the score that last moved it: f16 holds normal
// numbers from 2^-14 to below 2^16, so that score's weight is 2^7 and the largest 2^15.
template <class T>
constexpr float kTop = std::is_same<T, F16>::value ? 7.0f : 0.0f;

template <int D>
struct FwdShape {
  static constexpr int kSlots = D == 128 ? 5 : 10;            // tiles of keys or values
  static constexpr uint32_t kTileBytes = 128u * D * 2u;       // of 128 rows
  static constexpr size_t kTiles = (2 + kSlots) * (size_t)kTileBytes;
  // Tensor memory: S0, S1, then O0, O1. With head_dim 64 there is room for the weights beside
  // the scores, so that the next scores are issued as soon as these have been read.
  static constexpr bool kBeside = D == 64;
  static constexpr int kS = 0, kO = 256, kOStep = kBeside ? 64 : 128;
  static constexpr int kP = kBeside ? 384 : 0, kPStep = kBeside ? 64 : 128, kPHalf = kBeside ? 32 : 64;
};
struct FwdShared {
  uint64_t q_full, q_empty, full[10], empty[10];
  uint64_t s_full[2], s_read[2], p_half[2], p_full[2], pv_done[2], o_full[2], drained;
  uint64_t met[2][4];        // of the two warps that share rows
  float row[2][2][128];      // what they exchange: a row's largest score, at a unit's end its sum
  uint32_t tmem;
  volatile int failed;
};
template <int D>
constexpr size_t kFwdSmem = FwdShape<D>::kTiles + sizeof(FwdShared);
static_assert(kFwdSmem<128> <= 232448 && kFwdSmem<64> <= 232448, "one CTA's shared memory (227 KB)");

// Tiles of keys that rows r0 .. of a unit see.
__device__ __forceinline__ int key_tiles(const PackedUnit& u, int causal, int r0) {
  if (r0 >= u.rows) return 0;
  const int last = u.i0 + min(u.rows, r0 + 128) - 1;
  return (seen_keys(causal, u.n, u.m, last) + kKeys - 1) / kKeys;
}

// kTrain: for a backward pass. The outputs' low bits are written, and rows are divided by
// the sum of their rounded weights: where few keys rule a row, the rounding then cancels
// (an error of dq of 2.4e-3 instead of 2.55e-3 at 1111 keys, rounding to bf16 alone
// being 1.65e-3, since the outputs enter the gradients), at two operations a pair. Other
// calls divide by the sum of the weights as they were (outputs 2.05e-3 off in bf16, 2.7e-4 in f16,
// where rounding the outputs alone leaves 1.64e-3 and 2.05e-4).
template <class T, int D, bool kTrain>
__global__ void __launch_bounds__(kThreads, 1)
    forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const PackedParams p, const PackedList list, uint8_t* flags) {
  using W = FwdShape<D>;
  constexpr int kSlots = W::kSlots;
  constexpr uint32_t kTile = W::kTileBytes;
  extern __shared__ __align__(1024) unsigned char raw[];
  FwdShared& S = *reinterpret_cast<FwdShared*>(raw + W::kTiles);
  const uint32_t base = smem_addr(raw), ring = base + 2 * kTile;
  if (base & 1023u) {  // (the dynamic part begins on such a boundary)
    if (threadIdx.x == 0) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&S.q_full, 1);
    mbar_init(&S.q_empty, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&S.s_full[s], 1);
      mbar_init(&S.s_read[s], 8);
      mbar_init(&S.p_half[s], 8);
      mbar_init(&S.p_full[s], 8);
      mbar_init(&S.pv_done[s], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&S.met[s][q], 2);
      mbar_init(&S.o_full[s], 1);
    }
    mbar_init(&S.drained, 1);
    S.failed = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tc::alloc(&S.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  constexpr uint32_t tmem = 0;  // (all of it is ours, so it begins at 0)
  grid_dependency_sync();
  const int work = *list.count * p.q_heads;  // (below 2^27)

  if (warp == kLoadWarp) {
    if (lane == 0) {
      int slot = 0, units = 0;
      uint32_t rounds = 0;  // of the ring
      long long issued = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int head, int row) {
        if (rounds > 0 && !(ok = bounded_wait(&S.empty[slot], (rounds - 1) & 1u, &S.failed))) return;
        mbar_arrive_expect_tx(&S.full[slot], kTile);
        const uint32_t dst = ring + (uint32_t)slot * kTile;
#pragma unroll
        for (int d = 0; d < D; d += 64) tc::load_3d(dst + (uint32_t)d * 256u, map, d, head, row, &S.full[slot]);
        ++issued;
        if (++slot == kSlots) {
          slot = 0;
          ++rounds;
        }
      };
      PackedUnit next = {};
      if (blockIdx.x < work) next = list.units[blockIdx.x / p.q_heads];
      for (int round = 0; ok; ++round) {
        const int w = unit_of(round);
        if (w >= work) break;
        const PackedUnit u = next;
        if (unit_of(round + 1) < work) next = list.units[unit_of(round + 1) / p.q_heads];
        const int head = w % p.q_heads, kh = head / p.G;
        const int tiles = max(key_tiles(u, p.causal, 0), key_tiles(u, p.causal, 128));
        if (!tiles) continue;
        if (units > 0 && !(ok = bounded_wait(&S.q_empty, (uint32_t)(units - 1) & 1u, &S.failed))) break;
        const int parts = u.rows > 128 ? 2 : 1;
        mbar_arrive_expect_tx(&S.q_full, (uint32_t)parts * kTile);
        for (int s = 0; s < parts; ++s)
#pragma unroll
          for (int d = 0; d < D; d += 64)
            tc::load_3d(base + (uint32_t)s * kTile + (uint32_t)d * 256u, &map_q, d, head, u.row0 + 128 * s, &S.q_full);
        ++units;
        for (int j = 0; j < tiles && ok; ++j) {
          load(&map_k, kh, u.other0 + j * kKeys);
          if (ok) load(&map_v, kh, u.other0 + j * kKeys);
        }
      }
      // every copy has landed before the CTA may end
      if (units) (void)mbar_wait_landed(&S.q_full, (uint32_t)(units - 1) & 1u);
      for (long long i = issued > kSlots ? issued - kSlots : 0; i < issued; ++i)
        (void)mbar_wait_landed(&S.full[i % kSlots], (uint32_t)(i / kSlots) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t lead = tc::elect();
    constexpr uint32_t id_s = tc::idesc<T>(128, kKeys, false, false), id_o = tc::idesc<T>(128, D, false, true);
    int units = 0;            // units with keys
    int slot = 0;             // the ring's next tile, and the parity of its round
    uint32_t phase = 0;
    int weights[2] = {0, 0};  // tiles of weights taken so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool done = bounded_warp_wait(bar, parity, &S.failed);
      tc::fence_after();
      return done;
    };
    auto advance = [&] {
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1u;
      }
    };
    auto scores = [&](int s, uint32_t ka) {
      const uint32_t qa = base + (uint32_t)s * kTile;
      const uint64_t q = tc::operand(qa), k = tc::operand(ka);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)  // (addresses count in 16 bytes)
        tc::mma_ss(W::kS + s * 128, q + (uint64_t)((i >> 2) * 1024 + (i & 3) * 2), k + (uint64_t)((i >> 2) * 1024 + (i & 3) * 2),
                   id_s, i > 0, lead);
      tc::commit(&S.s_full[s], lead);
    };
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.q_heads];
      const int n[2] = {tc::uniform(key_tiles(u, p.causal, 0)), tc::uniform(key_tiles(u, p.causal, 128))};
      const int tiles = max(n[0], n[1]);
      if (!tiles) continue;
      if (!(ok = wait(&S.q_full, (uint32_t)units & 1u)) || !(ok = wait(&S.full[slot], phase))) break;
      ++units;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (n[s] > 0) scores(s, ring + (uint32_t)slot * kTile);
      tc::commit(&S.empty[slot], lead);
      if (tiles == 1) tc::commit(&S.q_empty, lead);
      advance();
      for (int j = 0; j < tiles; ++j) {
        // this tile's values and the next one's keys, ahead of the waits for weights
        const int v = slot;
        if (!(ok = wait(&S.full[v], phase))) break;
        advance();
        const bool more = j + 1 < tiles;
        if (more && !(ok = wait(&S.full[slot], phase))) break;
        const uint64_t vd = tc::operand(ring + (uint32_t)v * kTile, 16384u);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok || j >= n[s]) continue;
          const uint32_t parity = (uint32_t)weights[s] & 1u;
          ++weights[s];
          // a quarter of the keys' weights of each half: keys 0-31 and 64-95, then the rest
          auto product = [&](int part) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = (i >> 1) * 4 + 2 * part + (i & 1);  // 16 keys
              tc::mma_ts(W::kO + s * W::kOStep, W::kP + s * W::kPStep + (k >> 2) * W::kPHalf + (k & 3) * 8,
                         vd + (uint64_t)(k * 128), id_o, j > 0 || part > 0 || i > 0, lead);
            }
          };
          if (W::kBeside && j + 1 < n[s]) {
            if (!(ok = wait(&S.s_read[s], parity))) continue;
            scores(s, ring + (uint32_t)slot * kTile);
          }
          if (!(ok = wait(&S.p_half[s], parity))) continue;
          product(0);
          if (!(ok = wait(&S.p_full[s], parity))) continue;
          product(1);
          if (W::kBeside) tc::commit(&S.pv_done[s], lead);
          if (j == n[s] - 1) tc::commit(&S.o_full[s], lead);
          if (!W::kBeside && j + 1 < n[s]) scores(s, ring + (uint32_t)slot * kTile);
        }
        if (!ok) break;
        tc::commit(&S.empty[v], lead);
        if (more) {
          tc::commit(&S.empty[slot], lead);
          advance();
        }
        if (j + 2 == tiles) tc::commit(&S.q_empty, lead);
      }
    }
    tc::commit(&S.drained, lead);  // nothing is left in flight when the tensor memory is freed
    (void)mbar_wait_landed(&S.drained, 0);
    __syncwarp();
  } else {
    const int s = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t scores = my + W::kS + s * 128 + half * 64, sums = my + W::kO + s * W::kOStep + half * (D / 2);
    const uint32_t weights = my + W::kP + s * W::kPStep + half * W::kPHalf;
    const float c = p.scale * kLog2e;
    int tile = 0, ends = 0;  // of this tile of queries: score tiles and units so far
    uint32_t meets = 0;
    bool ok = true;
    // The two warps that share rows: `come` says that this one has written or read what
    // they exchange, `meet` waits for the other to have said so.
    auto come = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.met[s][quarter]);
    };
    auto meet = [&] { return bounded_warp_wait(&S.met[s][quarter], meets++ & 1u, &S.failed); };
    come();  // nothing is read yet
    for (int round = 0; ok; ++round) {
      const int w = unit_of(round);
      if (w >= work) break;
      const PackedUnit u = list.units[w / p.q_heads];
      const int head = w % p.q_heads, r = s * 128 + row;
      const int n = key_tiles(u, p.causal, s * 128);
      const int vis = r < u.rows ? seen_keys(p.causal, u.n, u.m, u.i0 + r) : 0;
      const int vis0 = seen_keys(p.causal, u.n, u.m, u.i0 + s * 128);  // the tile's first row sees least
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      [[maybe_unused]] float2 rounded = make_float2(0.0f, 0.0f);  // sums of the weights, and of the rounded ones
      if (!(ok = meet())) break;  // the sums of the unit before are read
      for (int j = 0; j < n; ++j, ++tile) {
        if (!(ok = bounded_warp_wait(&S.s_full[s], (uint32_t)tile & 1u, &S.failed))) break;
        tc::fence_after();
        const bool border = (j + 1) * kKeys > vis0;  // some row does not see all of the tile
        uint32_t x[32];  // (64 do not fit beside the rest of a thread's 96 registers)
        auto mask = [&](int c0) {
          if (border) {
            const int left = vis - j * kKeys - half * 64 - c0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= left) x[i] = 0xff800000u;
          }
        };
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c0 = 32; c0 >= 0; c0 -= 32) {
          tc::ld32(scores + c0, x);
          tc::wait_ld32(x);
          mask(c0);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) top4[e] = fmaxf(top4[e], __uint_as_float(x[i + e]));
        }
        float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        // (written again only when the partner has given its weights of this tile, so it has read)
        S.row[s][half][row] = top;
        come();
        if (!(ok = meet())) break;
        top = fmaf(fmaxf(top, S.row[s][half ^ 1][row]), c, -kTop<T>);
        const bool move = top > m + kSlack || (m == -INFINITY && top > m);
        // the product before: where the weights lie over the scores it was issued ahead of these, so it is done
        if (W::kBeside && tile > 0 && !(ok = bounded_warp_wait(&S.pv_done[s], (uint32_t)(tile - 1) & 1u, &S.failed))) break;
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? (m == -INFINITY ? 0.0f : ex2_approx(m - top)) : 1.0f;
          if (j > 0) {
            if (W::kBeside) tc::fence_after();
#pragma unroll 1
            for (int d = 0; d < D / 2; d += 16) {
              uint32_t y[16];
              tc::ld16(sums + d, y);
              tc::wait_ld16(y);
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tc::st16(sums + d, y);
            }
          }
          l2 = mul2(l2, make_float2(f, f));
          if (kTrain) rounded = mul2(rounded, make_float2(f, f));
          if (move) m = top;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < 64; i += 32) {
          if (i) {
            tc::ld32(scores + i, x);  // (what lies over the scores so far are weights of the first 32)
            tc::wait_ld32(x);
            if (W::kBeside) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&S.s_read[s]);
            }
            mask(i);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, r2);
            const float2 wt = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            l2 = add2(l2, wt);
            x[e] = T::pack(wt.x, wt.y);  // (pairs take the place of what has been read)
            if (kTrain) rounded = add2(rounded, make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)));
          }
          tc::st16(weights + i / 2, x);
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(i ? &S.p_full[s] : &S.p_half[s]);
        }
      }
      if (!ok) break;

      // ---- the rows' ends: half of the columns each
      come();
      if (!(ok = meet())) break;  // the last maximum is read
      S.row[s][half][row] = l2.x + l2.y;
      come();
      if (!(ok = meet())) break;
      const float l = S.row[s][0][row] + S.row[s][1][row];
      come();  // the sums are read
      float by = l;
      if (kTrain) {
        if (!(ok = meet())) break;
        S.row[s][half][row] = rounded.x + rounded.y;
        come();
        if (!(ok = meet())) break;
        by = S.row[s][0][row] + S.row[s][1][row];
        come();
      }
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.o_full[s], (uint32_t)ends & 1u, &S.failed))) break;
        ++ends;
        tc::fence_after();
      }
      const float inv = by == 0.0f ? 0.0f : __frcp_rn(by);
      const int rows = u.rows - s * 128 - quarter * 32;  // of this warp's 32
      const long long tok0 = u.row0 + s * 128 + quarter * 32;
      unsigned char* out = p.o.p + 2 * (tok0 * p.o.ts + (long long)head * p.o.hs) + half * D;
      unsigned char* low_out = reinterpret_cast<unsigned char*>(p.low) + (tok0 * p.q_heads + head) * D + half * (D / 2);
      float2 probe = make_float2(0.0f, 0.0f);  // NaN once a result is not finite
      const bool none = l == 0.0f;
#pragma unroll 1
      for (int d = 0; d < D / 2; d += 32) {
        uint32_t y[32], o[16];
        if (n > 0) {
          tc::ld32(sums + d, y);
          tc::wait_ld32(y);
        }
        if (__any_sync(0xffffffffu, none)) {  // a row that sees nothing is 0, whatever the products left there
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = none ? 0u : y[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 f = mul2(make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), make_float2(inv, inv));
          o[i] = T::pack(f.x, f.y);
          y[2 * i] = __float_as_uint(f.x);
          y[2 * i + 1] = __float_as_uint(f.y);
          probe = fma2(f, make_float2(0.0f, 0.0f), probe);
        }
        if (kTrain) {
          uint32_t low[8];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t two = (uint32_t)(uint8_t)low_bits(__uint_as_float(y[2 * i]), o[i] & 0xffffu) |
                                 (uint32_t)(uint8_t)low_bits(__uint_as_float(y[2 * i + 1]), o[i] >> 16) << 8;
            low[i >> 1] = i & 1 ? low[i >> 1] | two << 16 : two;
          }
          store_rows<2>(low, low_out + d, (long long)p.q_heads * D, rows, lane);
        }
        store_rows<4>(o, out + 2 * d, 2 * p.o.ts, rows, lane);
      }
      tc::fence_before();
      const bool there = r < u.rows;
      if (there && half == 0 && p.lse)
        p.lse[(tok0 + lane) * p.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      // (a sum of weights that is not finite leaves NaN everywhere, which nothing mends)
      const bool odd = __any_sync(0xffffffffu, probe.x + probe.y != 0.0f && there && l < INFINITY);
      if (lane == 0) flags[(size_t)w * kForwardFlags + s * 8 + 2 * quarter + half] = odd;
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, 512);
  if (tid == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

template <class T, int D, bool kTrain>
int launch(const PackedParams& p, const PackedList& list, uint8_t* flags, int sms, cudaStream_t stream) {
  using W = FwdShape<D>;
  constexpr bool bf16 = std::is_same<T, Bf16>::value;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(forward_kernel<T, D, kTrain>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFwdSmem<D>);
    if (e != cudaSuccess) return (int)e;
    ready[dev] = true;
  }
  CUtensorMap q, k, v;
  if (!map_heads(&q, bf16, p.q, p.q_tokens, p.q_heads, D, 128)) return (int)cudaErrorInvalidValue;
  k = v = q;  // (without keys nothing is loaded)
  if (p.kv_tokens && (!map_heads(&k, bf16, p.k, p.kv_tokens, p.kv_heads, D, kKeys) ||
                      !map_heads(&v, bf16, p.v, p.kv_tokens, p.kv_heads, D, kKeys)))
    return (int)cudaErrorInvalidValue;
  const long long most = (long long)most_units(p.q_tokens, p.B, kForwardRows) * p.q_heads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kFwdSmem<D>;
  return (int)cudaLaunchKernelEx(&cfg, forward_kernel<T, D, kTrain>, q, k, v, p, list, flags);
}

}  // namespace

int launch_forward_tc(const PackedParams& p, int dtype, int d, const PackedList& list, uint8_t* flags, int sms,
                      void* stream) {
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == DFLASH_F16)
    return d == 64 ? launch<F16, 64, false>(p, list, flags, sms, st) : launch<F16, 128, false>(p, list, flags, sms, st);
  if (p.low)
    return d == 64 ? launch<Bf16, 64, true>(p, list, flags, sms, st) : launch<Bf16, 128, true>(p, list, flags, sms, st);
  return d == 64 ? launch<Bf16, 64, false>(p, list, flags, sms, st) : launch<Bf16, 128, false>(p, list, flags, sms, st);
}

}  // namespace dflash
