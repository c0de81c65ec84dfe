// dflash_packed_fwd.cu -- attention over packed sequences on the 5th-generation
// tensor cores.
//
// One pass over the keys with a running maximum and sum per row. A unit is 256
// queries of one sequence and head, two tiles of 128 rows that share every tile of
// 128 keys; persistent CTAs, one per SM, take every gridDim-th unit of a list that
// begins with the largest.
//
// What bounds it: the products, 2 x 128 x 128 x D multiply-adds per tile of keys
// and of queries, against 128 x 128 exponentials. So the two tiles alternate: while
// the tensor cores work on one, 128 threads, a row each, turn the other's scores
// into weights. A thread reads its row of scores for the maximum, then 2^(x - m) goes
// back over the scores as 16-bit pairs, from where the product with V reads them
// (half a row stays in registers between the two; a whole one spills). m may lag behind by kSlack powers of 2, so that
// the sums in tensor memory are rarely rescaled; they are quiet then anyway, since
// the product before was issued ahead of these scores.
//  * warp 9: loads. Queries, and the tiles of keys and values in a ring, by TMA; tiles
//    that reach past a sequence's end hold the next one's rows, which count as masked.
//  * warp 8: products. For each tile of keys and each tile of queries: O += P V, then
//    the next S = Q K^T over the scores that P has replaced.
//  * warps 0-3 and 4-7: the weights of the first and the second tile, and the rows'
//    ends.
// Rows with a result that is not finite are flagged (see dflash_packed.cuh). Every
// wait is bounded; a CTA that gives up raises DFLASH_STATUS_TIMEOUT.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_packed_mma.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 320, kMmaWarp = 8, kLoadWarp = 9;
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
  static constexpr size_t kSmem = 1024 + (2 + kSlots) * (size_t)kTileBytes;
  static constexpr int kS = 0, kO = 256;                      // tensor memory: S0, S1, O0, O1
};
struct FwdShared {
  uint64_t q_full, q_empty, full[10], empty[10];
  uint64_t s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  volatile int failed;
};
static_assert(FwdShape<128>::kSmem + sizeof(FwdShared) <= 232448, "one CTA's shared memory (227 KB)");

// Tiles of keys that rows r0 .. of a unit see.
__device__ __forceinline__ int key_tiles(const PackedUnit& u, int causal, int r0) {
  if (r0 >= u.rows) return 0;
  const int last = u.i0 + min(u.rows, r0 + 128) - 1;
  return (seen_keys(causal, u.n, u.m, last) + kKeys - 1) / kKeys;
}

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const PackedParams p, const PackedList list, uint8_t* flags) {
  using W = FwdShape<D>;
  constexpr int kSlots = W::kSlots;
  constexpr uint32_t kTile = W::kTileBytes;
  extern __shared__ unsigned char raw[];
  __shared__ FwdShared S;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u, ring = base + 2 * kTile;
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
      mbar_init(&S.p_full[s], 128);
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
  const uint32_t tmem = S.tmem;
  grid_dependency_sync();
  const long long work = (long long)*list.count * p.q_heads;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      int slot = 0, units = 0;
      uint32_t round = 0;
      long long issued = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int head, int row) {
        if (round > 0 && !(ok = bounded_wait(&S.empty[slot], (round - 1) & 1u, &S.failed))) return;
        mbar_arrive_expect_tx(&S.full[slot], kTile);
        const uint32_t dst = ring + (uint32_t)slot * kTile;
#pragma unroll
        for (int d = 0; d < D; d += 64) tc::load_3d(dst + (uint32_t)d * 256u, map, d, head, row, &S.full[slot]);
        ++issued;
        if (++slot == kSlots) {
          slot = 0;
          ++round;
        }
      };
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.q_heads];
        const int head = (int)(w % p.q_heads), kh = head / p.G;
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
    if (lane == 0) {
      constexpr uint32_t id_s = tc::idesc<T>(128, kKeys, false, false), id_o = tc::idesc<T>(128, D, false, true);
      int units = 0, t = 0;     // units with keys, ring tiles before this unit
      int weights[2] = {0, 0};  // tiles of weights taken so far
      bool ok = true;
      auto full = [&](int i) {
        if (!bounded_wait(&S.full[i % kSlots], (uint32_t)(i / kSlots) & 1u, &S.failed)) return false;
        tc::fence_after();
        return true;
      };
      auto scores = [&](int s, int i) {
        const uint32_t qa = base + (uint32_t)s * kTile, ka = ring + (uint32_t)(i % kSlots) * kTile;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + W::kS + s * 128, tc::operand(qa + (uint32_t)((k >> 2) * 16384 + (k & 3) * 32)),
                     tc::operand(ka + (uint32_t)((k >> 2) * 16384 + (k & 3) * 32)), id_s, k > 0);
        tc::commit(&S.s_full[s]);
      };
      for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
        const PackedUnit u = list.units[w / p.q_heads];
        const int n[2] = {key_tiles(u, p.causal, 0), key_tiles(u, p.causal, 128)}, tiles = max(n[0], n[1]);
        if (!tiles) continue;
        if (!(ok = bounded_wait(&S.q_full, (uint32_t)units & 1u, &S.failed)) || !(ok = full(t))) break;
        ++units;
        for (int s = 0; s < 2; ++s)
          if (n[s] > 0) scores(s, t);
        tc::commit(&S.empty[t % kSlots]);
        if (tiles == 1) tc::commit(&S.q_empty);
        for (int j = 0; j < tiles && ok; ++j) {
          const int v = t + 2 * j + 1, next = t + 2 * j + 2;
          if (!(ok = full(v))) break;
          const uint32_t va = ring + (uint32_t)(v % kSlots) * kTile;
          bool loaded = false;
          for (int s = 0; s < 2 && ok; ++s) {
            if (j < n[s]) {
              if (!(ok = bounded_wait(&S.p_full[s], (uint32_t)weights[s] & 1u, &S.failed))) break;
              ++weights[s];
              tc::fence_after();
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                tc::mma_ts(tmem + W::kO + s * 128, tmem + W::kS + s * 128 + 8 * k, tc::operand(va + k * 2048u, 16384u), id_o,
                           j > 0 || k > 0);
              if (j == n[s] - 1) tc::commit(&S.o_full[s]);
            }
            if (j + 1 < n[s]) {
              if (!loaded && !(ok = full(next))) break;
              loaded = true;
              scores(s, next);
            }
          }
          if (!ok) break;
          tc::commit(&S.empty[v % kSlots]);
          if (j + 1 < tiles) tc::commit(&S.empty[next % kSlots]);
          if (j + 2 == tiles) tc::commit(&S.q_empty);
        }
        t += 2 * tiles;
      }
      tc::commit(&S.drained);  // nothing is left in flight when the tensor memory is freed
      (void)mbar_wait_landed(&S.drained, 0);
    }
    __syncwarp();
  } else {
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t my = tmem + ((uint32_t)((warp & 3) * 32) << 16), scores = my + W::kS + s * 128, sums = my + W::kO + s * 128;
    const float c = p.scale * kLog2e;
    int tile = 0, ends = 0;  // of this tile of queries: score tiles and units so far
    bool ok = true;
    for (long long w = blockIdx.x; w < work && ok; w += gridDim.x) {
      const PackedUnit u = list.units[w / p.q_heads];
      const int head = (int)(w % p.q_heads), r = s * 128 + row;
      const int n = key_tiles(u, p.causal, s * 128);
      const int vis = r < u.rows ? seen_keys(p.causal, u.n, u.m, u.i0 + r) : 0;
      const int vis0 = seen_keys(p.causal, u.n, u.m, u.i0 + s * 128);  // the tile's first row sees least
      float m = -INFINITY;
      float2 l2 = make_float2(0.0f, 0.0f);
      for (int j = 0; j < n; ++j, ++tile) {
        if (!(ok = bounded_warp_wait(&S.s_full[s], (uint32_t)tile & 1u, &S.failed))) break;
        tc::fence_after();
        // half a row of scores at a time; the first half stays in registers
        const int left = (j + 1) * kKeys > vis0 ? vis - j * kKeys : kKeys;
        uint32_t x[64];
        auto read = [&](int c0) {
          tc::ld32(scores + c0, x);
          tc::ld32(scores + c0 + 32, x + 32);
          tc::wait_ld32(x);
          tc::wait_ld32(x + 32);
          if (__any_sync(0xffffffffu, left < kKeys)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (c0 + i >= left) x[i] = 0xff800000u;
          }
        };
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c0 = 64; c0 >= 0; c0 -= 64) {
          read(c0);
#pragma unroll
          for (int i = 0; i < 64; i += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) top4[e] = fmaxf(top4[e], __uint_as_float(x[i + e]));
        }
        const float top = fmaf(fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])), c, -kTop<T>);
        const bool move = top > m + kSlack || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? (m == -INFINITY ? 0.0f : ex2_approx(m - top)) : 1.0f;
          if (j > 0) {
            // the product before was issued ahead of these scores, so it is done
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t y[32];
              tc::ld32(sums + d, y);
              tc::wait_ld32(y);
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tc::st32(sums + d, y);
            }
          }
          l2.x *= f;
          l2.y *= f;
          if (move) m = top;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
#pragma unroll
        for (int c0 = 0; c0 < 128; c0 += 64) {
          if (c0) read(c0);  // (the weights of the first half replace scores of the first half)
#pragma unroll
          for (int i = 0; i < 64; i += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y =
                  fma2(make_float2(__uint_as_float(x[i + 2 * e]), __uint_as_float(x[i + 2 * e + 1])), c2, r2);
              const float2 wt = make_float2(ex2_approx(y.x), ex2_approx(y.y));
              l2 = add2(l2, wt);
              pk[e] = T::pack(wt.x, wt.y);
            }
            tc::st16(scores + (c0 + i) / 2, pk);
          }
        }
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(&S.p_full[s]);
      }
      if (!ok) break;

      // ---- the rows' ends
      const bool there = r < u.rows;
      const long long tok = u.row0 + r, at = tok * p.q_heads + head;
      unsigned char* out = p.o.p + 2 * (tok * p.o.ts + (long long)head * p.o.hs);
      const float l = l2.x + l2.y;
      bool odd = false;
      if (n > 0) {
        if (!(ok = bounded_warp_wait(&S.o_full[s], (uint32_t)ends & 1u, &S.failed))) break;
        ++ends;
        tc::fence_after();
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t y[32];
        if (n > 0) {
          tc::ld32(sums + d, y);
          tc::wait_ld32(y);
        }
        if (!there) continue;
        uint32_t w32[16], low[8];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // (a row that sees nothing is 0, whatever the products left there)
          const float a = l == 0.0f ? 0.0f : __uint_as_float(y[2 * i]) * inv,
                      b = l == 0.0f ? 0.0f : __uint_as_float(y[2 * i + 1]) * inv;
          w32[i] = T::pack(a, b);
          odd |= !(fabsf(a) < INFINITY) || !(fabsf(b) < INFINITY);
          if (p.low) {
            const uint32_t two = (uint32_t)(uint8_t)low_bits(a, w32[i] & 0xffffu) |
                                 (uint32_t)(uint8_t)low_bits(b, w32[i] >> 16) << 8;
            low[i >> 1] = i & 1 ? low[i >> 1] | two << 16 : two;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<uint4*>(out + 2 * d)[i] = make_uint4(w32[4 * i], w32[4 * i + 1], w32[4 * i + 2], w32[4 * i + 3]);
        if (p.low)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            reinterpret_cast<uint4*>(p.low + at * D + d)[i] =
                make_uint4(low[4 * i], low[4 * i + 1], low[4 * i + 2], low[4 * i + 3]);
      }
      if (there && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      // (a sum of weights that is not finite leaves NaN everywhere, which nothing mends)
      odd = __any_sync(0xffffffffu, odd && there && l < INFINITY);
      if (lane == 0) flags[w * kForwardFlags + warp] = odd;
      tc::fence_before();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::dealloc(tmem, 512);
  if (tid == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

template <class T, int D>
int launch(const PackedParams& p, const PackedList& list, uint8_t* flags, int sms, cudaStream_t stream) {
  using W = FwdShape<D>;
  constexpr bool bf16 = std::is_same<T, Bf16>::value;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(forward_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W::kSmem);
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
  cfg.dynamicSmemBytes = W::kSmem;
  return (int)cudaLaunchKernelEx(&cfg, forward_kernel<T, D>, q, k, v, p, list, flags);
}

}  // namespace

int launch_forward_tc(const PackedParams& p, int dtype, int d, const PackedList& list, uint8_t* flags, int sms,
                      void* stream) {
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == DFLASH_BF16)
    return d == 64 ? launch<Bf16, 64>(p, list, flags, sms, st) : launch<Bf16, 128>(p, list, flags, sms, st);
  return d == 64 ? launch<F16, 64>(p, list, flags, sms, st) : launch<F16, 128>(p, list, flags, sms, st);
}

}  // namespace dflash
