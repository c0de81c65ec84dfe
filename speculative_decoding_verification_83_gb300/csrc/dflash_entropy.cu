// dflash_entropy.cu -- cross entropy over the whole vocabulary of hidden states
// through the vocabulary projection, without keeping the logits, and its
// gradients.
//
// z = h W^T, loss_i = w_i (log sum_v e^(z_iv) - z_i,label),
// g_iv = u_i w_i (e^(z_iv) / s_i - [v = label_i]), dh = g W, dW = g^T h.
// Four products of rows x V x K: the logits for the loss, again for g, and the two
// gradients. All run on pairs of SMs of the 5th-generation tensor cores, which is
// what bounds them; few rows are bound by reading W once.
//
// The loss: the epilogue turns each 256 x 256 tile of logits, still in tensor
// memory, into each row's largest logit and sum of exponentials over 128 columns
// (8 bytes for 128 logits), and picks out the labels' logits; a small kernel joins
// them. The gradients go through the vocabulary in pieces: the epilogue writes a
// piece of g in bf16 (kPieceBytes at most, or 4096 entries' worth of more than 2^16 rows; a
// rounding of half a step of the type in which the products want it), from which dW's rows of the piece and the
// piece's part of dh follow. A row's g is often ruled by its label's entry, and one
// rounding then decides the error of the whole row: what it leaves of that entry
// is kept in fp32 and added to dh, and to dW for a label's first kHits rows. dh is summed in fp32 over pieces, in up to kMaxSplits
// buffers where its tiles are too few to fill the SMs; every sum has a fixed
// order.
//
// The product kernel: clusters of two CTAs, persistent over 256 x 256 tiles. Warp 0
// loads [128 x 64] tiles of both operands by TMA into a ring of kStages; an operand
// whose inner index is not the contiguous one is loaded as it lies and read
// transposed. Warp 1 issues the pair's MMAs into one of two 256-column accumulators,
// warps 2-9 turn the other one into the epilogue's result; what goes to memory goes
// through shared memory and tiled stores, which clip at the edges. 1024 rows of 5120
// over 248320 entries, one after the other in 6.0 to 6.7 ms, as the power limit
// allows: logits 1370 us (1.90 PFLOP/s), g 1385, dW 1585 (its 2.5 GB of stores cost 200), dh 1500.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_norm.cuh"
#include "dflash_tcgen05.cuh"
#include "dflash_train.h"

namespace dflash {
namespace {

constexpr int kTile = 256;   // rows and columns of a pair's tile
constexpr int kStep = 64;    // inner values per stage
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = 128u * kStep * 2u;
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kStageOut = 4096;  // a warp's 32 rows of 128 bytes on their way out
constexpr float kLog2e = 1.4426950408889634f;

enum Epilogue { kStats, kLogitGrad, kStoreBf16, kSumF32 };

struct RowGrad {  // what a row's g is computed from
  float m, scale, g;  // e^(z - m) scale, minus g at the label
  int label;          // -1: none in reach, kDead: the row takes no part
};
constexpr int kDead = -2;

struct GemmParams {
  int m, n, k;               // extents
  int tiles_m, tiles_n, splits, k_per_split;  // k_per_split: in stages
  int n_fast;                // tiles of one row of tiles follow each other
  int a_x, a_y, b_x, b_y;    // where the operands begin in their maps: along the inner index (x) and across it (y)
  int chunk;                 // kStats: stages summed in tensor memory at a time
  // kStats
  float2* parts;             // [2 tiles_n][rows_pitch]
  int rows_pitch;
  const int32_t* labels;
  float* label_logit;
  // kLogitGrad
  const RowGrad* rows;
  int label0;                // the piece's first vocabulary entry
  float* rest;               // per row: what rounding left of the label's entry
  // kStoreBf16: a row's rest times its hidden state goes to its label's row
  const int32_t* used;       // the labels of k rows, kDead: takes no part
  const unsigned char* h;
  long long h_stride;
  // kSumF32
  int add;                   // to what is there
  int split_rows;            // rows between the splits' buffers
  uint32_t* status;
};

// Rows of a label whose rests join dW. Each of n rows beyond them adds its own rounding of the label's
// entry, half a step of bf16 at most: where rows differ, about sqrt(n - 4) / n of a half step of their sum's
// size is left out; rows that repeat have equal rests, and (n - 4) / n of one is, almost what rounding every
// entry leaves. All of them would take as long as the products where rows share few labels.
constexpr int kHits = 4;
struct GemmShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  volatile int failed;
};
constexpr size_t kGemmSmem = 1024 + (size_t)kStages * 2 * kOperandBytes + kEpiWarps * kStageOut;
static_assert(kGemmSmem + sizeof(GemmShared) <= 232448, "one CTA's shared memory (227 KB)");

__device__ __forceinline__ bool wait_from(uint64_t* bar, uint32_t parity, unsigned long long t0) {
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, GemmShared& S) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0u && (S.failed || global_timer_ns() - t0 > kWaitLimitNs)) return false;
  }
}
__device__ __forceinline__ bool wait_bar_cluster(uint64_t* bar, uint32_t parity, GemmShared& S) {
  if (tc::try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (tc::try_wait_cluster(bar, parity)) return true;
    if ((it & 31u) == 0u && (S.failed || global_timer_ns() - t0 > kWaitLimitNs)) return false;
  }
}

struct TileAt {
  int m, n, k0, steps, split;  // tile numbers, first stage and count of stages
};
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
  TileAt a;
  const int per = p.tiles_m * p.tiles_n;
  a.split = t / per;
  const int r = t - a.split * per;
  if (p.n_fast) {
    a.m = r / p.tiles_n;
    a.n = r - a.m * p.tiles_n;
  } else {
    a.n = r / p.tiles_m;
    a.m = r - a.n * p.tiles_m;
  }
  a.k0 = a.split * p.k_per_split;
  a.steps = max(0, min(p.k_per_split, (p.k + kStep - 1) / kStep - a.k0));
  return a;
}

// D = A B^T over A [m, k] and B [n, k]. kAMn / kBMn: the operand lies as [k, m] or
// [k, n] in memory (its outer index is the contiguous one).
template <bool kAMn, bool kBMn, Epilogue kEpi>
__global__ void __launch_bounds__(kGemmThreads, 1) __cluster_dims__(2, 1, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_out, const GemmParams p) {
  extern __shared__ unsigned char raw[];
  __shared__ GemmShared S;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cluster_rank();
  const int tiles = p.tiles_m * p.tiles_n * p.splits, first = blockIdx.x / 2, pairs = gridDim.x / 2;
  auto a_mem = [&](int s) { return base + (uint32_t)s * 2u * kOperandBytes; };
  auto b_mem = [&](int s) { return base + (uint32_t)s * 2u * kOperandBytes + kOperandBytes; };

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&S.full[s], 1);   // the first CTA's load warp; both CTAs' bytes
      mbar_init(&S.empty[s], 1);  // the pair's products
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&S.acc_full[a], 1);
      mbar_init(&S.acc_empty[a], 2 * kEpiWarps);
    }
    S.failed = 0;
    fence_barrier_init();
  }
  if (warp == 1) tc::alloc_pair(&S.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers are there before a load or an arrival reaches them
  tc::fence_after();
  constexpr uint32_t tmem = 0;  // (all of it is ours, so it begins at 0)

  if (warp == 0) {
    if (lane == 0) {
      long long it = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += pairs) {
        const TileAt at = tile_at(p, t);
        const int am = at.m * kTile + rank * 128, bn = at.n * kTile + rank * 128;
        for (int ks = 0; ks < at.steps; ++ks, ++it) {
          const int s = (int)(it % kStages);
          if (it >= kStages && !wait_bar(&S.empty[s], (uint32_t)((it / kStages) & 1) ^ 1u, S)) {
            S.failed = 1;
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 4u * kOperandBytes);
          const uint32_t bar = tc::in_first_cta(&S.full[s]);
          const int k = (at.k0 + ks) * kStep;
          // (past an operand's edges zeros are filled in)
          if (kAMn) {
            tc::load_2d_pair(a_mem(s), &map_a, p.a_y + am, p.a_x + k, bar);
            tc::load_2d_pair(a_mem(s) + kOperandBytes / 2, &map_a, p.a_y + am + 64, p.a_x + k, bar);
          } else {
            tc::load_2d_pair(a_mem(s), &map_a, p.a_x + k, p.a_y + am, bar);
          }
          if (kBMn) {
            tc::load_2d_pair(b_mem(s), &map_b, p.b_y + bn, p.b_x + k, bar);
            tc::load_2d_pair(b_mem(s) + kOperandBytes / 2, &map_b, p.b_y + bn + 64, p.b_x + k, bar);
          } else {
            tc::load_2d_pair(b_mem(s), &map_b, p.b_x + k, p.b_y + bn, bar);
          }
        }
      }
      // every load has landed once the products that read it have freed its stage
      const unsigned long long t1 = global_timer_ns();
      for (long long q = it > kStages ? it - kStages : 0; q < it; ++q)
        (void)wait_from(&S.empty[q % kStages], (uint32_t)((q / kStages) & 1), t1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t id = tc::idesc<Bf16>(kTile, kTile, kAMn, kBMn);
      const uint32_t lead = tc::elect();
      int slot = 0, s = 0, use = 0;  // accumulator, stage
      uint32_t phase = 0;
      bool ok = true;
      const int chunk = kEpi == kStats ? p.chunk : 1 << 30;
      for (int t = first, left = 0; t < tiles && ok; t += left > 0 ? 0 : pairs) {
        if (left <= 0) left = tile_at(p, t).steps;
        const int steps = min(left, chunk);
        if (use > 0 && !__all_sync(0xffffffffu, wait_bar_cluster(&S.acc_empty[slot], (uint32_t)((use - 1) & 1), S))) {
          ok = false;
          break;
        }
        tc::fence_after();
        for (int ks = 0; ks < steps; ++ks) {
          if (!__all_sync(0xffffffffu, wait_bar(&S.full[s], phase, S))) {
            ok = false;
            break;
          }
          tc::fence_after();
          const uint64_t ad = tc::operand(a_mem(s), kAMn ? kOperandBytes / 2 : 16u);
          const uint64_t bd = tc::operand(b_mem(s), kBMn ? kOperandBytes / 2 : 16u);
#pragma unroll
          for (int kk = 0; kk < kStep / 16; ++kk)  // 16 inner values: 32 bytes of a row, or 16 rows
            tc::mma_pair((uint32_t)(slot * kTile), ad + (uint64_t)((kAMn ? 128 : 2) * kk),
                         bd + (uint64_t)((kBMn ? 128 : 2) * kk), id, (ks | kk) != 0, lead);
          tc::commit_pair(&S.empty[s], lead);
          if (++s == kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc::commit_pair(&S.acc_full[slot], lead);
        left -= chunk;
        use += slot;
        slot ^= 1;
      }
      if (!ok) S.failed = 1;
    }
  } else {
    // ---- epilogue: a warp reads the lanes of quarter warp % 4, half of the columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t out_mem = base + (uint32_t)kStages * 2u * kOperandBytes + (uint32_t)(warp - 2) * kStageOut;
    int lt = 0;
    bool pending = false;  // a store still reads the staging rows
    auto staged = [&](auto&& write, const CUtensorMap* map, int x, int y, bool add) {
      if (pending && lane == 0) tc::store_wait_read();
      __syncwarp();
      write();
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (add)
          tc::add_2d(map, out_mem, x, y);
        else
          tc::store_2d(map, out_mem, x, y);
        tc::store_commit();
      }
      pending = true;
    };
    // one arrival a warp on the first CTA's barrier, before its products overwrite the slot
    auto release = [&](int slot) {
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(&S.acc_empty[slot]);
        else
          tc::arrive_cluster(tc::in_first_cta(&S.acc_empty[slot]));
      }
    };
    // piece c of this lane's 128-byte row
    auto put = [&](int c, uint4 v) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out_mem + (uint32_t)lane * 128u +
                                                                    (uint32_t)((c ^ (lane & 7)) << 4)),
                   "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    };
    for (int t = first; t < tiles; t += pairs, ++lt) {
      const TileAt at = tile_at(p, t);
      [[maybe_unused]] bool all = true;
      const int row0 = at.m * kTile + rank * 128 + q * 32, row = row0 + lane;
      const int col0 = at.n * kTile + half * 128;
      [[maybe_unused]] int label = -1;
      [[maybe_unused]] RowGrad rg = {0.0f, 0.0f, 0.0f, kDead};
      if (kEpi == kStats && row < p.m) label = p.labels[row];
      if (kEpi == kLogitGrad && row < p.m) rg = p.rows[row];
      // The first rows whose label is this lane's entry, while the products run; 256 rows are looked at at a time.
      [[maybe_unused]] int hits[kHits];
      if constexpr (kEpi == kStoreBf16) {
#pragma unroll
        for (int i = 0; i < kHits; ++i) hits[i] = -1;
        for (int r0 = 0; r0 < p.k; r0 += 256) {
          int at[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = r0 + 32 * e + lane;
            at[e] = r < p.k ? p.used[r] - p.label0 - row0 : -1;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            for (uint32_t found = __ballot_sync(0xffffffffu, at[e] >= 0 && at[e] < 32); found; found &= found - 1) {
              const int k = __ffs(found) - 1;
              int r = __shfl_sync(0xffffffffu, at[e], k) == lane ? r0 + 32 * e + k : -1;
#pragma unroll
              for (int i = 0; i < kHits; ++i)
                if (hits[i] < 0) {
                  hits[i] = r;
                  r = -1;
                }
            }
        }
      }
      if (!__all_sync(0xffffffffu, wait_bar(&S.acc_full[lt & 1], (uint32_t)((lt >> 1) & 1), S))) {
        S.failed = 1;
        break;
      }
      tc::fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((lt & 1) * kTile + half * 128);
      if constexpr (kEpi == kStats) {
        // All but the last chunk of the inner index are added up in registers: every addition in
        // tensor memory cuts bits off, and over 5120 inner values that came to 2.4e-6 of a loss
        // (4.5e-7 in chunks of 1024). The gradients' products do not: what they make is rounded to bf16.
        float total[128];
        for (int left = at.steps - p.chunk, k = 0;; left -= p.chunk, ++k) {
          const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)((lt & 1) * kTile + half * 128);
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t x[32];
            tc::ld32(from + c, x);
            tc::wait_ld32(x);
#pragma unroll
            for (int e = 0; e < 32; ++e) total[c + e] = k ? total[c + e] + __uint_as_float(x[e]) : __uint_as_float(x[e]);
          }
          if (left <= 0) break;
          release(lt & 1);
          ++lt;
          if (!(all = __all_sync(0xffffffffu, wait_bar(&S.acc_full[lt & 1], (uint32_t)((lt >> 1) & 1), S)))) break;
          tc::fence_after();
        }
        if (!all) {
          S.failed = 1;
          break;
        }
        float m = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(total[c + e]);
          const int left = p.n - (col0 + c);  // columns that exist
          if (left < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) x[e] = 0xff800000u;
          }
          const int at_label = label - (col0 + c);
          if (at_label >= 0 && at_label < 32 && at_label < left) {
            float z = 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e == at_label) z = __uint_as_float(x[e]);
            p.label_logit[row] = z;
          }
          float top = m;
#pragma unroll
          for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(x[e]));
          const float ref = top == -INFINITY ? 0.0f : top;
          sum *= ex2_approx((m - ref) * kLog2e);
          float part = 0.0f;
#pragma unroll
          for (int e = 0; e < 32; ++e) part += ex2_approx((__uint_as_float(x[e]) - ref) * kLog2e);
          sum += part;
          m = top;
        }
        if (row < p.m) p.parts[(size_t)(2 * at.n + half) * p.rows_pitch + row] = make_float2(m, sum);
      } else if constexpr (kEpi == kLogitGrad) {
        for (int c = 0; c < 128; c += 64) {
          uint32_t x[64];
          tc::ld32(acc + c, x);
          tc::ld32(acc + c + 32, x + 32);
          tc::wait_ld32(x);
          tc::wait_ld32(x + 32);
          const bool dead = rg.label == kDead;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            x[e] = __float_as_uint(ex2_approx((__uint_as_float(x[e]) - rg.m) * kLog2e) * rg.scale);
          const int at_label = rg.label - (p.label0 + col0 + c);
          if (at_label >= 0 && at_label < 64) {
            float z = 0.0f;
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (e == at_label) {
                z = __uint_as_float(x[e]) - rg.g;
                x[e] = __float_as_uint(z);
              }
            p.rest[row] = z - __uint_as_float(Bf16::pack(z, 0.0f) << 16);
          }
          if (col0 + c < p.n && row0 < p.m)
            staged(
                [&] {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      w[j] = dead ? 0u
                                  : Bf16::pack(__uint_as_float(x[8 * i + 2 * j]), __uint_as_float(x[8 * i + 2 * j + 1]));
                    put(i, make_uint4(w[0], w[1], w[2], w[3]));
                  }
                },
                &map_out, col0 + c, row0, false);
        }
      } else if constexpr (kEpi == kStoreBf16) {
        for (int c = 0; c < 128; c += 64) {
          uint32_t x[64];
          tc::ld32(acc + c, x);
          tc::ld32(acc + c + 32, x + 32);
          tc::wait_ld32(x);
          tc::wait_ld32(x + 32);
#pragma unroll
          for (int i = 0; i < kHits; ++i) {
            if (!__any_sync(0xffffffffu, hits[i] >= 0)) break;
            if (hits[i] < 0) continue;
            const float f = p.rest[hits[i]];
            const uint4* src = reinterpret_cast<const uint4*>(p.h + 2 * (hits[i] * p.h_stride + col0 + c));
            uint4 u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = col0 + c + 8 * j < p.n ? src[j] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float v[8];
              unpack8<Bf16>(u[j], v);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[8 * j + e] = __float_as_uint(fmaf(f, v[e], __uint_as_float(x[8 * j + e])));
            }
          }
          __syncwarp();
          if (col0 + c < p.n && row0 < p.m)
            staged(
                [&] {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      w[j] = Bf16::pack(__uint_as_float(x[8 * i + 2 * j]), __uint_as_float(x[8 * i + 2 * j + 1]));
                    put(i, make_uint4(w[0], w[1], w[2], w[3]));
                  }
                },
                &map_out, col0 + c, row0, false);
        }
      } else {
        for (int c = 0; c < 128; c += 32) {
          uint32_t x[32];
          tc::ld32(acc + c, x);
          tc::wait_ld32(x);
          if (at.steps == 0) {  // a short last piece leaves nothing to the last splits
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = 0u;
          }
          if (col0 + c < p.n && row0 < p.m)
            staged(
                [&] {
#pragma unroll
                  for (int i = 0; i < 8; ++i) put(i, make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
                },
                &map_out, col0 + c, at.split * p.split_rows + row0, p.add != 0);
        }
      }
      release(lt & 1);
    }
    if (lane == 0) tc::store_wait();
  }

  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // no load, commit or arrival of the pair still reaches either CTA
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc_pair(tmem, 512);
  }
  if (tid == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

// ---- few rows
// Up to kFew rows are bound by reading W once, so its rows become the products' M: a
// stage is 16 KB of W and 2 KB of hidden states, and kFewStages of them are in flight
// where the other kernel has 6 with as many bytes of padded rows (7 rows of 5120 over
// 248320 entries: 382 against 499 us, 6.66 TB/s). A lane of the epilogue owns a vocabulary
// entry of the tile and keeps each row's largest logit and sum over all tiles of its CTA;
// lanes are joined once, at the CTA's end.
constexpr int kFew = 32, kFewStages = 12;
constexpr uint32_t kFewBytes = kFew / 2 * kStep * 2u;  // hidden states of a stage and CTA
constexpr int kFewThreads = 32 * 6;
struct FewShared {
  uint64_t full[kFewStages], empty[kFewStages];
  uint64_t acc_full[2], acc_empty[2];
  uint32_t tmem;
  volatile int failed;
  int labels[kFew];
};
constexpr size_t kFewSmem = 1024 + (size_t)kFewStages * (kOperandBytes + kFewBytes);
static_assert(kFewSmem + sizeof(FewShared) <= 232448, "one CTA's shared memory (227 KB)");

__global__ void __launch_bounds__(kFewThreads, 1) __cluster_dims__(2, 1, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h, const GemmParams p) {
  extern __shared__ unsigned char raw[];
  __shared__ FewShared S;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cluster_rank();
  const int first = blockIdx.x / 2, pairs = gridDim.x / 2, stages = (p.k + kStep - 1) / kStep;
  auto w_mem = [&](int s) { return base + (uint32_t)s * kOperandBytes; };
  auto h_mem = [&](int s) { return base + kFewStages * kOperandBytes + (uint32_t)s * kFewBytes; };

  if (tid == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&S.acc_full[a], 1);
      mbar_init(&S.acc_empty[a], 2 * 4);
    }
    S.failed = 0;
    fence_barrier_init();
  }
  if (tid < kFew) S.labels[tid] = tid < p.m ? p.labels[tid] : -1;
  if (warp == 1) tc::alloc_pair(&S.tmem, 512);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();

  if (warp == 0) {
    if (lane == 0) {
      long long it = 0;
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < p.tiles_n && ok; t += pairs)
        for (int ks = 0; ks < stages; ++ks, ++it) {
          if (it >= kFewStages) {
            const unsigned long long t0 = global_timer_ns();
            if (!wait_from(&S.empty[s], phase ^ 1u, t0)) {
              S.failed = 1;
              ok = false;
              break;
            }
          }
          if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2u * (kOperandBytes + kFewBytes));
          const uint32_t bar = tc::in_first_cta(&S.full[s]);
          tc::load_2d_pair(w_mem(s), &map_w, ks * kStep, t * kTile + rank * 128, bar);
          tc::load_2d_pair(h_mem(s), &map_h, ks * kStep, rank * (kFew / 2), bar);
          if (++s == kFewStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      const unsigned long long t1 = global_timer_ns();
      for (long long q = it > kFewStages ? it - kFewStages : 0; q < it; ++q)
        (void)wait_from(&S.empty[q % kFewStages], (uint32_t)((q / kFewStages) & 1), t1);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t id = tc::idesc<Bf16>(kTile, kFew, false, false);
      const uint32_t lead = tc::elect();
      int slot = 0, s = 0, use = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; t < p.tiles_n && ok; t += pairs)
        for (int k0 = 0; k0 < stages && ok; k0 += p.chunk) {
          if (use > 0) {
            const unsigned long long t0 = global_timer_ns();
            bool done = tc::try_wait_cluster(&S.acc_empty[slot], (uint32_t)((use - 1) & 1));
            while (!done && global_timer_ns() - t0 <= kWaitLimitNs)
              done = tc::try_wait_cluster(&S.acc_empty[slot], (uint32_t)((use - 1) & 1));
            if (!(ok = __all_sync(0xffffffffu, done))) break;
          }
          tc::fence_after();
          const int steps = min(p.chunk, stages - k0);
          for (int ks = 0; ks < steps; ++ks) {
            if (!(ok = __all_sync(0xffffffffu, wait_from(&S.full[s], phase, global_timer_ns())))) break;
            tc::fence_after();
            const uint64_t wd = tc::operand(w_mem(s)), hd = tc::operand(h_mem(s));
#pragma unroll
            for (int kk = 0; kk < kStep / 16; ++kk)
              tc::mma_pair((uint32_t)(slot * kFew), wd + (uint64_t)(2 * kk), hd + (uint64_t)(2 * kk), id, (ks | kk) != 0, lead);
            tc::commit_pair(&S.empty[s], lead);
            if (++s == kFewStages) {
              s = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc::commit_pair(&S.acc_full[slot], lead);
          use += slot;
          slot ^= 1;
        }
      if (!ok) S.failed = 1;
    }
  } else {
    const int q = warp & 3;
    float m[kFew], sum[kFew];
#pragma unroll
    for (int c = 0; c < kFew; ++c) m[c] = -INFINITY, sum[c] = 0.0f;
    int lt = 0;
    bool ok = true;
    for (int t = first; t < p.tiles_n && ok; t += pairs) {
      float total[kFew];
      for (int k0 = 0; k0 < stages; k0 += p.chunk, ++lt) {
        if (!(ok = __all_sync(0xffffffffu, wait_from(&S.acc_full[lt & 1], (uint32_t)((lt >> 1) & 1), global_timer_ns())))) break;
        tc::fence_after();
        uint32_t x[kFew];
        tc::ld32(((uint32_t)(q * 32) << 16) + (uint32_t)((lt & 1) * kFew), x);
        tc::wait_ld32(x);
#pragma unroll
        for (int c = 0; c < kFew; ++c) total[c] = k0 ? total[c] + __uint_as_float(x[c]) : __uint_as_float(x[c]);
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0)
            mbar_arrive(&S.acc_empty[lt & 1]);
          else
            tc::arrive_cluster(tc::in_first_cta(&S.acc_empty[lt & 1]));
        }
      }
      if (!ok) break;
      const int v = t * kTile + rank * 128 + q * 32 + lane;
      if (v < p.n) {
#pragma unroll
        for (int c = 0; c < kFew; ++c) {
          const float z = total[c], top = fmaxf(m[c], z), ref = top == -INFINITY ? 0.0f : top;
          sum[c] = sum[c] * ex2_approx((m[c] - ref) * kLog2e) + ex2_approx((z - ref) * kLog2e);
          m[c] = top;
          if (S.labels[c] == v) p.label_logit[c] = z;
        }
      }
    }
    if (!ok) S.failed = 1;
    // the CTA's lanes together
#pragma unroll
    for (int c = 0; c < kFew; ++c) {
      const float top = warp_max_f32(m[c]), ref = top == -INFINITY ? 0.0f : top;
      // (a sum over nothing is 0, or NaN)
      float part = sum[c] * (m[c] == -INFINITY ? 1.0f : ex2_approx((m[c] - ref) * kLog2e));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == 0 && c < p.m) p.parts[((size_t)blockIdx.x * 4 + q) * p.rows_pitch + c] = make_float2(top, part);
    }
  }

  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc_pair(0, 512);
  }
  if (tid == 0 && S.failed) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
}

// Joins the statistics of a row's tiles: 32 rows a block, 32 runs of parts.
__global__ void __launch_bounds__(1024)
    join_kernel(const float2* parts, int n_parts, int pitch, const float* label_logit, const EntropyParams p) {
  __shared__ float2 run[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
  auto add = [](float2 a, float2 b) {  // a sum over nothing is 0, or NaN
    const float m = fmaxf(a.x, b.x);
    const float fa = a.x == -INFINITY ? 1.0f : ex2_approx((a.x - m) * kLog2e);
    const float fb = b.x == -INFINITY ? 1.0f : ex2_approx((b.x - m) * kLog2e);
    return make_float2(m, a.y * fa + b.y * fb);
  };
  float2 s = make_float2(-INFINITY, 0.0f);
  if (row < p.rows)
    for (int i = w; i < n_parts; i += 32) s = add(s, parts[(size_t)i * pitch + row]);
  run[w][lane] = s;
  __syncthreads();
  if (w || row >= p.rows) return;
  for (int i = 1; i < 32; ++i) s = add(s, run[i][lane]);
  const int label = p.labels[row];
  const float weight = p.weight ? p.weight[row] : 1.0f;
  const bool out = label < -1 || label >= p.V, dead = label == -1 || out || weight == 0.0f;
  float loss = 0.0f;
  uint32_t bits = out ? DFLASH_STATUS_BAD_TOKEN : 0u;
  if (!dead) {
    loss = ((s.x - label_logit[row]) + logf(s.y)) * weight;
    if (loss != loss) bits |= DFLASH_STATUS_BAD_ROW;
  }
  p.loss[row] = loss;
  if (p.stats) p.stats[row] = s;
  if (bits) raise_status(p.status, bits);
}

// What each row's gradient is computed from, and the hidden states with the rows
// that take no part set to 0 (their values may be anything, and 0 times anything
// may not be 0 in dW). One block a row.
__global__ void __launch_bounds__(128) rows_kernel(const EntropyParams p, RowGrad* rows, float* rest, int32_t* used,
                                                   uint16_t* h_used) {
  const int r = blockIdx.x, label = p.labels[r];
  const float u = (p.upstream ? p.upstream[(long long)r * p.upstream_stride] : 1.0f);
  const float weight = p.weight ? p.weight[r] : 1.0f;
  const bool dead = label < 0 || label >= p.V || weight == 0.0f || u == 0.0f;
  if (threadIdx.x == 0) {
    const float2 s = p.stats[r];
    const float g = u * weight;
    RowGrad x = {s.x, g / s.y, g, label};
    if (dead) x = {0.0f, 0.0f, 0.0f, kDead};
    rows[r] = x;
    rest[r] = 0.0f;
    used[r] = x.label;
  }
  if (!h_used) return;
  const uint4* src = reinterpret_cast<const uint4*>(p.h + 2 * (long long)r * p.h_stride);
  uint4* dst = reinterpret_cast<uint4*>(h_used + (size_t)r * p.K);
  for (int i = threadIdx.x; i < p.K / 8; i += 128) dst[i] = dead ? make_uint4(0u, 0u, 0u, 0u) : src[i];
}

// dh from its fp32 sums, the splits in order, and the rests of the labels' entries; 0 for
// rows that take no part.
__global__ void __launch_bounds__(256) hidden_kernel(const EntropyParams p, const float* sums, int splits,
                                                     size_t split_stride, const RowGrad* rows, const float* rest) {
  const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= (size_t)p.rows * p.K) return;
  const int r = (int)(at / p.K), k = (int)(at - (size_t)r * p.K), label = rows[r].label;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (label != kDead) {
    const uint4 w = *reinterpret_cast<const uint4*>(p.w + 2 * (label * p.w_stride + k));
    const float f = rest[r];
    float x[8];
    unpack8<Bf16>(w, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= f;
    for (int s = 0; s < splits; ++s) {
      const float* src = sums + s * split_stride + at;
      const float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
      x[0] += a.x, x[1] += a.y, x[2] += a.z, x[3] += a.w, x[4] += b.x, x[5] += b.y, x[6] += b.z, x[7] += b.w;
    }
    v = pack8<Bf16>(x);
  }
  *reinterpret_cast<uint4*>(p.dh + 2 * at) = v;
}

// ---- workspaces
// Of g at a time. Beyond 2^16 rows a piece keeps kLeastPiece entries, 8 KB a row: each piece's part
// of dh is added to fp32 sums, 8 bytes moved for 2 products an entry of the piece.
constexpr long long kPieceBytes = 512ll << 20;
constexpr int kLeastPiece = 16 * kTile;
constexpr int kMaxSplits = 8;
constexpr int kPairs = 76;  // the splits' rule goes by a whole GPU's pairs of SMs

size_t up(size_t n) { return (n + 255) / 256 * 256; }
int tiles_of(long long n) { return (int)((n + kTile - 1) / kTile); }

constexpr int kMaxPairs = 128;  // of SMs, where the workspace counts them
constexpr int kForwardRows = 16384;  // whose statistics are held at a time
struct ForwardPlan {
  int n_parts, pitch;
  size_t parts, labels, bytes;
};
ForwardPlan forward_plan(int rows, int V) {
  ForwardPlan f;
  rows = rows < kForwardRows ? rows : kForwardRows;
  f.n_parts = 2 * tiles_of(V);
  if (rows <= kFew) f.n_parts = 8 * (tiles_of(V) < kMaxPairs ? tiles_of(V) : kMaxPairs);
  f.pitch = (rows + 31) / 32 * 32;
  f.parts = 0;
  f.labels = up((size_t)f.n_parts * f.pitch * sizeof(float2));
  f.bytes = f.labels + up((size_t)rows * sizeof(float));
  return f;
}
struct BackwardPlan {
  int piece, pitch, splits;  // vocabulary entries of a piece, of a row of g
  int split_rows;            // rows of a split's sums: whole stores
  size_t rows, rest, used, h, g, sums, bytes;
};
BackwardPlan backward_plan(int rows, int V, int K) {
  BackwardPlan b;
  long long piece = kPieceBytes / 2 / rows / kTile * kTile;
  if (piece < kLeastPiece) piece = kLeastPiece;
  if (piece > V) piece = V;
  b.piece = (int)piece;
  b.pitch = (b.piece + 63) / 64 * 64;
  // the split whose tiles fill whole rounds of the pairs best; a further one has to gain 4% to pay
  // for the sums that it writes
  const long long tiles = (long long)tiles_of(rows) * tiles_of(K);
  b.splits = 1;
  double best = 0.0;
  for (int s = 1; s <= kMaxSplits && s * 16 * kStep <= b.pitch; ++s) {
    const double rounds = (double)((tiles * s + kPairs - 1) / kPairs), full = (double)(tiles * s) / kPairs / rounds;
    if (full > best + 0.04) {
      best = full;
      b.splits = s;
    }
  }
  b.split_rows = (rows + 31) / 32 * 32;
  b.rows = 0;
  b.rest = up((size_t)rows * sizeof(RowGrad));
  b.used = b.rest + up((size_t)rows * sizeof(float));
  b.h = b.used + up((size_t)rows * sizeof(int32_t));
  b.g = b.h + up((size_t)rows * K * 2);
  b.sums = b.g + up((size_t)rows * b.pitch * 2);
  b.bytes = b.sums + up((size_t)b.splits * b.split_rows * K * sizeof(float));
  return b;
}

template <bool kAMn, bool kBMn, Epilogue kEpi>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, GemmParams p, int sms,
                        cudaStream_t stream) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(gemm_kernel<kAMn, kBMn, kEpi>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  p.tiles_m = tiles_of(p.m);
  p.tiles_n = tiles_of(p.n);
  const int stages = (p.k + kStep - 1) / kStep;
  p.k_per_split = (stages + p.splits - 1) / p.splits;
  p.chunk = 1024 / kStep;
  const long long tiles = (long long)p.tiles_m * p.tiles_n * p.splits;
  const long long pairs = sms / 2 < 1 ? 1 : sms / 2;
  gemm_kernel<kAMn, kBMn, kEpi>
      <<<(unsigned)(2 * (tiles < pairs ? tiles : pairs)), kGemmThreads, kGemmSmem, stream>>>(a, b, out, p);
  return cudaGetLastError();
}
cudaError_t launch_few(const CUtensorMap& w, const CUtensorMap& h, GemmParams p, int sms, int* n_parts, cudaStream_t stream) {
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(few_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  p.tiles_n = tiles_of(p.n);
  p.chunk = 1024 / kStep;
  int pairs = sms / 2 < 1 ? 1 : sms / 2;
  if (pairs > kMaxPairs) pairs = kMaxPairs;
  if (pairs > p.tiles_n) pairs = p.tiles_n;
  *n_parts = 8 * pairs;
  few_rows_kernel<<<(unsigned)(2 * pairs), kFewThreads, kFewSmem, stream>>>(w, h, p);
  return cudaGetLastError();
}
constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kF32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;

}  // namespace

size_t entropy_workspace(int rows, int V, int K, bool backward) {
  return backward ? backward_plan(rows, V, K).bytes : forward_plan(rows, V).bytes;
}

int launch_entropy(const EntropyParams& p, int sms, void* stream) {
  const ForwardPlan f = forward_plan(p.rows, p.V);
  const cudaStream_t st = (cudaStream_t)stream;
  for (int r0 = 0; r0 < p.rows; r0 += kForwardRows) {
    EntropyParams q = p;
    q.rows = p.rows - r0 < kForwardRows ? p.rows - r0 : kForwardRows;
    q.h += 2 * r0 * p.h_stride;
    q.labels += r0;
    q.loss += r0;
    if (p.weight) q.weight += r0;
    if (p.stats) q.stats += r0;
    CUtensorMap h, w;
    if (!tc::map_2d(&h, kBf16, 2, q.h, q.rows, p.K, 2 * p.h_stride, 128) ||
        !tc::map_2d(&w, kBf16, 2, p.w, p.V, p.K, 2 * p.w_stride, 128))
      return (int)cudaErrorInvalidValue;
    GemmParams g = {};
    g.m = q.rows;
    g.n = p.V;
    g.k = p.K;
    g.splits = 1;
    g.parts = reinterpret_cast<float2*>(p.ws + f.parts);
    g.rows_pitch = f.pitch;
    g.labels = q.labels;
    g.label_logit = reinterpret_cast<float*>(p.ws + f.labels);
    g.status = p.status;
    int n_parts = f.n_parts;
    cudaError_t e;
    if (q.rows <= kFew && p.rows <= kFew) {
      CUtensorMap few;
      if (!tc::map_2d(&few, kBf16, 2, q.h, q.rows, p.K, 2 * p.h_stride, kFew / 2)) return (int)cudaErrorInvalidValue;
      e = launch_few(w, few, g, sms, &n_parts, st);
    } else {
      e = launch_gemm<false, false, kStats>(h, w, w, g, sms, st);
    }
    if (e != cudaSuccess) return (int)e;
    join_kernel<<<(unsigned)((q.rows + 31) / 32), 1024, 0, st>>>(g.parts, n_parts, f.pitch, g.label_logit, q);
    e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  return 0;
}

int launch_entropy_grad(const EntropyParams& p, int sms, void* stream) {
  const BackwardPlan b = backward_plan(p.rows, p.V, p.K);
  const cudaStream_t st = (cudaStream_t)stream;
  RowGrad* rows = reinterpret_cast<RowGrad*>(p.ws + b.rows);
  float* rest = reinterpret_cast<float*>(p.ws + b.rest);
  int32_t* used = reinterpret_cast<int32_t*>(p.ws + b.used);
  unsigned char *h_used = p.ws + b.h, *g_mem = p.ws + b.g, *sums = p.ws + b.sums;
  rows_kernel<<<(unsigned)p.rows, 128, 0, st>>>(p, rows, rest, used, p.dw ? reinterpret_cast<uint16_t*>(h_used) : nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return (int)e;
  CUtensorMap h, w, w_mn, hu, sum;
  if (!tc::map_2d(&h, kBf16, 2, p.h, p.rows, p.K, 2 * p.h_stride, 128) ||
      !tc::map_2d(&w, kBf16, 2, p.w, p.V, p.K, 2 * p.w_stride, 128) ||
      !tc::map_2d(&w_mn, kBf16, 2, p.w, p.V, p.K, 2 * p.w_stride, 64) ||
      !tc::map_2d(&hu, kBf16, 2, h_used, p.rows, p.K, 2ll * p.K, 64) ||
      !tc::map_2d(&sum, kF32, 4, sums, (long long)b.splits * b.split_rows, p.K, 4ll * p.K, 32))
    return (int)cudaErrorInvalidValue;
  for (int v0 = 0; v0 < p.V; v0 += b.piece) {
    const int width = p.V - v0 < b.piece ? p.V - v0 : b.piece;
    CUtensorMap g_out, g_k, g_mn;
    if (!tc::map_2d(&g_out, kBf16, 2, g_mem, p.rows, width, 2ll * b.pitch, 32) ||
        !tc::map_2d(&g_k, kBf16, 2, g_mem, p.rows, width, 2ll * b.pitch, 128) ||
        !tc::map_2d(&g_mn, kBf16, 2, g_mem, p.rows, width, 2ll * b.pitch, 64))
      return (int)cudaErrorInvalidValue;
    GemmParams q = {};
    q.status = p.status;
    q.splits = 1;
    q.m = p.rows;
    q.n = width;
    q.k = p.K;
    q.b_y = v0;
    q.rows = rows;
    q.label0 = v0;
    q.rest = rest;
    e = launch_gemm<false, false, kLogitGrad>(h, w, g_out, q, sms, st);
    if (e != cudaSuccess) return (int)e;
    if (p.dw) {
      CUtensorMap dw;
      if (!tc::map_2d(&dw, kBf16, 2, p.dw + 2ll * v0 * p.K, width, p.K, 2ll * p.K, 32)) return (int)cudaErrorInvalidValue;
      GemmParams d = {};
      d.status = p.status;
      d.splits = 1;
      d.m = width;
      d.n = p.K;
      d.k = p.rows;
      d.n_fast = 1;
      d.label0 = v0;
      d.rest = rest;
      d.used = used;
      d.h = p.h;
      d.h_stride = p.h_stride;
      e = launch_gemm<true, true, kStoreBf16>(g_mn, hu, dw, d, sms, st);
      if (e != cudaSuccess) return (int)e;
    }
    if (p.dh) {
      GemmParams d = {};
      d.status = p.status;
      d.splits = b.splits;
      d.m = p.rows;
      d.n = p.K;
      d.k = width;
      d.b_x = v0;
      d.add = v0 > 0;
      d.split_rows = b.split_rows;
      e = launch_gemm<false, true, kSumF32>(g_k, w_mn, sum, d, sms, st);
      if (e != cudaSuccess) return (int)e;
    }
  }
  if (p.dh) {
    const size_t n = (size_t)p.rows * p.K;
    hidden_kernel<<<(unsigned)((n / 8 + 255) / 256), 256, 0, st>>>(p, reinterpret_cast<const float*>(sums), b.splits,
                                                                  (size_t)b.split_rows * p.K, rows, rest);
    e = cudaGetLastError();
  }
  return (int)e;
}

}  // namespace dflash
