// dflash_attention_tc.cu -- attention over the paged cache for blocks whose
// query rows (new tokens x heads that share a key/value head) number more than
// 16 (8-bit caches: 32): the products run on the 5th-generation tensor cores, with
// scores, weights and sums in tensor memory.
//
// Mathematics and work list as in dflash_attention.cu; here a unit has R = 32,
// 64 or 128 query rows and a tile kKeys = 128 keys (64 for head_dim 256).
// What bounds it is still the one pass over the cache: the products take about
// 1000 of the about 2800 cycles in which a tile's 64 KB arrive, so the rows that
// pad M to 128 cost nothing. They are put to use instead: the R rows are laid
// out 128 / R times, and copy c takes the keys c kKeys R / 128 ... of every tile
// as if the others were masked. Each thread of the softmax owns one row of
// tensor memory and R / 128 of a tile's columns, which needs no exchange between
// lanes; the copies' results are joined once, at the end of the unit.
//
// Roles (one CTA per SM, persistent over its run of tiles):
//  * warps 5-8 fill a ring of stages with 16-byte asynchronous copies, placed
//    for the tensor cores' 128-byte swizzle; any page size, stride and order;
//    keys that do not exist are zero-filled. The copies arrive on the stage's
//    barrier as they land.
//  * warp 4: one thread issues S = Q K^T (both from shared memory, into one of
//    two score buffers) up to two tiles ahead of O += P V (P from tensor memory,
//    V read in place as the transposed operand).
//  * warps 0-3: softmax. A thread reads its scores (tcgen05.ld), takes 2^(x -
//    m), writes P back as 16-bit pairs. When a row's running maximum m moves,
//    its warp rescales O in tensor memory, which has to wait for the product
//    before. m may lag behind by 8 powers of 2 (weights up to 256), which spares
//    most of that: at 128 rows 152 against 178 us with a lag of 2 or 4, at
//    head_dim 256 266 against 291 us. The largest weights are then no longer
//    exactly 1 and their rounding shows: in bf16 an error of 2.2e-3 of the result
//    against 1.8e-3 with m exact (the output's rounding alone: 1.7e-3; one weight
//    ruling a row adds at most as much again in quadrature).
// A unit's end costs a CTA about kEndTiles tiles (O out of tensor memory, Q in),
// so the list of work counts it. 8-bit caches (head_dim 64 and 128) go through a
// ring of raw tiles and are widened, exactly, into the operand tiles, by 8 warps.
// Measured on one GB300, 64 query and 8 key/value heads of 128, 32 requests of up
// to 16384 positions, blocks of 8 (64 rows a head), bf16: 219 us, 5.5 TB/s of keys
// and values, 82% of a copy's rate, against 696 us by the warps' products, which
// read the cache four times there; blocks of 4 (32 rows) 197 us, 6.1 TB/s. What
// is left is the units' ends and uneven runs. At 128 rows (half the positions:
// 150 us, 4.1 TB/s, 520 TFLOP/s) and head_dim 64 (150 us, 4.0 TB/s) the softmax's
// 128 threads bound it; at head_dim 256 (266 us, 4.5 TB/s) two stages are few for
// the latency of a load; e4m3 (297 us for half the bytes) has two operand stages, and
// waits for the widening between a load and its products.
// Every wait is bounded; a CTA that gives up raises DFLASH_STATUS_TIMEOUT,
// lets its copies land and frees its tensor memory.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "dflash_attention.cuh"

namespace dflash {
namespace {

constexpr int kTcCtas = 160;
constexpr int kMmaWarp = 4;
constexpr int kLoadWarp0 = 5, kMaxLoadWarps = 8;
// A unit's end and the next one's beginning take a CTA about as long as this
// many tiles: the list counts them, so that runs with many ends are shorter.
constexpr int kEndTiles = 3;
constexpr float kSlack = 8.0f;  // by how many powers of 2 a score may exceed the one that last moved its row's reference
// Where the reference lies below that score. f16 holds normal numbers from 2^-14
// to below 2^16: with the score's weight at 2^7 the largest is 2^15, weights down
// to 2^-21 of the score's are rounded by half a step of their own, smaller ones to
// multiples of 2^-31 of it (at 2^0 they were lost from 2^-25 on). A slack of 2
// and 2^13 would be good to 2^-27 and take 178 instead of 151 us at 128 rows.
template <class T>
constexpr float kTop = std::is_same<T, F16>::value ? 7.0f : 0.0f;
constexpr int kFlags = 8;       // units whose "unsound" flag may be pending at once

template <int D, bool kF8>
struct TcShape {
  static constexpr int kLoadWarps = kF8 ? 8 : 4;  // widening takes twice the warps
  static constexpr int kThreads = 32 * (kLoadWarp0 + kLoadWarps);
  static constexpr int kKeys = D == 256 ? 64 : 128;
  static constexpr int kStages = D == 64 ? (kF8 ? 3 : 6) : D == 128 ? (kF8 ? 2 : 3) : 2;
  // 8-bit caches: tiles as they lie in the cache, in flight or waiting to be widened
  static constexpr int kRaw = !kF8 ? 0 : D == 64 ? 6 : 2;
  static constexpr int kRawBytes = kKeys * D * 2;  // K and V
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kRowBytes = kF8 ? D : 2 * D;     // a cache row
  static constexpr int kHalf = kKeys * D * 2;           // K or V of a stage
  static constexpr size_t kSmem = 1024 + (size_t)kQBytes + (size_t)kStages * 2 * kHalf + (size_t)kRaw * kRawBytes;
  // tensor memory columns
  static constexpr int kO = 0, kS = D, kP = kS + 2 * kKeys, kUsed = kP + kKeys;
  static_assert(kUsed <= 512, "tensor memory");
};

struct TcShared {  // next to the dynamic part: 227 KB in all
  uint64_t full[6], empty[6];    // per stage
  uint64_t s_full[2], p_full[2];  // per score buffer
  uint64_t pv_done[2];           // per buffer of weights
  uint64_t q_full, drained, together;
  uint32_t tmem;
  volatile int failed;
  int unsound[kFlags];           // per unit (ordinal in the CTA): values were replaced, see load
  int odd;                       // a result of the unit is not finite
  uint32_t mask[6][kMaxLoadWarps];      // per stage and load warp: its keys that exist
  uint32_t raw_mask[kMaxLoadWarps][6];  // 8-bit caches, per load warp and raw tile: the same,
  int raw_unit[kMaxLoadWarps][6];       // and its unit, with bit 0 set if some rows see less of it than others
  int first_b;
  long long first_pre, sums[kLoadWarp0 + kMaxLoadWarps];
  Part parts[128];
};

static_assert(TcShape<128, false>::kSmem + sizeof(TcShared) <= 232448 && TcShape<128, true>::kSmem <= TcShape<128, false>::kSmem,
              "one CTA's shared memory (227 KB)");

// ---- PTX wrappers (one CTA per tensor core group) ------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// D (+)= A[shared memory] B[shared memory]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// D (+)= A[tensor memory] B[shared memory]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 16 bytes to shared memory as they arrive; zeros where there is nothing to read
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
// waits for the loads issued so far; the values pass through, so that nothing
// computed from them moves ahead of the wait
__device__ __forceinline__ void wait_ld8(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// N consecutive columns of this thread's lane, 8 at a time
__device__ __forceinline__ void ld8(uint32_t a, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
__device__ __forceinline__ void ld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void st8(uint32_t a, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void st32(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t a, uint32_t (&r)[N]) {
  if constexpr (N % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 32) ld32(a + i, r + i);
#pragma unroll
    for (int i = 0; i < N; i += 32) wait_ld32(r + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 8) ld8(a + i, r + i);
#pragma unroll
    for (int i = 0; i < N; i += 8) wait_ld8(r + i);
  }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t a, const uint32_t (&r)[N]) {
  if constexpr (N % 32 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 32) st32(a + i, r + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 8) st8(a + i, r + i);
  }
}

// Shared-memory operand descriptor, 128-byte swizzle. K-major (Q, K): rows of
// 128 bytes, 8-row groups 1024 bytes apart (stride offset); one product's 16
// inner values lie inside a row. MN-major (V, whose rows are the inner index):
// 64 outer values per 128-byte row, 8 inner rows per group 1024 bytes apart
// (stride offset), the next 64 outer values a slab further (leading offset).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t leading) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)((leading & 0x3ffffu) >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

// A bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, TcShared& S) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0u && (S.failed || global_timer_ns() - t0 > kWaitLimitNs)) {
      S.failed = 1;
      return false;
    }
  }
}
// The same for a warp: its lanes go on together or give up together, since what
// follows are shuffles and votes of the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, TcShared& S) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, S));
}
// A barrier of the 128 softmax threads whose wait is bounded like the others
// (a hardware barrier would hang if one warp had given up).
__device__ __forceinline__ bool softmax_sync(uint32_t& phase, TcShared& S) {
  mbar_arrive(&S.together);
  const bool ok = tc_wait(&S.together, phase & 1u, S);
  ++phase;
  return __all_sync(0xffffffffu, ok);
}

// A position in the list of units. A unit takes tiles + kEndTiles places; the
// tiles come first.
template <int R, int kKeys>
struct Cursor {
  int b, h, rb, L, first, n, tiles, rbs, ordinal;
  long long start;
  __device__ __forceinline__ void request(const AttnParams& p) {
    bool bad = false;
    request_tokens(p.tk, b, first, n, bad);
    L = clamped_len(p, b, bad);
    tiles = tiles_of<kKeys>(L);
    rbs = row_blocks<R>(n, p.G);
  }
  // The first tile at place t or after it, before t_end (t_end: there is none);
  // request b0 is the one t falls in, pre the places before that.
  __device__ __forceinline__ long long seek(const AttnParams& p, int b0, long long pre, long long t, long long t_end) {
    b = b0;
    request(p);
    const long long k = (t - pre) / (tiles + kEndTiles);
    h = (int)(k / rbs);
    rb = (int)(k - (long long)h * rbs);
    start = pre + k * (tiles + kEndTiles);
    ordinal = 0;
    return t < start + tiles ? t : next(p, t_end);
  }
  __device__ __forceinline__ long long end(long long t_end) const { return min(t_end, start + tiles); }
  // Moves to the next unit and returns its first tile, or t_end.
  __device__ __forceinline__ long long next(const AttnParams& p, long long t_end) {
    if (start + tiles + kEndTiles >= t_end) return t_end;
    start += tiles + kEndTiles;
    ++ordinal;
    if (++rb < rbs) return start;
    rb = 0;
    if (++h < p.c.kv_heads) return start;
    h = 0;
    do {
      ++b;
      request(p);
    } while (rbs == 0);  // (the list goes on, so there is one)
    return start;
  }
  // The tile after t, or t_end.
  __device__ __forceinline__ long long step(const AttnParams& p, long long t, long long t_end) {
    return t + 1 < start + tiles ? min(t + 1, t_end) : next(p, t_end);
  }
};

// 8 e4m3 values (two words) as 8 values of T, exactly
template <class T>
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
  uint32_t w[4];
  widen4(a, w[0], w[1]);
  widen4(b, w[2], w[3]);
  if constexpr (std::is_same<T, Bf16>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = F16::unpack(w[i]);
      w[i] = Bf16::pack(f.x, f.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T, bool kF8, int D, int R>
__global__ void __launch_bounds__(TcShape<D, kF8>::kThreads, 1) attention_tc_kernel(const AttnParams p, const AttnGeometry geo) {
  using W = TcShape<D, kF8>;
  constexpr int kKeys = W::kKeys, kStages = W::kStages;
  constexpr int kCopies = 128 / R, kCols = kKeys / kCopies;  // a thread's columns of a tile
  constexpr int kChunk = kCols < 64 ? kCols : 64;            // ... in registers at a time
  constexpr int kLoadWarps = W::kLoadWarps, kTcThreads = W::kThreads;
  constexpr int kMine = kKeys / kLoadWarps;                  // a load warp's keys of a tile
  constexpr int kGroup = kChunk < kMine ? kChunk : kMine;
  constexpr uint32_t kMineMask = kMine == 32 ? 0xffffffffu : (1u << kMine) - 1u;
  extern __shared__ unsigned char raw[];
  __shared__ TcShared S;
  unsigned char* mem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_mem = smem_addr(mem), ring = q_mem + W::kQBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&S.full[i], kLoadWarps * (kF8 ? 32 : 33));  // every loading thread, and each warp's mask
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 128);
      mbar_init(&S.pv_done[i], 1);
    }
    mbar_init(&S.q_full, 128);
    mbar_init(&S.drained, 1);
    mbar_init(&S.together, 128);
    for (int i = 0; i < kFlags; ++i) S.unsound[i] = 0;
    S.odd = 0;
    S.failed = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&S.tmem, 512);
  grid_dependency_sync();

  // ---- the list: tiles before each request, this CTA's run and its first request
  bool bad = false;
  long long mine = 0, before = 0, total = 0;
  const int per = (p.tk.B + kTcThreads - 1) / kTcThreads;
  const int b_lo = min(p.tk.B, tid * per), b_hi = min(p.tk.B, b_lo + per);
  auto request_tiles = [&](int b) {
    int first, n;
    request_tokens(p.tk, b, first, n, bad);
    return (long long)row_blocks<R>(n, p.G) * p.c.kv_heads * (tiles_of<kKeys>(clamped_len(p, b, bad)) + kEndTiles);
  };
  for (int b = b_lo; b < b_hi; ++b) mine += request_tiles(b);
  before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) S.sums[warp] = before;
  before -= mine;
  __syncthreads();
  for (int w = 0; w < kTcThreads / 32; ++w) {
    if (w < warp) before += S.sums[w];
    total += S.sums[w];
  }
  const long long run = max((long long)kMinRun, (total + gridDim.x - 1) / gridDim.x);
  const long long t_begin = (long long)blockIdx.x * run, t_end = min(total, t_begin + run);
  if (blockIdx.x == 0) {
    if (tid == 0) *reinterpret_cast<long long*>(p.ws) = run;
    if (bad) raise_status(p.status, DFLASH_STATUS_BAD_LENGTH);
  }
  if (t_begin < t_end && before <= t_begin && t_begin < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = request_tiles(b);
      if (t_begin < at + n) {
        S.first_b = b;
        S.first_pre = at;
        break;
      }
      at += n;
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S.tmem;

  SplitUnit split = {0, 0, 0, 0, 0, 0, 0};
  if (t_begin < t_end) {
    Cursor<R, kKeys> u;
    const long long t_first = u.seek(p, S.first_b, S.first_pre, t_begin, t_end);
    bool ok = true;

    if (warp >= kLoadWarp0) {
      // ---- loads: this warp's share of every tile's keys
      constexpr int kPieces = W::kRowBytes / 16;     // 16-byte pieces of a row in the cache
      constexpr int kLoads = kMine * kPieces / 32;   // per lane, for K and for V each
      const int lw = warp - kLoadWarp0;
      // The page index of a tile's keys is asked for two tiles ahead: lane l
      // looks after key l of the warp's share.
      struct Ahead {
        long long t;    // the tile (t_end: none)
        int id, slot, head, unit;  // unit: its ordinal twice, plus 1 where some rows see less of the tile than others
        bool there;
      };
      bool bad_page = false;
      auto ask = [&](long long t) {
        Ahead a = {t, 0, 0, 0, 0, false};
        if (t < t_end) {
          const int key = (int)(t - u.start) * kKeys + lw * kMine + (lane & (kMine - 1));
          a.there = key < u.L;
          a.head = u.h;
          a.unit = 2 * u.ordinal + (p.causal && u.n > 1 && (t - u.start + 1) * kKeys > u.L - u.n ? 1 : 0);
          if (a.there) {
            int page;
            split_position(p.c, key, page, a.slot);
            a.id = p.c.table[(long long)u.b * p.c.table_stride + page];
          }
        }
        return a;
      };
      // the row's place, once the index is here
      auto place = [&](Ahead& a) {
        if (a.there && (a.id < 0 || a.id >= p.c.num_pages)) {
          bad_page = true;
          a.there = false;
        }
        return a.there ? row_offset(p.c, a.id, a.head, a.slot) : 0u;
      };
      Ahead now = ask(t_first), next = now;
      if (t_first < t_end) next = ask(u.step(p, t_first, t_end));
      auto move_on = [&]() {
        now = next;
        if (next.t < t_end) next = ask(u.step(p, next.t, t_end));
      };
      // Under a causal mask a tile may hold values that only some rows see:
      // those that are not finite are replaced by 0 here, and the unit's end is
      // told.
      [[maybe_unused]] auto sanitise = [&](int st, int ordinal) {
        const uint32_t vb = (uint32_t)(W::kQBytes + st * 2 * W::kHalf + W::kHalf);
        bool found = false;
#pragma unroll 4
        for (int i = 0; i < kLoads; ++i) {
          const int at = i * 32 + lane, r = lw * kMine + at / kPieces, c = at % kPieces;
          uint32_t* w = reinterpret_cast<uint32_t*>(mem + vb + (c >> 3) * (kKeys * 128) + r * 128 +
                                                    (((c & 7) ^ (r & 7)) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x = w[e];
            if (drop_not_finite<T, false>(x)) {
              w[e] = x;
              found = true;
            }
          }
        }
        if (found) S.unsound[ordinal % kFlags] = 1;
      };
      int st = 0;
      uint32_t round = 0;
      if constexpr (!kF8) {
        while (now.t < t_end) {
          const uint32_t next_off = place(now), mask = __ballot_sync(0xffffffffu, now.there);
          if (round > 0 && !(ok = warp_wait(&S.empty[st], (round - 1) & 1u, S))) break;
          __syncwarp();
          const uint32_t kb = ring + st * 2 * W::kHalf;
#pragma unroll
          for (int i = 0; i < kLoads; ++i) {
            const int at = i * 32 + lane, r = at / kPieces, c = at % kPieces;
            const uint32_t off = __shfl_sync(0xffffffffu, next_off, r);
            const size_t o = ((size_t)off + c) * 16u;
            const int row = lw * kMine + r;
            const uint32_t d = kb + (c >> 3) * (kKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
            const bool there = (mask >> r) & 1u;
            copy16(d, p.c.k + o, there);
            copy16(d + W::kHalf, p.c.v + o, there);
          }
          if (lane == 0) {
            S.mask[st][lw] = mask;
            mbar_arrive(&S.full[st]);
          }
          if (now.unit & 1) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            sanitise(st, now.unit >> 1);
            mbar_arrive(&S.full[st]);
          } else {
            // arrives by itself once this thread's copies have landed
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&S.full[st]))
                         : "memory");
          }
          move_on();
          if (++st == kStages) {
            st = 0;
            ++round;
          }
        }
      } else {
        // 8-bit caches: a thread copies its pieces as they are into a ring of
        // its own, kRaw tiles deep, and widens them into the tile's stage
        constexpr int kRaw = W::kRaw;
        unsigned char* mine = mem + W::kQBytes + kStages * 2 * W::kHalf + lw * (W::kRawBytes / kLoadWarps) + lane * 16;
        int slot = 0, issued = 0, done = 0, from = 0;
        auto issue = [&]() {
          if (now.t < t_end) {
            const uint32_t next_off = place(now), mask = __ballot_sync(0xffffffffu, now.there);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
              const int at = i * 32 + lane, r = at / kPieces, c = at % kPieces;
              const uint32_t off = __shfl_sync(0xffffffffu, next_off, r);
              const size_t o = ((size_t)off + c) * 16u;
              const bool there = (mask >> r) & 1u;
              const uint32_t d = smem_addr(mine + slot * W::kRawBytes + i * 512);
              copy16(d, p.c.k + o, there);
              copy16(d + kLoads * 512, p.c.v + o, there);
            }
            if (lane == 0) {
              S.raw_mask[lw][slot] = mask;
              S.raw_unit[lw][slot] = now.unit;
            }
            ++issued;
            move_on();
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          slot = slot + 1 == kRaw ? 0 : slot + 1;
        };
        for (int i = 0; i < kRaw - 1; ++i) issue();
        for (;;) {
          issue();
          if (done == issued) break;
          asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 1) : "memory");
          __syncwarp();
          const uint32_t mask = S.raw_mask[lw][from];
          const int unit = S.raw_unit[lw][from];
          if (round > 0 && !(ok = warp_wait(&S.empty[st], (round - 1) & 1u, S))) break;
          unsigned char* kb = mem + W::kQBytes + st * 2 * W::kHalf;
          bool found = false;
#pragma unroll 4
          for (int i = 0; i < 2 * kLoads; ++i) {
            uint4 w = *reinterpret_cast<const uint4*>(mine + from * W::kRawBytes + i * 512);
            const bool is_v = i >= kLoads;
            const int at = (is_v ? i - kLoads : i) * 32 + lane, row = lw * kMine + at / kPieces, c = 2 * (at % kPieces);
            if (is_v && (unit & 1)) {
              found |= drop_not_finite<T, true>(w.x);
              found |= drop_not_finite<T, true>(w.y);
              found |= drop_not_finite<T, true>(w.z);
              found |= drop_not_finite<T, true>(w.w);
            }
            unsigned char* d = kb + (is_v ? W::kHalf : 0) + (c >> 3) * (kKeys * 128) + row * 128;
            *reinterpret_cast<uint4*>(d + (((c & 7) ^ (row & 7)) << 4)) = widen8<T>(w.x, w.y);
            *reinterpret_cast<uint4*>(d + ((((c + 1) & 7) ^ (row & 7)) << 4)) = widen8<T>(w.z, w.w);
          }
          if (found) S.unsound[(unit >> 1) % kFlags] = 1;
          if (lane == 0) S.mask[st][lw] = mask;
          fence_async_smem();
          mbar_arrive(&S.full[st]);
          ++done;
          from = from + 1 == kRaw ? 0 : from + 1;
          if (++st == kStages) {
            st = 0;
            ++round;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (bad_page) raise_status(p.status, DFLASH_STATUS_BAD_PAGE);
    } else if (warp == kMmaWarp) {
      // ---- products
      if (lane == 0) {
        constexpr uint32_t type = std::is_same<T, Bf16>::value ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t id_s = (1u << 4) | type | ((uint32_t)(kKeys >> 3) << 17) | (8u << 24);
        constexpr uint32_t id_o = (1u << 4) | type | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
        int j0 = 0, units = 0;  // tiles before this unit's, units begun
        for (long long t = t_first; t < t_end && ok;) {
          const int n = (int)(u.end(t_end) - t);  // the unit's tiles here
          // tile j0 + i has landed
          auto landed = [&](int i) { return mbar_test_wait(&S.full[(j0 + i) % kStages], (uint32_t)((j0 + i) / kStages) & 1u); };
          // S = Q K^T of tile j0 + i, which has landed
          auto scores = [&](int i) {
            const int j = j0 + i;
            fence_async_smem();  // the copies, which the barrier has shown, before the asynchronous proxy reads them
            fence_after();
            const uint32_t kb = ring + (j % kStages) * 2 * W::kHalf;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tmem + W::kS + (j & 1) * kKeys, operand(q_mem + (k >> 2) * 16384 + (k & 3) * 32, 16),
                     operand(kb + (k >> 2) * (kKeys * 128) + (k & 3) * 32, 16), id_s, k > 0);
            mma_commit(&S.s_full[j & 1]);
          };
          ok = tc_wait(&S.q_full, (uint32_t)units & 1u, S);
          ++units;
          int issued = 0;  // scores
          for (int i = 0; i < n && ok; ++i) {
            const int j = j0 + i, st = j % kStages, buf = j & 1;
            if (issued == i) {
              if (!(ok = tc_wait(&S.full[st], (uint32_t)(j / kStages) & 1u, S))) break;
              scores(issued++);
            }
            if (issued == i + 1 && i + 1 < n && landed(i + 1)) scores(issued++);
            if (!(ok = tc_wait(&S.p_full[buf], (uint32_t)(j >> 1) & 1u, S))) break;
            // The tile's scores have been read: the next but one's go first, so
            // that the softmax never waits for the product with V.
            while (issued <= i + 2 && issued < n && landed(issued)) scores(issued++);
            fence_after();
            const uint32_t vb = ring + st * 2 * W::kHalf + W::kHalf;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(tmem + W::kO, tmem + W::kP + buf * (kKeys / 2) + 8 * k, operand(vb + k * 2048, kKeys * 128), id_o,
                     i > 0 || k > 0);
            mma_commit(&S.empty[st]);
            mma_commit(&S.pv_done[buf]);
          }
          j0 += n;
          t = u.next(p, t_end);
        }
        mma_commit(&S.drained);  // nothing is left in flight when the tensor memory is freed
        mbar_wait_landed(&S.drained, 0);
      }
      __syncwarp();
    } else {
      // ---- softmax: this thread's row of tensor memory
      const uint32_t my = tmem + ((uint32_t)(warp * 32) << 16);
      const int copy = tid / R, row = tid % R;
      {
        uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kKeys; i += 8) st8(my + W::kP + i, zero);  // both buffers: the other copies' keys stay 0
        wait_st();
      }
      float c = p.scale * kLog2e;
      [[maybe_unused]] bool flip = false, flat = false;  // 8-bit caches: a negative, a zero scale of K
      float* scratch = reinterpret_cast<float*>(mem);  // Q's place, between units
      int j = 0;  // tiles before this one
      uint32_t syncs = 0;
      // P V of tile j is done. A parity names one of two phases: this thread has
      // waited for tile j - 2's, and tile j + 2's waits for this thread.
      auto product_done = [&](int j) { return tc_wait(&S.pv_done[j & 1], (uint32_t)(j >> 1) & 1u, S); };
      long long t = t_first;
      while (t < t_end && ok) {
        const long long u_end = u.end(t_end), u_begin = t;
        // ---- Q, laid out kCopies times
        const int rows_here = min(R, u.n * p.G - u.rb * R);
        constexpr int kPieces = D / 8;
#pragma unroll
        for (int i = 0; i < R * kPieces / 128; ++i) {
          const int at = i * 128 + tid, qr = at / kPieces, cc = at % kPieces;
          const bool there = qr < rows_here;
          const int g = u.rb * R + (there ? qr : 0), ti = g / p.G;
          const unsigned char* src = p.q + 2 * ((long long)(u.first + ti) * p.q_ts +
                                                (long long)(u.h * p.G + g - ti * p.G) * p.q_hs + 8 * cc);
#pragma unroll
          for (int k = 0; k < kCopies; ++k) {
            const int rr = k * R + qr;
            copy16(q_mem + (cc >> 3) * 16384 + rr * 128 + (((cc & 7) ^ (rr & 7)) << 4), src, there);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (kF8) {
          // the comparison of scores is on unscaled ones: their factor is made positive
          c = p.scale * kLog2e * (p.c.k_scale ? p.c.k_scale[u.h] : 1.0f);
          flip = c < 0.0f;
          flat = c == 0.0f;
          c = flat ? 1.0f : fabsf(c);
        }
        fence_async_smem();
        mbar_arrive(&S.q_full);
        const int tok = (u.rb * R + row) / p.G;
        const int vis = row >= rows_here ? 0 : p.causal ? min(u.L, max(0, u.L - u.n + tok + 1)) : u.L;

        float m = kNegInf, l = 0.0f;
        for (; t < u_end && ok; ++t, ++j) {
          const int st = j % kStages, buf = j & 1;
          ok = tc_wait(&S.s_full[buf], (uint32_t)(j >> 1) & 1u, S);
          ok = ok && tc_wait(&S.full[st], (uint32_t)(j / kStages) & 1u, S);  // for the mask
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t scores = my + W::kS + buf * kKeys + copy * kCols;
          const int key0 = (int)(t - u.start) * kKeys + copy * kCols;
          uint32_t all = S.mask[st][0];
#pragma unroll
          for (int w = 1; w < kLoadWarps; ++w) all &= S.mask[st][w];
          const bool whole_tile = (int)(t - u.start + 1) * kKeys <= u.L - (p.causal ? u.n : 0) &&
                                  (all & kMineMask) == kMineMask;
          // scores of the columns from c0 on, unscaled, -inf where masked
          auto read = [&](int c0, uint32_t (&x)[kChunk]) {
            tmem_load<kChunk>(scores + c0, x);
            if constexpr (kF8) {
              if (flip || flat)
#pragma unroll
                for (int i = 0; i < kChunk; ++i) x[i] = flat ? 0u : x[i] ^ 0x80000000u;
            }
            if (whole_tile) return;
#pragma unroll
            for (int g = 0; g < kChunk; g += kGroup) {
              const int k = copy * kCols + c0 + g;
              // bit i: the key of column g + i is there and before `vis`
              const int left = vis - (key0 + c0 + g);
              const uint32_t before = left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1u;
              const uint32_t seen = (S.mask[st][k / kMine] >> (k % kMine)) & before;
#pragma unroll
              for (int i = 0; i < kGroup; ++i)
                if (!((seen >> i) & 1u)) x[g + i] = __float_as_uint(kNegInf);
            }
          };
          uint32_t x[kChunk];
          float top = kNegInf;
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += kChunk) {
            read(c0, x);
#pragma unroll
            for (int i = 0; i < kChunk; ++i) top = fmaxf(top, __uint_as_float(x[i]));
          }
          top = fmaf(top, c, -kTop<T>);
          const bool move = top > m + kSlack || (m == kNegInf && top > m);
          if (__any_sync(0xffffffffu, move)) {
            const float f = move ? (m == kNegInf ? 0.0f : ex2(m - top)) : 1.0f;
            if (t > u_begin) {
              // O holds sums: they are rescaled, after the last product
              ok = product_done(j - 1);
              if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
              }
              fence_after();
              for (int d = 0; d < D; d += 32) {
                uint32_t y[32];
                tmem_load<32>(my + W::kO + d, y);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                tmem_store<32>(my + W::kO + d, y);
              }
              wait_st();
            }
            l *= f;
            if (move) m = top;
          }
          const float ref = m == kNegInf ? 0.0f : m;
          if (j > 1) ok = product_done(j - 2);  // which read this buffer of weights
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += kChunk) {
            if (kCols > kChunk) read(c0, x);  // again: not all of a row's scores fit in registers
            uint32_t w[kChunk / 2];
#pragma unroll
            for (int i = 0; i < kChunk / 2; ++i) {
              const float a = ex2(fmaf(__uint_as_float(x[2 * i]), c, -ref)),
                          b = ex2(fmaf(__uint_as_float(x[2 * i + 1]), c, -ref));
              l += a + b;
              w[i] = T::pack(a, b);
            }
            tmem_store<kChunk / 2>(my + W::kP + buf * (kKeys / 2) + (copy * kCols + c0) / 2, w);
          }
          wait_st();
          fence_before();
          mbar_arrive(&S.p_full[buf]);
        }
        if (!ok) break;

        // ---- the unit (or this CTA's run of it) ends
        ok = product_done(j - 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        fence_after();
        const bool whole = u_begin == u.start && u_end == u.start + u.tiles;
        S.parts[tid] = {m, l};
        const int unsound = *reinterpret_cast<volatile int*>(&S.unsound[u.ordinal % kFlags]);
        if (!(ok = softmax_sync(syncs, S))) break;
        // the row's maximum and sum over its copies, and this copy's factor
        float best = kNegInf, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) best = fmaxf(best, S.parts[k * R + row].m);
#pragma unroll
        for (int k = 0; k < kCopies; ++k) sum += part_sum(S.parts[k * R + row], best);
        float factor = m == kNegInf ? 0.0f : ex2(m - best);
        if (whole) {
          factor *= reciprocal_or_zero(sum);
          if (kF8 && p.c.v_scale) factor *= p.c.v_scale[u.h];
        }
        const long long slot = 2LL * blockIdx.x + (u_begin == t_begin ? 0 : 1);
        const int g = u.rb * R + row, ti = g / p.G;
        const long long q_tok = u.first + ti, q_head = u.h * p.G + g - ti * p.G;
        const bool writes = copy == 0 && row < rows_here;  // the first copy's thread writes the row
        unsigned char* out_row = p.out + 2 * (q_tok * p.o_ts + q_head * p.o_hs);
        float* part_row = reinterpret_cast<float*>(p.ws + geo.o()) + (slot * R + row) * D;
        if (writes) {
          if (!whole) {
            reinterpret_cast<Part*>(p.ws + geo.ml())[slot * R + row] = {best, sum};
          } else if (p.lse) {
            p.lse[q_tok * ((long long)p.G * p.c.kv_heads) + q_head] = (best + log2f(sum)) * kLn2;
          }
        }
        // The other copies leave their rows in shared memory (Q's place: as many
        // columns at a time as it holds), the first adds them to its own. Pieces
        // of 16 bytes are exchanged within 8 so that 8 lanes meet 8 bank groups.
        constexpr int kRound = kCopies == 4 ? D / 2 : D;
        float probe = 0.0f;  // NaN once a result is not finite
        for (int r0 = 0; r0 < D && ok; r0 += kRound) {
          if (kCopies > 1) {
            if (copy > 0) {
              float4* dst = reinterpret_cast<float4*>(scratch) + (size_t)(tid - R) * (kRound / 4);
#pragma unroll 1
              for (int d = 0; d < kRound; d += 32) {
                uint32_t y[32];
                tmem_load<32>(my + W::kO + r0 + d, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  dst[d / 4 + (i ^ (lane & 7))] =
                      make_float4(__uint_as_float(y[4 * i]) * factor, __uint_as_float(y[4 * i + 1]) * factor,
                                  __uint_as_float(y[4 * i + 2]) * factor, __uint_as_float(y[4 * i + 3]) * factor);
              }
            }
            if (!(ok = softmax_sync(syncs, S))) break;
          }
          if (copy == 0) {
#pragma unroll 1
            for (int d = 0; d < kRound; d += 32) {
              uint32_t y[32];
              __syncwarp();
              tmem_load<32>(my + W::kO + r0 + d, y);
              float x[32];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float4 o = make_float4(__uint_as_float(y[4 * i]) * factor, __uint_as_float(y[4 * i + 1]) * factor,
                                       __uint_as_float(y[4 * i + 2]) * factor, __uint_as_float(y[4 * i + 3]) * factor);
#pragma unroll
                for (int k = 1; k < kCopies; ++k) {
                  const float4 e = reinterpret_cast<const float4*>(scratch)[(size_t)((k - 1) * R + row) * (kRound / 4) +
                                                                            d / 4 + (i ^ (lane & 7))];
                  o = make_float4(o.x + e.x, o.y + e.y, o.z + e.z, o.w + e.w);
                }
                x[4 * i] = o.x;
                x[4 * i + 1] = o.y;
                x[4 * i + 2] = o.z;
                x[4 * i + 3] = o.w;
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) probe = fmaf(x[i], 0.0f, probe);
              if (writes) {
                if (whole) {
                  uint4* dst = reinterpret_cast<uint4*>(out_row + 2 * (r0 + d));
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(T::pack(x[8 * i], x[8 * i + 1]), T::pack(x[8 * i + 2], x[8 * i + 3]),
                                        T::pack(x[8 * i + 4], x[8 * i + 5]), T::pack(x[8 * i + 6], x[8 * i + 7]));
                } else {
                  float4* dst = reinterpret_cast<float4*>(part_row + r0 + d);
#pragma unroll
                  for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
              }
            }
          }
          // (a row whose sum of weights is not finite has NaN everywhere)
          if (writes && probe != 0.0f && sum < INFINITY) S.odd = 1;
          // the scratch, Q and S.parts are written again
          ok = softmax_sync(syncs, S);
        }
        if (!ok) break;
        if (__builtin_expect(unsound || *reinterpret_cast<volatile int*>(&S.odd), 0)) {
          // results that values which are not finite decide
          int* first = reinterpret_cast<int*>(scratch);
          for (int i = tid; i < 3 * D; i += 128) first[i] = kNever;
          if (!(ok = softmax_sync(syncs, S))) break;
          find_not_finite<T, kF8, D>(p, u.b, u.h, (int)(u_begin - u.start) * kKeys,
                                     (int)min((long long)u.L, (u_end - u.start) * kKeys), first, tid, 128);
          if (!(ok = softmax_sync(syncs, S))) break;
          if (tid == 0) S.odd = 0;
          if (writes && sum < INFINITY) {
            for (int d = 0; d < D; ++d) {
              const float v = not_finite_value<D>(first, d, vis);
              if (v == 0.0f) continue;
              if (whole)
                reinterpret_cast<uint16_t*>(out_row)[d] = (uint16_t)T::pack(v, 0.0f);
              else
                part_row[d] = v;
            }
          }
          if (!(ok = softmax_sync(syncs, S))) break;
        }
        if (tid == 0) S.unsound[u.ordinal % kFlags] = 0;
        fence_before();
        if (u_begin == u.start && !whole) split = {u.start, u.tiles, u.h, u.rb, u.first, u.n, 0};
        t = u.next(p, t_end);
      }
    }
    if (!ok && lane == 0) raise_status(p.status, DFLASH_STATUS_TIMEOUT);
  }
  if (tid == 0) split_units(p)[blockIdx.x] = split;
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

template <class T, bool kF8, int D, int R>
int launch(const AttnParams& p, int sms, void* stream) {
  using W = TcShape<D, kF8>;
  const AttnGeometry geo = tc_geometry(R, D);
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return (int)e;
  if (dev < 0 || dev >= 64) return (int)cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(attention_tc_kernel<T, kF8, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)W::kSmem);
    if (e != cudaSuccess) return (int)e;
    ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = (cudaStream_t)stream;
  const int grid = sms < kTcCtas ? sms : kTcCtas;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(W::kThreads);
  cfg.dynamicSmemBytes = W::kSmem;
  e = cudaLaunchKernelEx(&cfg, attention_tc_kernel<T, kF8, D, R>, p, geo);
  if (e != cudaSuccess) return (int)e;
  return launch_join(p, geo, grid, std::is_same<T, Bf16>::value ? DFLASH_BF16 : DFLASH_F16, kF8, D, stream);
}
template <class T, int R>
int pick(const AttnParams& p, bool f8, int d, int sms, void* stream) {
  if (f8) return d == 64 ? launch<T, true, 64, R>(p, sms, stream) : launch<T, true, 128, R>(p, sms, stream);
  return d == 64    ? launch<T, false, 64, R>(p, sms, stream)
         : d == 128 ? launch<T, false, 128, R>(p, sms, stream)
                    : launch<T, false, 256, R>(p, sms, stream);
}

}  // namespace

AttnGeometry tc_geometry(int rows, int head_dim) { return {rows, head_dim == 256 ? 64 : 128, kTcCtas}; }

int launch_attention_tc(const AttnParams& p, int rows, int dtype, bool f8, int head_dim, int sms, void* stream) {
  if (dtype == DFLASH_BF16)
    return rows == 32   ? pick<Bf16, 32>(p, f8, head_dim, sms, stream)
           : rows == 64 ? pick<Bf16, 64>(p, f8, head_dim, sms, stream)
                        : pick<Bf16, 128>(p, f8, head_dim, sms, stream);
  return rows == 32   ? pick<F16, 32>(p, f8, head_dim, sms, stream)
         : rows == 64 ? pick<F16, 64>(p, f8, head_dim, sms, stream)
                      : pick<F16, 128>(p, f8, head_dim, sms, stream);
}

}  // namespace dflash
