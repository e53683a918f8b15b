// Attention over the 8-bit paged cache on the tensor cores (see q8_attn.cuh for
// what is computed and how the work is split).
//
// The cached codes go from TMA straight into tcgen05.mma: nothing converts them.
// Both products are taken with the cache as the M operand, so that the few
// query rows of a verification step fill the small N side:
//   S^T [128 keys x NO]    = K  [128 x D]   * (Qhi + Qlo)^T       e4m3 x e4m3
//   O^T [D x NO]          += V^T [D x 128]  * (P0 + P1 + P2)^T    e4m3 x e5m2
// K is read along D, V along its other side (D is contiguous), both through the
// swizzle that TMA wrote. A block scale belongs to a key, that is to a TMEM lane
// of S^T, so scaling costs one product for K's and is folded into the
// probabilities for V's.
//   Queries: each row is scaled by a power of two to [128, 256) and split into two
// e4m3 terms (4 + 4 bits: a bf16 number exactly, down to 2^-9 of the row's
// largest). Probabilities: p is rounded to 9 bits (2^-9 relative) and split
// into three e5m2 terms of at most 3 bits, exactly; e5m2 is the upper byte of
// fp16, so a term is a byte of the fp16 number and the rest one subtraction.
// 9 bits leave the bf16 output's own rounding the larger error. e5m2's smallest step
// is 2^-24 of the row's reference (in what a key contributes, probability times V scale),
// and the terms cut below it. So that many small keys do not lose in one direction,
// each has a number between 0 and a step added first, by turns of its position: a key is
// off by less than a step, and N of them by about half a step times sqrt(N), while the
// denominator takes p in fp32. Rounding to nearest instead would drop every key under
// half a step: 2^-8 of the row's weight for 131072 of them; a finer step takes a smaller
// distance by which keys may exceed the reference, and moving it more often: steps of 2^-27
// cost 1 to 9 % (48 query rows 290 to 317 us, 20 rows 206 to 210).
//   Softmax: a row's reference m is the largest z_j + log2(V scale of j) (rounded up
// to a binade) of the first tile, and is only moved when a later one exceeds it by
// 7.75: then O and l are rescaled once; otherwise a tile costs no reduction over its
// keys. l stays per thread (one key of every tile) until the item ends.
//
// Roles: one or two groups of 4 softmax warps (thread = key of the tile, each group
// its own query rows), two copy warps, an MMA warp and a warp that prepares the next
// item's queries. K and V tiles share one ring of slots, released separately. Two
// CTAs per SM hide each other's latencies.
//
// Bound by memory up to 24 query rows of a kv head: 256 rows of 512-4096 tokens, 8 kv
// heads x 128, 20 query rows, 1.23 GB: 207 us = 6.0 TB/s (0.88 of the copy peak); 8 rows
// 200 us; 2 rows of 100-131 thousand tokens 84 us (5.6 TB/s). With D = 64 and beyond that
// by the softmax warps' instructions (about 12 for each 32 scores): D = 64 174 us
// (3.6 TB/s), 32 rows 222 us, 48 rows 293 us, 64 rows 376 us; a window of 4096 over 56 rows
// 134 us (3.1 TB/s). Short rows (100-600 tokens) by the changes of items: 82 us, 48 query
// rows 125 us (94 and 166 before the queries were prepared two items ahead and in fewer
// steps). The steps that mattered:
// the hot loop must stay small (waits out of line, one copy of each block of code:
// 334 to 242 us for the 20-row case), the copies of 16-token blocks need two warps,
// an item's queries must be converted before it begins (230 to 206 us), an item's end
// reads its shared memory before its first store (3 us), and nothing may go
// through local memory, which this much shared memory pushes out to L2.
// Not kept, for the 20-row case: two groups taking the tiles in turn (374 us), three
// CTAs per SM with short rings (351 us), tiles called into L2 ahead of the copies
// (281 us), the copies' coordinates made uniform by shuffles (316 us); for many rows,
// exponentials taken before the references are tested (177 instead of 139 us: spills).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8_attn.cuh"
#include "tc.cuh"

namespace sv {

constexpr int kTcScaleRing = 8;             // tiles whose scales are held
constexpr int kTcItems = 3;                 // items whose rows are described at a time
constexpr int kTcMaxPages = 16;             // blocks of one tile
constexpr float kTcUnset = 1e30f;           // minus the reference of a row that has seen no key
constexpr float kTcSlack = 7.75f;           // binades by which keys may exceed the reference
constexpr float kTcLift = 256.0f;           // 1 enters as 2^8: 2^8 2^7.75 < 1.75 2^15, e5m2's largest
// V scales are 2^-100 to 2^120 and enter as half of it: with the lift they stay below 2^128,
// and a row's sum, whose probabilities go up to 2^7.75 over the V scale, too.
constexpr float kTcVDown = 0.5f;
constexpr float kTcMaxSum = 0x1.fffffep126f;
constexpr int kTcSmem = 113 * 1024 - 512;   // of one CTA, two per SM

struct TcGuard {
  uint64_t limit_ns;  // of a wait
  int abort;          // one has run out
  __device__ __forceinline__ bool aborted() const {
    return *reinterpret_cast<const volatile int*>(&abort) != 0;
  }
};

template <int NR>
struct TcShared {
  alignas(16) float row_c[kTcItems][NR];  // query row's scale * softmax_scale * log2(e)
  alignas(16) float row_nm[NR];     // minus the reference of the exponentials
  alignas(16) float row_a[NR];      // root of the rescale factor, then the output's factor
  alignas(16) float part[4][NR];    // the warps' maxima, then sums
  alignas(16) float zero[NR];
  alignas(16) uint64_t row_to[NR];  // where the row's outputs go
  Segment seg[kTcItems];            // the items that the queries belong to
  int row_off[kTcItems][NR];        // row of q and out from the item's first, -1: none
  int row_t[kTcItems][NR];          // query (T for rows that do not exist)
  uint32_t row_mask[kTcItems][NR];
  alignas(16) float ks[kTcScaleRing][kTcMaxPages], vs[kTcScaleRing][kTcMaxPages];
  int2 tile[kTcScaleRing];  // first position; whether every query sees every key
  uint64_t full[8], empty[8], scales_full[kTcScaleRing], s_full[2], s_empty[2], p_full,
      pv_done, q_full[kTcItems], q_empty[2], item_empty[kTcItems], drained;
  int64_t warp_sum[16];
  int issued[8];  // the last index of the ring that was copied to each slot, -1: none
  uint32_t tmem;
  TcGuard guard;
};

// Softmax threads: one group of 128 (a thread a key) up to 24 rows, beyond that two
// groups with half the rows each, as a thread holds an exponent and a sum per row.
template <int NR, int D>
struct TcShape {
  static constexpr int NO = (NR + 15) / 16 * 16;
  static constexpr int kGroups = NR > 24 ? 2 : 1;
  static constexpr int kSoftmax = 128 * kGroups;
  static constexpr int kThreads = kSoftmax + 128;          // 256: 128 registers, 384: 80
  static constexpr int W = NR / kGroups;                   // rows of a group
  static constexpr int kSlot = kAttnTile * D;
  static constexpr int kQ = 2 * NR * D;
  static constexpr int kP = 3 * NO * kAttnTile;
  static constexpr int kSmall = 2 * kQ + kP + int(sizeof(TcShared<NR>));
  static constexpr int kFit = (kTcSmem - kSmall) / kSlot;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  // The three terms of P side by side as one operand of three times the columns: V is
  // read once instead of three times, and O's three parts are summed at the end.
  static constexpr int kTerms = NR <= 48 ? 3 : 1;
  static constexpr int kSBufs = 2;  // buffers of scores
  static constexpr int kCols = (kSBufs + kTerms) * NO;
  static constexpr int kAlloc = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static constexpr size_t kBytes = size_t(kSlots) * kSlot + kSmall;
  static_assert(kCols <= 256 && kSlots >= 3, "two CTAs per SM");
  static_assert(size_t(kP) >= (kThreads + 1) * 8, "the plan's sums lie there first");
};

// A ring of N slots or buffers: the place of the next use and the phase it is in.
template <int N>
struct TcRing {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// Bounded wait. Once one has given up, every one that would wait returns at once, and what
// it was for may not be there. The copies and the preparation of queries end then, before
// a false completion lets them write to memory in use; the products run out their loop,
// the softmax groups the item that they have (the barriers among them have to stay
// matched). What is in flight ends before the CTA does, the error bit is set and the
// outputs are not to be used. The loop is a function of its own: inlined at every wait it
// made the hot code outgrow the instruction caches (256 rows of 512-4096 tokens, 20 query
// rows: 223 us inlined, 207 us so).
__device__ __noinline__ void tc_wait_long(uint64_t* bar, uint32_t parity, TcGuard* guard,
                                          int32_t* err) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (guard->aborted()) return;
    if (mbar_try_wait(bar, parity, kSuspendNs)) return;
    if (global_ns() - t0 > guard->limit_ns) break;
  }
  *reinterpret_cast<volatile int*>(&guard->abort) = 1;
  if (err) atomicOr(err, SPEC_DERR_TIMEOUT);
}
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, TcGuard* guard,
                                        int32_t* err) {
  if (!mbar_try_wait(bar, parity, kSuspendNs)) tc_wait_long(bar, parity, guard, err);
}

// Barriers of one softmax group (ids 1 and 2).
__device__ __forceinline__ void bar_group(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}
__device__ __forceinline__ bool bar_group_or(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(group + 1), "r"(uint32_t(x))
      : "memory");
  return r != 0;
}

// The smallest e in [-101, 119] with |x| <= 2^e (119 for larger ones).
__device__ __forceinline__ int scale_binade(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  const int e = int(u >> 23) - 127 + ((u & 0x7fffffu) != 0);
  return max(-101, min(119, e));
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// N times eight rows summed over the warp's keys: lanes exchange halves of the rows
// until each holds one (7 shuffles), then the four lanes of a row finish it. Lane i
// has row reduce8_row(i) of each eight in v[.][0].
__device__ __forceinline__ int reduce8_row(int lane) {
  return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
}
template <int N>
__device__ __forceinline__ void reduce8(float (*v)[8], int lane) {
#pragma unroll
  for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int x = 0; x < N; ++x)
#pragma unroll
      for (int q = 0; q < n; ++q) {
        const float give = up ? v[x][q] : v[x][q + n], keep = up ? v[x][q + n] : v[x][q];
        v[x][q] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1)
#pragma unroll
    for (int x = 0; x < N; ++x) v[x][0] += __shfl_xor_sync(0xffffffffu, v[x][0], o);
}

// Which of w rows of an item, the first of them row `base` of the kv head, see
// position p, as bits. Rows are ordered by query, so those of a chain are a range of
// them; `mask` is null for a chain. Arguments by value: what a function takes by
// reference goes through local memory, that is (with this much shared memory) L2.
__device__ __noinline__ uint32_t seen_rows(int L, int n, int end, int G, int window, int sinks,
                                           int base, int w, const uint32_t* mask, const int* row_t,
                                           int p) {
  if (p >= end) return 0u;
  if (mask && p >= L) {
    uint32_t m = 0;
#pragma unroll 1
    for (int r = 0; r < w; ++r) m |= uint32_t(row_t[r] < n && (mask[r] >> (p - L) & 1u)) << r;
    return m;
  }
  const int first = max(0, p - L);
  // compared before it is added: a window may be as large as an int
  const int last = window == 0 || p < sinks || window >= n - (p - L) ? n : max(0, p - L + window);
  const int lo = max(0, first * G - base), hi = min(w, last * G - base);
  if (hi <= lo) return 0u;
  return (hi == 32 ? ~0u : (1u << hi) - 1u) & (~0u << lo);
}

// Zeroes row `key` of a V tile: what lies there is not a number of the sequence
// (and 0 * NaN is NaN).
template <int D>
__device__ __noinline__ void clear_row(uint8_t* tile, int key) {
  uint4* v = reinterpret_cast<uint4*>(tile + key * D);
#pragma unroll 1
  for (int x = 0; x < D / 16; ++x)  // the lanes start in different banks
    v[(x + key) % (D / 16)] = make_uint4(0u, 0u, 0u, 0u);
}

// The row of q and out where an item's kv head begins.
__device__ __forceinline__ int64_t first_row(const AttnArgs& a, const Segment& g) {
  return int64_t(g.b) * a.T * a.H * a.G + g.h * a.G;
}

// An item's queries as two e4m3 terms a number, by warp w of n: kPerRow lanes a row,
// N numbers each; and what the softmax needs to know of the rows. The two terms take as
// many bytes as the bf16 numbers, which are copied to where their terms will be, all of
// them in flight at once, and converted in place. This warp is what items of a few tiles
// wait for: with loads one step ahead, 16 numbers a lane and the rows' description in the
// same loop (1100 cycles a step) 256 rows of 100-600 tokens took 143 us with 48 query
// rows, so 126 us. 16 numbers a lane there: 130 us; 32 with 20 query rows: 82 instead of
// 80 us.
template <int NR, int D>
__device__ __forceinline__ void prepare_rows(const AttnArgs& a, TcShared<NR>& sh, const Segment& g,
                                             uint8_t* qs, int qb, int w, int n) {
  constexpr int N = NR > 24 ? 32 : 16, kPerRow = D / N, kRows = 32 / kPerRow;
  const int lane = threadIdx.x & 31, part = lane % kPerRow;
  const int rows = min(a.rows_per_block, a.R - g.rb * a.rows_per_block);
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q)) +
                   first_row(a, g) * (D / 8) + N / 8 * part;
  // row / G: the quotient is at most 32, and half a row keeps it 1 / (2 G) off the integers
  const float inv_g = 1.0f / float(a.G);
  const int row0 = g.rb * a.rows_per_block, skip = a.H * a.G - a.G;
  auto query = [&](int r) { return int((float(row0 + r) + 0.5f) * inv_g); };
  // this lane's 16 bytes of a row: of its upper terms, and NR * D bytes on of its lower
  // ones (the swizzle is the same, as the rows differ by a multiple of 8)
  auto place = [&](int r, int y) {
    return qs + r * D + ((N / 16 * part + y) ^ (D == 128 ? r & 7 : (r >> 1) & 3)) * 16;
  };
  const int r0 = w * kRows + lane / kPerRow;
#pragma unroll 1
  for (int r = r0; r < NR; r += n * kRows) {
    const bool ok = r < rows;  // else zeros
    const uint4* x = q + (ok ? int64_t(row0 + r + query(r) * skip) * (D / 8) : 0);
#pragma unroll
    for (int y = 0; y < N / 8; ++y)
      cp_async16(place(r, y >> 1) + (y & 1) * NR * D, x + y, ok);
  }
#pragma unroll 1
  for (int x = w * 32 + lane; x < NR; x += n * 32) {  // a lane a row
    const bool live = x < rows;
    const int t = query(x);
    sh.row_t[qb][x] = live ? t : a.T;
    sh.row_off[qb][x] = live ? row0 + x + t * skip : -1;  // t H G + (row - t G)
    sh.row_mask[qb][x] = a.tree && live ? a.tree[int64_t(g.b) * a.T + t] : 0u;
  }
  cp_async_wait_all();
#pragma unroll 1
  for (int row = r0; row - lane / kPerRow < NR; row += n * kRows) {
    uint32_t u[N / 2];
#pragma unroll
    for (int y = 0; y < N / 8; ++y) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row < NR) v = *reinterpret_cast<const uint4*>(place(row, y >> 1) + (y & 1) * NR * D);
      u[4 * y] = v.x;
      u[4 * y + 1] = v.y;
      u[4 * y + 2] = v.z;
      u[4 * y + 3] = v.w;
    }
    uint32_t two = 0;
#pragma unroll
    for (int y = 0; y < N / 2; ++y) two = __vmaxu2(two, u[y] & 0x7fff7fffu);
    uint32_t top = max(two << 16, two & 0xffff0000u);
#pragma unroll
    for (int s = kPerRow / 2; s > 0; s >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
    // |f| 2^-e in [128, 256) at the largest; e stays in range for bf16 subnormals
    const int e = max(int(top >> 23) - 127 - 7, -110);
    const float down = q8_pow2(-e);
    const float2 down2 = make_float2(down, down);
    uint32_t hw[N / 4], lw[N / 4];
#pragma unroll
    for (int y = 0; y < N / 4; ++y) {
      uint32_t h[2], o[2];  // a bf16 number of this range is one of fp16 as well
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float2 f = __fmul2_rn(make_float2(__uint_as_float(u[2 * y + z] << 16),
                                                __uint_as_float(u[2 * y + z] & 0xffff0000u)),
                                    down2);
        uint32_t v, w;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(f.y), "f"(f.x));
        h[z] = f16x2_to_e4m3(v);
        w = e4m3x2_to_f16(h[z]);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(w) : "r"(v), "r"(w));
        o[z] = f16x2_to_e4m3(w);
      }
      hw[y] = h[0] | h[1] << 16;
      lw[y] = o[0] | o[1] << 16;
    }
    if (row < NR) {
#pragma unroll
      for (int y = 0; y < N / 16; ++y) {
        uint8_t* to = place(row, y);
        const uint32_t *h = hw + 4 * y, *l = lw + 4 * y;
        *reinterpret_cast<uint4*>(to) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(to + NR * D) = make_uint4(l[0], l[1], l[2], l[3]);
      }
      // a row with an infinity or a NaN: its scores are NaN
      if (part == 0)
        sh.row_c[qb][row] =
            top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : q8_pow2(e) * a.scale_log2;
    }
  }
}

template <int NR, int D>
__global__ void __launch_bounds__(TcShape<NR, D>::kThreads, 2)
    attn_tc_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map) {
  using S = TcShape<NR, D>;
  constexpr int NS = S::kSlots, NO = S::NO, SB = S::kSBufs;
  constexpr int kTmaWarp = S::kSoftmax / 32, kMmaWarp = kTmaWarp + 2, kQWarp = kTmaWarp + 3;
  constexpr uint32_t kSwz = D == 128 ? 2 : 4;  // TMA and operands: 128- or 64-byte swizzle
  extern __shared__ __align__(1024) uint8_t sm[];  // ring, queries, P, the rest
  uint8_t* q_s = sm + NS * S::kSlot;
  uint8_t* p_s = q_s + 2 * S::kQ;
  TcShared<NR>& sh = *reinterpret_cast<TcShared<NR>*>(p_s + S::kP);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, nc = gridDim.x;
  int64_t* prefix = reinterpret_cast<int64_t*>(p_s);  // before the first item only

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kTcScaleRing; ++i) mbar_init(&sh.scales_full[i], 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], S::kSoftmax);
      mbar_init(&sh.q_empty[i], 1);
    }
    for (int i = 0; i < kTcItems; ++i) {
      mbar_init(&sh.q_full[i], 32);
      mbar_init(&sh.item_empty[i], S::kSoftmax);
    }
    mbar_init(&sh.p_full, S::kSoftmax);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < 8; ++i) sh.issued[i] = -1;
    sh.guard.abort = 0;
    sh.guard.limit_ns = a.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, S::kAlloc);
    tmem_relinquish();
    if (lane == 0) tma_prefetch_map(&map);
  }
  if (tid < NR) sh.zero[tid] = 0.0f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  const AttnPlan plan = attn_plan(a, prefix, sh.warp_sum, nc, c);
  const bool work = plan.u0 < plan.u1;
  Segment g;
  if (work) g = find_segment(a, prefix, plan.u0, plan.u1);
  __syncthreads();
  const int tiles = int(plan.u1 - plan.u0);
  auto last_of_cta = [&](const Segment& s) { return s.u + (s.t1 - s.t0) >= plan.u1; };

  if (work && (warp < kTmaWarp || warp == kQWarp)) {
    // ---------------------------------------------------------------- queries
    // The first item's are taken by the softmax warps too; the next ones' by a warp of
    // their own, while the item before is worked on. One place in the code for both.
    // The queries' buffer is free again with the item's last scores; what describes its
    // rows is used to the item's end, and has one place more.
    TcRing<2> qbuf;
    TcRing<kTcItems> item;
    int w = warp < kTmaWarp ? warp : warp - 3, n = S::kSoftmax / 32 + 1;
    for (bool first = true;; first = false) {
      if (!first) {
        tc_wait(&sh.q_empty[qbuf.at], qbuf.phase ^ 1, &sh.guard, a.err);
        tc_wait(&sh.item_empty[item.at], item.phase ^ 1, &sh.guard, a.err);
        if (__any_sync(0xffffffffu, sh.guard.aborted())) break;
      }
      prepare_rows<NR, D>(a, sh, g, q_s + qbuf.at * S::kQ, item.at, w, n);
      fence_async_smem();
      if (first) asm volatile("bar.sync 3, %0;" ::"n"(S::kSoftmax + 32) : "memory");
      if (warp < kTmaWarp) break;
      w = 0;
      n = 1;
      if (lane == 0) sh.seg[item.at] = g;
      mbar_arrive(&sh.q_full[item.at]);
      if (first && lane == 0) write_join(a, plan, &g, c);
      qbuf.next();
      item.next();
      if (last_of_cta(g)) break;
      next_segment(a, g, plan.u1);
    }
  }
  if (work && (warp == kTmaWarp || warp == kTmaWarp + 1)) {
    // ---------------------------------------------------------------- TMA
    // One warp for K (and the scales), one for V: a lane issues a block's copy, the
    // lanes of a warp one after the other (some 100 cycles each), which for blocks of 16
    // tokens is what one warp could not do fast enough. The ring's slots are taken in the
    // order K_0, then K_(j+1) and V_j in turn, as the products take them: a V tile loaded
    // with its K tile would hold its slot for longer.
    const bool is_v = warp != kTmaWarp;
    const int bs = min(a.bs, kAttnTile);  // rows of one copy
    const int pages = kAttnTile / bs;
    auto page_id = [&](int k) {
      const int pos = tile_start(g.s, k) + lane * bs;
      return lane < pages && needed(g.s, pos, bs) ? a.bt[int64_t(g.b) * a.MB + pos / a.bs] : -2;
    };
    int k = g.t0;
    TcRing<kTcScaleRing> sring;
    int id = page_id(k);
    for (int j = 0; j < tiles; ++j) {
      if (is_v && g.b == a.stall_row) break;
      const int cur = id;
      const bool ok = cur >= 0 && cur < a.NB;
      const int p0 = tile_start(g.s, k);
      const int c1 = a.bs <= kAttnTile ? 0 : p0 % a.bs;
      const int plane = ok ? cur * a.planes_per_block + a.plane0 + g.h : 0;
      const float* sp = a.scales + (ok ? cur * a.block_scales : 0) + g.h;
      const bool open =
          !is_v && __all_sync(0xffffffffu, ok || lane >= pages) && tile_open(a, g.s, p0);
      if (++k == g.t1 && j + 1 < tiles) {
        next_segment(a, g, plan.u1);
        k = g.t0;
      }
      if (j + 1 < tiles) id = page_id(k);  // in flight while this tile's slot is awaited
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * uint32_t(bs) * D;
      const int i = is_v ? 2 * j + (j + 1 < tiles ? 2 : 1) : max(0, 2 * j - 1);
      const int slot = i % NS;
      tc_wait(&sh.empty[slot], ((i / NS) & 1) ^ 1, &sh.guard, a.err);
      if (__any_sync(0xffffffffu, sh.guard.aborted())) break;
      if (lane == 0) {
        sh.issued[slot] = i;
        mbar_arrive_expect_tx(&sh.full[slot], bytes);
      }
      __syncwarp();
      if (ok)
        tma_tile_3d(sm + slot * S::kSlot + lane * bs * D, &map, 0, c1, plane + (is_v ? a.H : 0),
                    &sh.full[slot]);
      if (is_v) continue;
      if (cur != -2 && !ok && a.err) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
      bool copying = false;
      if (lane < pages) {
        float* ks = &sh.ks[sring.at][lane];
        float* vs = &sh.vs[sring.at][lane];
        if (ok) {
          cp_async4(ks, sp);
          cp_async4(vs, sp + a.H);
          copying = true;
        } else {
          // a block that cannot be read: NaN scores; one that is not needed: zeros
          *ks = cur == -2 ? 0.0f : __uint_as_float(0x7fc00000u);
          *vs = 0.0f;
        }
      }
      if (lane == 31) sh.tile[sring.at] = make_int2(p0, open);  // pages <= 16: it copies nothing
      if (copying) cp_async_arrive(&sh.scales_full[sring.at]);
      else mbar_arrive(&sh.scales_full[sring.at]);
      sring.next();
    }
    cp_async_wait_all();  // (done with already, unless the loop was left)
  } else if (work && warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc_s = tc_idesc(0, 0, 0, 0, 128, NO);
      constexpr uint32_t idesc_o = tc_idesc(0, 1, 1, 1, 128, S::kTerms * NO);
      const uint64_t slot0 = tc_desc(smem_u32(sm), 16, 8 * D, kSwz);
      const uint64_t v_slot0 = tc_desc(smem_u32(sm), 0, 8 * D, kSwz);
      const uint64_t q0 = tc_desc(smem_u32(q_s), 16, 8 * D, kSwz);
      const uint64_t p0 = tc_desc(smem_u32(p_s), 128, 2048, 0);
      int k = g.t0;  // tile of the next scores
      TcRing<NS> ring;
      TcRing<SB> sbuf;
      TcRing<2> qbuf;
      TcRing<kTcItems> item;
      uint32_t p_phase = 0;
      auto scores = [&]() {  // returns whether the tile is its item's first
        const bool first = k == g.t0;
        if (first) tc_wait(&sh.q_full[item.at], item.phase, &sh.guard, a.err);
        tc_wait(&sh.full[ring.at], ring.phase, &sh.guard, a.err);
        tc_wait(&sh.s_empty[sbuf.at], sbuf.phase ^ 1, &sh.guard, a.err);
        tc_fence_after();
        const uint64_t k_desc = slot0 + ring.at * (S::kSlot / 16);
        const uint64_t q_desc = q0 + qbuf.at * (S::kQ / 16);
        // both terms of the queries into one sum (columns past the rows are not read)
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          tc_mma_f8(tmem + sbuf.at * NO, k_desc + 2 * x, q_desc + 2 * x, idesc_s, x > 0);
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          tc_mma_f8(tmem + sbuf.at * NO, k_desc + 2 * x, q_desc + NR * D / 16 + 2 * x, idesc_s, true);
        tc_commit(&sh.empty[ring.at]);
        tc_commit(&sh.s_full[sbuf.at]);
        ring.next();
        sbuf.next();
        if (++k == g.t1) {
          tc_commit(&sh.q_empty[qbuf.at]);
          if (!last_of_cta(g)) next_segment(a, g, plan.u1);
          k = g.t0;
          qbuf.next();
          item.next();
        }
        return first;
      };
      auto outputs = [&](bool first) {
        tc_wait(&sh.full[ring.at], ring.phase, &sh.guard, a.err);
        tc_wait(&sh.p_full, p_phase, &sh.guard, a.err);
        p_phase ^= 1;
        tc_fence_after();
        // V as stored: D contiguous, groups of 8 keys 8 D bytes apart. With D = 64 the
        // second half of M repeats the first (offset 0) and is ignored.
        const uint64_t v_desc = v_slot0 + ring.at * (S::kSlot / 16);
#pragma unroll
        for (int x = 0; x < kAttnTile / 32; ++x)
#pragma unroll
          for (int m = 0; m < 3; m += S::kTerms)
            tc_mma_f8(tmem + SB * NO, v_desc + x * (32 * D / 16),
                      p0 + (m * NO * kAttnTile + x * 512) / 16, idesc_o,
                      !(first && x == 0 && m == 0));
        tc_commit(&sh.empty[ring.at]);
        tc_commit(&sh.pv_done);
        ring.next();
      };
      bool first = scores();
      for (int j = 0; j < tiles; ++j) {
        bool next = false;
        // The order of the copies, always: the ring's waits are by parity, and a slot
        // freed out of turn would let a copy warp pass one that is two rounds behind.
        if (j + 1 < tiles) next = scores();
        outputs(first);
        first = next;
      }
    }
    __syncwarp();
  } else if (work && warp < kTmaWarp) {
    // ---------------------------------------------------------------- softmax
    constexpr int W = S::W, chunks = W / 8;  // rows of a group, in eights
    const int group = warp >> 2, gw = warp & 3, key = tid & 127, col0 = group * W;
    float* const nm = sh.row_nm + col0;
    float* const ra = sh.row_a + col0;
    const uint32_t lane_addr = tmem + (uint32_t(gw * 32) << 16) + col0;
    const uint32_t o_addr = lane_addr + SB * NO;
    const int page = key >> (a.bs >= kAttnTile ? 7 : 31 - __clz(a.bs));
    TcRing<kTcItems> item;
    int j = 0;  // tile of the CTA
    auto wait_outputs = [&]() {  // of the tile before
      tc_wait(&sh.pv_done, (j & 1) ^ 1, &sh.guard, a.err);
    };
    for (;; item.next()) {
      const int qb = item.at;
      tc_wait(&sh.q_full[qb], item.phase, &sh.guard, a.err);
      const Segment& g = sh.seg[qb];  // read where it is needed: registers are scarce here
      const int j_first = j, j_end = j + (g.t1 - g.t0);
      if (key < W) nm[key] = sh.row_off[qb][col0 + key] >= 0 ? kTcUnset : 0.0f;
      if (bar_group_or(group, sh.guard.aborted())) break;  // the item may never be described
      float2 l[W / 2];
#pragma unroll
      for (int r = 0; r < W / 2; ++r) l[r] = make_float2(0.0f, 0.0f);

#pragma unroll 1
      for (; j < j_end; ++j) {
        const int se = j % kTcScaleRing, sb = j & 1;
        tc_wait(&sh.scales_full[se], j / kTcScaleRing & 1, &sh.guard, a.err);
        const float vs = sh.vs[se][page];
        float ks = sh.ks[se][page];
        const int2 info = sh.tile[se];
        const bool open = info.y;
        if (!(fabsf(vs) <= FLT_MAX)) ks = __uint_as_float(0x7fc00000u);
        const float vr = vs * kTcVDown;
        const float lv = float(scale_binade(vr));  // vr <= 2^lv
        const float2 ks2 = make_float2(ks, ks);
        uint32_t seen = ~0u;
        if (!open)
          seen = seen_rows(g.s.L, g.s.n, g.s.end, a.G, a.window, a.sinks,
                           g.rb * a.rows_per_block + col0, W,
                           a.tree ? sh.row_mask[qb] + col0 : nullptr, sh.row_t[qb] + col0,
                           info.x + key);
        tc_wait(&sh.s_full[sb], (j >> 1) & 1, &sh.guard, a.err);
        tc_fence_after();
        const uint32_t s_addr = lane_addr + sb * NO;
        // s k c (- m) of N eights of rows from the x-th
        auto exponents = [&](int x, auto count, const float* minus, float2* y) {
          constexpr int N = decltype(count)::value;
          float z[8 * N];
#pragma unroll
          for (int i = 0; i < N; ++i) tmem_ld8(s_addr + 8 * (x + i), z + 8 * i);
          float4 cs[2 * N], ms[2 * N];
#pragma unroll
          for (int q = 0; q < 2 * N; ++q) {
            cs[q] = *reinterpret_cast<const float4*>(&sh.row_c[qb][col0 + 8 * x + 4 * q]);
            ms[q] = *reinterpret_cast<const float4*>(minus + 8 * x + 4 * q);
          }
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 2 * N; ++q) {
            const float4 c4 = cs[q], m4 = ms[q];
            const float2 s0 = make_float2(z[4 * q], z[4 * q + 1]);
            const float2 s1 = make_float2(z[4 * q + 2], z[4 * q + 3]);
            y[2 * q] = __ffma2_rn(__fmul2_rn(s0, ks2), make_float2(c4.x, c4.y),
                                  make_float2(m4.x, m4.y));
            y[2 * q + 1] = __ffma2_rn(__fmul2_rn(s1, ks2), make_float2(c4.z, c4.w),
                                      make_float2(m4.z, m4.w));
          }
          if (!open) {
            const uint32_t bits = seen >> (8 * x);
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
              if (!(bits >> (2 * i) & 1u)) y[i].x = -INFINITY;
              if (!(bits >> (2 * i + 1) & 1u)) y[i].y = -INFINITY;
            }
          }
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        // Up to 24 rows a thread the exponents stay in registers between the test of the
        // references and the exponentials. 32 do not fit beside the sums (a spill goes to L2:
        // shared memory takes L1's place), and are taken twice.
        constexpr bool kKeep = W <= 24;
        float2 y[kKeep ? W / 2 : 1];
        auto all_exponents = [&](const float* minus) {
#pragma unroll
          for (int x = 0; x + 1 < chunks; x += 2) exponents(x, Two(), minus, y + 4 * x);
          if (chunks % 2) exponents(chunks - 1, One(), minus, y + 4 * (chunks - 1));
        };
        // Usually one pass: relative to the references, none of which has to move. The
        // first tile and one that exceeds them take the plain scores (again).
        bool relative = j > j_first;
        for (;;) {
          if (kKeep) all_exponents(relative ? nm : sh.zero);
          if (!relative) break;
          float top = -INFINITY;
          if (kKeep) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) top = fmaxf(top, fmaxf(y[i].x, y[i].y));
          } else {
#pragma unroll
            for (int x = 0; x < chunks; ++x) {
              float2 e[4];
              exponents(x, One(), nm, e);
#pragma unroll
              for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(e[i].x, e[i].y));
            }
          }
          if (!bar_group_or(group, top > kTcSlack - lv)) break;
          relative = false;
        }
        if (!relative) {
          // move the references to this tile's maxima (a NaN score is passed over: it makes
          // its row's sum NaN by itself)
          auto maxima = [&](int at, float2 e) {
            const float m0 = warp_max(e.x + lv), m1 = warp_max(e.y + lv);
            if (lane == 0) *reinterpret_cast<float2*>(&sh.part[gw][col0 + at]) = make_float2(m0, m1);
          };
          if (kKeep) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) maxima(2 * i, y[i]);
          } else {
#pragma unroll 1
            for (int x = 0; x < chunks; ++x) {
              float2 e[4];
              exponents(x, One(), sh.zero, e);
#pragma unroll
              for (int i = 0; i < 4; ++i) maxima(8 * x + 2 * i, e[i]);
            }
          }
          bar_group(group);
          if (key < W) {
            const float* mp = sh.part[0] + col0 + key;
            const float old = -nm[key];
            const float m = fmaxf(fmaxf(fmaxf(mp[0], mp[NR]), fmaxf(mp[2 * NR], mp[3 * NR])), old);
            nm[key] = -m;
            // the root: references may move by 230 binades with the V scales, and a sum that
            // holds as many still counts
            ra[key] = ex2_approx(0.5f * (old - m));
          }
          bar_group(group);
          if (kKeep) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i)
              y[i] = __fadd2_rn(y[i], *reinterpret_cast<const float2*>(nm + 2 * i));
          }
          if (j > j_first) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
              const float2 root = *reinterpret_cast<const float2*>(ra + 2 * i);
              l[i] = __fmul2_rn(__fmul2_rn(l[i], root), root);
            }
            wait_outputs();
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < S::kTerms * chunks; ++x) {
              const int r = 8 * (x % chunks);
              const uint32_t at = o_addr + x / chunks * NO + r;
              float o[8];
              tmem_ld8(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 8; ++q) o[q] *= ra[r + q] * ra[r + q];
              tmem_st8(at, o);
            }
            tmem_wait_st();
          }
        }
        if (kKeep) {
          tc_fence_before();
          mbar_arrive(&sh.s_empty[sb]);
        }
        wait_outputs();  // P may be replaced
        const float2 lift = make_float2(vr * kTcLift, vr * kTcLift);
        // What the key adds before the terms cut to multiples of 2^-16: (2 x + 1) 2^-24 (an
        // fp16 subnormal, so its bits are 2 x + 1), x from 0 to 127 by turns of the position.
        uint32_t turn = ((uint32_t(key) * 79u + uint32_t(info.x >> 7) * 37u) & 127u) * 2u + 1u;
        turn = (turn | (vr < 0.0f ? 0x8000u : 0u)) * 0x00010001u;
        uint8_t* p_to = p_s + key * 16;
#pragma unroll
        for (int x = 0; x < chunks; ++x) {
          float2 e[4];
          if (!kKeep) exponents(x, One(), nm, e);
          uint32_t t[3][2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t h[2];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int i = 4 * x + 2 * q + w;
              const float2 z = kKeep ? y[kKeep ? i : 0] : e[2 * q + w];
              const float2 p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
              l[i] = __fadd2_rn(l[i], p);
              const float2 v = __fmul2_rn(p, lift);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[w]) : "f"(v.y), "f"(v.x));
              h[w] = (h[w] + 0x00020002u) & 0xfffcfffcu;  // 9 bits, half up
              asm("add.rn.f16x2 %0, %0, %1;" : "+r"(h[w]) : "r"(turn));
            }
            auto rest = [](uint32_t v) {
              uint32_t o;
              asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(v), "r"(v & 0xff00ff00u));
              return o;
            };
            t[0][q] = __byte_perm(h[0], h[1], 0x7531);
            h[0] = rest(h[0]);
            h[1] = rest(h[1]);
            t[1][q] = __byte_perm(h[0], h[1], 0x7531);
            h[0] = rest(h[0]);
            h[1] = rest(h[1]);
            t[2][q] = __byte_perm(h[0], h[1], 0x7531);
          }
          const int col = col0 + 8 * x;
          uint8_t* d = p_to + (col >> 4) * 2048 + (col & 8);
#pragma unroll
          for (int m = 0; m < 3; ++m)
            *reinterpret_cast<uint2*>(d + m * NO * kAttnTile) = make_uint2(t[m][0], t[m][1]);
        }
        if (!kKeep) {
          tc_fence_before();
          mbar_arrive(&sh.s_empty[sb]);
        }
        if (!open && group == 0 && (!(ks == ks) || !needed(g.s, info.x + key, 1))) {
          const int vi = 2 * j + (j + 1 < tiles ? 2 : 1);  // loads before it: j or j + 1 of K
          tc_wait(&sh.full[vi % NS], (vi / NS) & 1, &sh.guard, a.err);
          clear_row<D>(sm + vi % NS * S::kSlot, key);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.p_full);
      }

      // ------------------------------------------------------------ the item's end
      {
        float v[chunks][8];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          v[i / 4][i % 4 * 2] = l[i].x;
          v[i / 4][i % 4 * 2 + 1] = l[i].y;
        }
        reduce8<chunks>(v, lane);
        if ((lane & 3) == 0)
#pragma unroll
          for (int x = 0; x < chunks; ++x) sh.part[gw][col0 + 8 * x + reduce8_row(lane)] = v[x][0];
      }
      bar_group(group);
      const bool whole = g.t0 == 0 && g.t1 == g.s.tiles;
      const int64_t slot = 2 * c + (g.u == plan.u0 ? 0 : 1);
      if (key < W) {
        const float* mp = sh.part[0] + col0 + key;
        float sum = mp[0] + mp[NR] + mp[2 * NR] + mp[3 * NR];
        // half a million keys above the reference whose values are all zero; a NaN stays
        if (sum > kTcMaxSum) sum = kTcMaxSum;
        // A part is left with its sum in [1, 2): references of parts differ by their V
        // scales, so a sum by itself may be as far from 1 as those.
        const int e = sum > 0.0f ? int(__float_as_uint(sum) >> 23) - 127 : 0;
        constexpr float unlift = 1.0f / (kTcLift * kTcVDown);
        const float down = q8_pow2(-e);
        ra[key] = (!whole ? down : sum == 0.0f ? 0.0f : __fdividef(down, sum * down)) * unlift;
        const int off = sh.row_off[qb][col0 + key];
        const int64_t part = slot * a.rows_per_block + col0 + key;
        sh.row_to[col0 + key] =
            whole ? reinterpret_cast<uint64_t>(static_cast<__nv_bfloat16*>(a.out) + (first_row(a, g) + off) * D)
                  : reinterpret_cast<uint64_t>(a.parts + part * D);
        if (!whole && off >= 0)
          a.stats[part] = make_float2(sum == 0.0f ? -INFINITY : -nm[key] + float(e),
                                      sum * q8_pow2(-e));
      }
      bar_group(group);
      wait_outputs();
      tc_fence_after();
      const bool last = last_of_cta(g);
      const int live = min(W, min(a.rows_per_block, a.R - g.rb * a.rows_per_block) - col0);
#pragma unroll 1
      for (int x = 0; x < chunks; ++x) {
        float o[S::kTerms][8];
#pragma unroll
        for (int m = 0; m < S::kTerms; ++m) tmem_ld8(o_addr + m * NO + 8 * x, o[m]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          const float4 f = *reinterpret_cast<const float4*>(ra + 8 * x + q);
          const float by[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
#pragma unroll
            for (int m = 1; m < S::kTerms; ++m) o[0][q + z] += o[m][q + z];
            o[0][q + z] *= by[z];
          }
        }
        if (D < 128 && key >= D) continue;
        uint64_t to[8];  // all read before the first store: it could be to any of them
#pragma unroll
        for (int q = 0; q < 8; q += 2) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&sh.row_to[col0 + 8 * x + q]);
          to[q] = v.x;
          to[q + 1] = v.y;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (8 * x + q < live) {
            if (whole) reinterpret_cast<__nv_bfloat16*>(to[q])[key] = __float2bfloat16(o[0][q]);
            else reinterpret_cast<float*>(to[q])[key] = o[0][q];
          }
      }
      tc_fence_before();  // the next item's products overwrite O after its p_full
      mbar_arrive(&sh.item_empty[qb]);
      if (last) break;
      bar_group(group);  // row_a, row_nm, part: every thread is done with the item
    }
  }
  if (warp == kQWarp) {
    // what needs no place in the row of the others' work
    if (!work && lane == 0) write_join(a, plan, nullptr, c);
    write_empty_rows<__nv_bfloat16>(a, c, nc, lane, 32);
  }
  tc_fence_before();
  __syncthreads();
  if (sh.guard.abort) {
    // nothing more is issued: what is in flight ends before the CTA's memory is another's
    if (warp == kTmaWarp)
      for (int x = 0; x < NS; ++x)
        if (sh.issued[x] >= 0) mbar_wait(&sh.full[x], (sh.issued[x] / NS) & 1);
    if (warp == kMmaWarp) {
      if (lane == 0) tc_commit(&sh.drained);
      __syncwarp();
      mbar_wait(&sh.drained, 0);
      __syncwarp();  // the warp frees the TMEM as one
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, S::kAlloc);
}

// ------------------------------------------------------------------ host
bool attn_tc_takes(int dtype, int D, int bs, int64_t planes) {
  const bool blocks = bs == 8 || bs == 16 || bs == 32 || bs == 64 || (bs >= 128 && bs % 128 == 0);
  return dtype == SPEC_BF16 && (D == 128 || D == 64) && blocks && planes <= INT32_MAX;
}

// Query rows of one block: all of them up to 64, else equal blocks of at most 64.
int attn_tc_rows(int R) {
  const int blocks = (R + 63) / 64;
  return (R + blocks - 1) / blocks;
}

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &st) != cudaSuccess ||
        st != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

template <int NR, int D>
int launch_shape(const AttnArgs& a, const CUtensorMap& map, int nc, cudaStream_t st) {
  auto kern = attn_tc_kernel<NR, D>;
  constexpr size_t smem = TcShape<NR, D>::kBytes;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kern, smem, done) != SPEC_OK) return SPEC_ECUDA;
  return launch_pdl(kern, dim3(nc), dim3(TcShape<NR, D>::kThreads), smem, st, a, map);
}

template <int D>
int launch_rows(const AttnArgs& a, const CUtensorMap& map, int nc, cudaStream_t st) {
  const int r = a.rows_per_block;
  if (r <= 8) return launch_shape<8, D>(a, map, nc, st);
  if (r <= 16) return launch_shape<16, D>(a, map, nc, st);
  if (r <= 24) return launch_shape<24, D>(a, map, nc, st);
  if (r <= 32) return launch_shape<32, D>(a, map, nc, st);
  if (r <= 48) return launch_shape<48, D>(a, map, nc, st);
  return launch_shape<64, D>(a, map, nc, st);
}

}  // namespace

int launch_attn_tc(const AttnArgs& a, const void* pool_base, int64_t planes, int sms, int max_ctas,
                   int* nc, void* stream) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return SPEC_ECUDA;
  CUtensorMap map;
  const cuuint64_t dims[3] = {cuuint64_t(a.D), cuuint64_t(a.bs), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(a.D), cuuint64_t(a.bs) * a.D};
  const cuuint32_t box[3] = {cuuint32_t(a.D), cuuint32_t(a.bs < kAttnTile ? a.bs : kAttnTile), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool_base), dims, strides, box,
          step, CU_TENSOR_MAP_INTERLEAVE_NONE,
          a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SPEC_ECUDA;
  *nc = 2 * sms < max_ctas ? 2 * sms : max_ctas;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.D == 128 ? launch_rows<128>(a, map, *nc, st) : launch_rows<64>(a, map, *nc, st);
}

}  // namespace sv
