// The prefix attention's products and softmax (kv_prefix.cuh says what is computed and
// how the work is split).
//
// With the queries of many rows there are enough of them to be the M operand:
//   S [128 queries x 128 keys]  = (Qhi + Qlo) [128 x D] * K^T   e4m3 x e4m3, fp32 sums in TMEM
//   O [128 queries x D]        += P [128 x 128] * V             bf16 x bf16, P in TMEM
// A thread owns a query: no maximum or sum crosses lanes. Two M tiles per CTA take turns, so
// that the tensor core works for one while the other's softmax runs: with more than 128
// queries they are two halves of the block and share each key tile, else both hold the same
// queries and take the key tiles by turns, each with a part of its own, added at the end.
//
// K goes from TMA into the products as it is cached (queries as in the other attention kernel:
// a row scaled by a power of two, two e4m3 terms a number, 4 + 4 bits). V is widened to bf16 on
// its way to shared memory, exactly: a code's exponent and fraction are moved to their place,
// then one product with scale * 2^120, exact for the powers of two that appending leaves (other
// scales take a path that multiplies in fp32 and rounds once to bf16). Widening K too kept the
// loading warps from keeping up. P is rounded to bf16 (2^-8 relative, as the output); the sums l
// take it in fp32 before. K's scales belong to 16 keys and enter the softmax as one factor each.
//   Softmax: a row's reference is a bound of its scores, in whole binades, 24 above the largest
// of those that set it; when a later one exceeds it, it is set anew, and O and l are scaled,
// exactly. A query's scores of a tile stay in registers from the maximum to the probabilities.
//
// Roles, of 4 warps each with registers moved to the softmax: two softmax groups; widening of V;
// a warp for each group's products, one that walks the work list and prepares queries, one that
// finds the tiles and starts their copies. One CTA per SM.
//
// Bound by the chain of a tile: scores 240 cycles after the last product is issued, softmax 1900
// to 2400, a turn's products 1500; a step of two M tiles takes 4450 cycles, its products 2050 (one
// warp for both groups' products, with 1100 cycles of its own code before each turn: 4860). 297 us
// for 5120 queries of each of 8 kv heads before 16000 shared keys, 336 GFLOP: 0.60 of the bf16 peak.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "kv_prefix.cuh"
#include "launch_util.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace sv {

constexpr int kPfSoftmax = 256, kPfLoad = 128, kPfThreads = kPfSoftmax + kPfLoad + 128;
constexpr int kPfSoftmaxRegs = 184, kPfLoadRegs = 64, kPfOtherRegs = 80;
static_assert(256 * kPfSoftmaxRegs + 128 * (kPfLoadRegs + kPfOtherRegs) == 65536,
              "what the groups give up is what the softmax takes");
constexpr int kPfItems = 6;     // items described at a time
constexpr int kPfQueries = 2;   // M tiles of queries held at a time
constexpr int kPfFactors = 16;  // M tiles whose rows' factors are held: more than kPfItems items have
constexpr int kPfTurns = 8;     // more than the steps between the groups
constexpr int kPfPart = 16;     // keys of a part of a tile: of one block (block_size % 16 == 0)
constexpr int kPfParts = kPfTile / kPfPart;
constexpr float kMaxBf16 = 0x1.fep127f;
// Binades between the largest score of a row and its reference when that is set: probabilities
// are 2^-24 to 1 then, in which bf16 and fp32 lose nothing (keys 2^-100 of the largest are lost).
constexpr float kPfHeadroom = 24.0f;

// Bounded waits. A wait ends when its barrier's phase does or when `abort` is set; the walking
// warp sets it (and the error bit) when no tile has been done for a while, and every role then
// leaves its loop. So a wait is a few instructions: with a clock of its own in each, the code
// of the loops outgrew the instruction cache.
struct PfGuard {
  int abort;
  int beat[2];   // tiles that each softmax group has done
  int done[2];   // whether it has ended
  __device__ __forceinline__ bool aborted() const {
    return *reinterpret_cast<const volatile int*>(&abort) != 0;
  }
};

// One piece of an item.
struct PfItem {
  int stop;       // no more items
  int two;        // two M tiles (else one, and its key tiles by turns)
  int row;        // one of the group
  int entry;      // the group's first member
  int h;
  int t0, t1;     // tiles of the item
  int q0, nq;     // first query of the block in its group, queries of the block
};

// A key tile: what the warps need of it.
struct PfTile {
  int plane[kPfParts], in_block[kPfParts];  // where the parts' V is (plane -1: nowhere)
  alignas(16) float ks[kPfParts];           // scales of K (1 where one of them is below 0),
  float raw_ks[kPfParts], vs[kPfParts];     // those of K then, of V
  int valid;                                // bits: parts that are copied
  int below, plain_v;                       // a scale of K is below 0; V's are 2^-100 .. 2^7
};

// kTiles: more than the key tiles between their finding and the end of their V: one being
// written, those in K's slots, one at each softmax group, those whose V is in slots.
template <int D>
struct PfShape {
  static constexpr int kCodeBytes = kPfTile * D;        // K or V as cached, a term of the queries
  static constexpr int kWideBytes = kPfTile * D * 2;    // V in bf16, an M tile of queries
  static constexpr int kKSlots = D == 128 ? 3 : 4, kRawSlots = kKSlots - 1;
  static constexpr int kVSlots = D == 128 ? 2 : 3;
  static constexpr int kTiles = 1 + kKSlots + 2 + kRawSlots + kVSlots + 4;
  struct Shared {
    PfTile tile[kTiles];
    PfItem item[kPfItems];
    float factor[kPfFactors][kPfTile];  // of the rows' scores
    float2 part[2][kPfTile];  // what one group tells the other at the end of an item
    int raw_tile[kRawSlots];  // whose V is there
    uint64_t item_full[kPfItems], item_empty[kPfItems];
    uint64_t raw_full[kRawSlots], raw_empty[kRawSlots];
    uint64_t q_full[kPfQueries], q_empty[kPfQueries];
    uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
    uint64_t turn[2][kPfTurns];
    uint64_t s_full[2], p_full[2], o_full[2], told[2], read[2], drained;
    uint32_t tmem;
    PfGuard guard;
  };
  static constexpr size_t kBytes = size_t(kKSlots + kRawSlots) * kCodeBytes +
                                   size_t(kVSlots + kPfQueries) * kWideBytes + sizeof(Shared);
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, const PfGuard* guard) {
  while (!mbar_try_wait(bar, parity, kSuspendNs))
    if (guard->aborted()) return false;
  return true;
}

template <int N>
struct PfRing {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1;
    }
  }
};

// Where a V tile holds 16-byte chunk c (of D / 8) of key r: halves of 64 numbers, rows of 128
// bytes, 128-byte swizzle. Where K, or a term of the queries, holds chunk c (of D / 16) of row
// r: rows of D bytes, swizzled over D bytes.
__device__ __forceinline__ uint32_t pf_place(int r, int c) {
  return uint32_t((c >> 3) * (kPfTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
template <int D>
__device__ __forceinline__ uint32_t pf_place8(int r, int c) {
  return uint32_t(r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
}

// The row of q and out ([B, T, H * G]) of query x of an item's block, or -1.
__device__ __forceinline__ int64_t pf_query(const PfArgs& a, const PfPlan& p, const PfItem& it,
                                            int x) {
  if (x >= it.nq) return -1;
  const int R = a.T * a.G, qi = it.q0 + x, e = qi / R, r = qi - e * R;
  const int b = it.entry + e < p.NE ? p.members[it.entry + e] : -1, t = r / a.G;
  if (b < 0 || b >= a.B || t >= p.rows[b].n) return -1;
  return (int64_t(b) * a.T + t) * a.H * a.G + it.h * a.G + (r - t * a.G);
}

// Two e4m3 codes to two bf16 numbers divided by 2^120: the sign to bit 15, the exponent's and
// fraction's 7 bits to 10 .. 4. `kSel` picks two bytes of w, each with its sign behind it.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t e4m3_in_bf16(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "n"(kSel));
  return (r << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// One lane of the warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(f[0]), "f"(f[1]),
               "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(n)
      : "memory");
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* f) {
  uint32_t* r = reinterpret_cast<uint32_t*>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// Waits for the loads; what uses f (or, with `tie` alone, comes after the wait) stays behind it.
__device__ __forceinline__ void tmem_tie32(float* f) {
  asm volatile(""
               : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]),
                 "+f"(f[7]), "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]),
                 "+f"(f[13]), "+f"(f[14]), "+f"(f[15]), "+f"(f[16]), "+f"(f[17]), "+f"(f[18]),
                 "+f"(f[19]), "+f"(f[20]), "+f"(f[21]), "+f"(f[22]), "+f"(f[23]), "+f"(f[24]),
                 "+f"(f[25]), "+f"(f[26]), "+f"(f[27]), "+f"(f[28]), "+f"(f[29]), "+f"(f[30]),
                 "+f"(f[31])
               :
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// D[tmem] (+)= A B; one thread issues. Scores: e4m3, K = 32, both in shared memory. Outputs: bf16,
// K = 16, A in TMEM. `hi`: the upper half of the descriptors.
__device__ __forceinline__ void pf_mma_s(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
__device__ __forceinline__ void pf_mma_o(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}

// An M tile of an item's queries (from query x0 of its block) as two e4m3 terms a number, and
// the factors of its rows' scores, by warp w of n. A row's bf16 numbers are copied to where
// their terms will be (as many bytes), all in flight at once, then converted in place, 32 a
// lane: scaled by a power of two to [128, 256) at the row's largest, and split.
template <int D>
__device__ __forceinline__ void pf_prepare(const PfArgs& a, const PfPlan& p, const PfItem& it, int x0,
                                        uint8_t* to, float* factor, int w, int n) {
  constexpr int kChunks = D / 8, kLanes = D / 32, kRows = 32 / kLanes, kTerm = kPfTile * D;
  const int lane = threadIdx.x & 31;
  const int rows = min(kPfTile, max(0, it.nq - x0));
  // raw chunk c of a row: even ones to the upper term's chunk c / 2, odd ones to the lower's
  for (int r0 = w * 32; r0 < kPfTile; r0 += n * 32) {
    const int64_t mine = pf_query(a, p, it, x0 + r0 + lane);
    if (mine < 0) factor[r0 + lane] = 0.0f;
#pragma unroll 4
    for (int x = 0; x < kChunks; ++x) {
      const int c = x * 32 + lane, r = c / kChunks, y = c % kChunks;
      const int64_t row = __shfl_sync(0xffffffffu, mine, r);
      cp_async16(to + (y & 1) * kTerm + pf_place8<D>(r0 + r, y >> 1),
                 static_cast<const __nv_bfloat16*>(a.q) + (row < 0 ? 0 : row) * D + y * 8, row >= 0);
    }
  }
  cp_async_wait_all();
  __syncwarp();
  for (int r0 = w * 32; r0 < rows; r0 += n * 32)
#pragma unroll 1
    for (int s = 0; s < 32; s += kRows) {
      const int r = r0 + s + lane / kLanes, part = lane % kLanes;
      uint32_t u[16];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint4 v = *reinterpret_cast<const uint4*>(
            to + (y & 1) * kTerm + pf_place8<D>(r, 2 * part + (y >> 1)));
        u[4 * y] = v.x;
        u[4 * y + 1] = v.y;
        u[4 * y + 2] = v.z;
        u[4 * y + 3] = v.w;
      }
      uint32_t two = 0;
#pragma unroll
      for (int y = 0; y < 16; ++y) two = __vmaxu2(two, u[y] & 0x7fff7fffu);
      uint32_t top = max(two << 16, two & 0xffff0000u);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // e stays in range for bf16 subnormals
      const int e = max(int(top >> 23) - 127 - 7, -110);
      const float down = q8_pow2(-e);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          uint32_t h[2], o[2];  // a bf16 number of this range is one of fp16 as well
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t x = u[8 * y + 2 * z + q];
            uint32_t v, g;
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(v)
                : "f"(__uint_as_float(x & 0xffff0000u) * down), "f"(__uint_as_float(x << 16) * down));
            h[q] = f16x2_to_e4m3(v);
            g = e4m3x2_to_f16(h[q]);
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(g) : "r"(v), "r"(g));
            o[q] = f16x2_to_e4m3(g);
          }
          hw[z] = h[0] | h[1] << 16;
          lw[z] = o[0] | o[1] << 16;
        }
        uint8_t* at = to + pf_place8<D>(r, 2 * part + y);
        *reinterpret_cast<uint4*>(at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(at + kTerm) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
      // a row with an infinity or a NaN: its scores are NaN
      if (part == 0)
        factor[r] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : q8_pow2(e) * a.scale_log2;
    }
}

// O of a row times `by`.
template <int D>
__device__ __forceinline__ void pf_rescale(uint32_t o_addr, float by) {
  float o[16];
#pragma unroll 1
  for (int y = 0; y < D; y += 16) {
    tmem_ld8(o_addr + y, o);
    tmem_ld8(o_addr + y + 8, o + 8);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      asm volatile("" : "+f"(o[x]));
      o[x] *= by;
    }
    tmem_st8(o_addr + y, o);
    tmem_st8(o_addr + y + 8, o + 8);
  }
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1)
    kv_prefix_attention_kernel(const __grid_constant__ PfArgs a,
                               const __grid_constant__ CUtensorMap map) {
  using S = PfShape<D>;
  constexpr int KS = S::kKSlots, RS = S::kRawSlots, VS = S::kVSlots, NT = S::kTiles;
  constexpr int kCode = S::kCodeBytes, kWide = S::kWideBytes;
  constexpr int kMmaWarp = (kPfSoftmax + kPfLoad) / 32, kWalkWarp = kMmaWarp + 2,
                kFindWarp = kMmaWarp + 3;
  extern __shared__ __align__(1024) uint8_t sm[];  // V, queries, K, V as cached, the rest
  uint8_t* q_s = sm + VS * kWide;
  uint8_t* k_s = q_s + kPfQueries * kWide;
  uint8_t* raw_s = k_s + KS * kCode;
  typename S::Shared& sh = *reinterpret_cast<typename S::Shared*>(raw_s + RS * kCode);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kPfItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], kPfSoftmax / 32 + 3);
    }
    for (int i = 0; i < RS; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kPfLoad / 32);
    }
    for (int i = 0; i < kPfQueries; ++i) {
      mbar_init(&sh.q_full[i], kPfSoftmax / 32);
      mbar_init(&sh.q_empty[i], 2);
    }
    for (int i = 0; i < KS; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.k_empty[i], 2);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&sh.v_full[i], kPfLoad / 32);
      mbar_init(&sh.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.told[i], 128);
      mbar_init(&sh.read[i], 128);
    }
    for (int i = 0; i < 2 * kPfTurns; ++i) mbar_init(&sh.turn[0][0] + i, 1);
    mbar_init(&sh.drained, 2);
    sh.guard.abort = sh.guard.beat[0] = sh.guard.beat[1] = sh.guard.done[0] = sh.guard.done[1] = 0;
    fence_mbar_init();
  }
  pdl_wait();
  const PfPlan plan = pf_plan(a, gridDim.x);
  if (int(blockIdx.x) >= plan.nc) return;  // (nothing to share: before the TMEM is taken)
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (warp == kFindWarp && lane == 0) tma_prefetch_map(&map);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  PfGuard* guard = &sh.guard;

  // Whether there is a next item (by a whole warp).
  auto next_item = [&](const PfRing<kPfItems>& ring) {
    const bool came = pf_wait(&sh.item_full[ring.at], ring.phase, guard);
    if (!__all_sync(0xffffffffu, came)) return false;
    return sh.item[ring.at].stop == 0;
  };

  // What the registers are moved for has to stand in a branch of its own.
  if (warp < kPfSoftmax / 32) {
    setmaxnreg_inc<kPfSoftmaxRegs>();
    // ---------------------------------------------------------------- softmax
    const int g = warp >> 2, row = tid & 127;
    const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + g * 128, o_addr = lane_addr + 256 + g * 128;
    PfRing<kPfItems> ring;
    uint32_t s_phase = 0, o_phase = 0, told_phase = 0;
    int seq = 0, count = 0;  // key tiles, M tiles of the items before
    bool begun = false;
    while (next_item(ring)) {
      PfItem& it = sh.item[ring.at];
      if (!begun) {
        for (int m = 0; m <= it.two; ++m) {
          pf_prepare<D>(a, plan, it, m * kPfTile, q_s + m * kWide, sh.factor[m], (warp + 4 * m) & 7,
                        kPfSoftmax / 32);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full[m]);
        }
        begun = true;
      }
      const int two = it.two, tiles = it.t1 - it.t0;
      const bool begins = it.t0 == 0;
      const int turns = two ? tiles : (tiles + 1 - g) / 2;
      const int x0 = (two ? g * kPfTile : 0) + row;
      const int64_t query = pf_query(a, plan, it, x0);
      const float* factor = sh.factor[(count + (two ? g : 0)) % kPfFactors];
      const int seq0 = seq;
      seq += tiles;
      count += 1 + two;
      const bool any = __any_sync(0xffffffffu, query >= 0);
      float c = 0.0f;
      float ref = -INFINITY, l = 0.0f;  // ref: a whole number, in log2 units
      bool stop = false;
#pragma unroll 1
      for (int i = 0; i < turns; ++i) {
        const bool came = pf_wait(&sh.s_full[g], s_phase, guard);
        s_phase ^= 1;
        stop = !__all_sync(0xffffffffu, came);
        if (stop) break;
        tc_fence_after();
        if (i == 0) c = factor[row];  // (the products waited for the queries)
        const PfTile& tile = sh.tile[(seq0 + (two ? i : 2 * i + g)) % NT];
        if (any) {
          // All of a query's scores at once: a load takes 500 to 800 cycles while products run.
          // (32 at a time, in a loop of a fifth of the code, the softmax took 3400 instead of
          // 1900 cycles.)
          float z[128];
#pragma unroll
          for (int y = 0; y < 4; ++y) tmem_ld32(s_addr + 32 * y, z + 32 * y);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 4; ++y) tmem_tie32(z + 32 * y);
          if (tile.below) {  // a scale below zero: the maximum of a part is not taken before it
#pragma unroll
            for (int x = 0; x < 128; ++x) z[x] *= tile.raw_ks[x / kPfPart];
          }
          float top = -INFINITY;
#pragma unroll
          for (int y = 0; y < kPfParts; ++y) {
            const float* v = z + kPfPart * y;
            float m0 = max3(v[0], v[1], v[2]), m1 = max3(v[3], v[4], v[5]);
            m0 = max3(m0, v[6], v[7]);
            m1 = max3(m1, v[8], v[9]);
            m0 = max3(m0, v[10], v[11]);
            m1 = max3(m1, v[12], v[13]);
            top = fmaxf(top, max3(m0, m1, fmaxf(v[14], v[15])) * tile.ks[y]);
          }
          top *= c;
          const bool moves = __any_sync(0xffffffffu, top > ref);
          float down = 1.0f;
          if (moves) {
            // The references move, by whole binades and some more, as in rows of a warp the
            // largest score would else grow at some row in every other tile.
            const float to = top > ref ? ceilf(top) + kPfHeadroom : ref;
            down = to == -INFINITY ? 1.0f : ex2_approx(ref - to);
            ref = to;
            l *= down;
          }
          const float minus = ref == -INFINITY ? 0.0f : -ref;
          float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
          for (int y = 0; y < kPfParts; ++y) {
            const float by = tile.ks[y] * c;
            const float2 by2 = make_float2(by, by), less2 = make_float2(minus, minus);
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < kPfPart; x += 2) {
              const float2 e =
                  __ffma2_rn(make_float2(z[16 * y + x], z[16 * y + x + 1]), by2, less2);
              const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
              if (x & 2) sum1 = __fadd2_rn(sum1, p);
              else sum0 = __fadd2_rn(sum0, p);
              const __nv_bfloat162 v = __floats2bfloat162_rn(p.x, p.y);
              w[x / 2] = *reinterpret_cast<const uint32_t*>(&v);
            }
            tmem_st8(s_addr + 8 * y, reinterpret_cast<const float*>(w));
          }
          l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
          // The output before this tile is done: its products were issued before the scores.
          if (moves && i > 0) pf_rescale<D>(o_addr, down);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&sh.p_full[g]);
        if (row == 0) *reinterpret_cast<volatile int*>(&sh.guard.beat[g]) = seq0 + i + 1;
      }
      // released only now: the factors' places are counted by items
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[ring.at]);
      ring.next();
      if (stop) break;
      if (turns == 0) continue;
      // ------------------------------------------------------------ the piece's end
      pf_wait(&sh.o_full[g], o_phase, guard);
      o_phase ^= 1;
      const bool both = !two && tiles > 1;
      float m = ref;
      float mine = 1.0f, other = 0.0f;
      if (both) {
        sh.part[g][row] = make_float2(m, l);
        mbar_arrive(&sh.told[g]);
        pf_wait(&sh.told[g ^ 1], told_phase, guard);
        const float2 st = sh.part[g ^ 1][row];
        const float mn = fmaxf(m, st.x), base = mn == -INFINITY ? 0.0f : mn;
        mine = ex2_approx(m - base);
        other = ex2_approx(st.x - base);
        l = l * mine + st.y * other;
        m = mn;
      }
      if (__any_sync(0xffffffffu, guard->aborted())) break;
      tc_fence_after();
      if (any) {
        const int64_t at = begins ? query : int64_t(blockIdx.x) * 256 + x0;
        float* to = (begins ? a.parts[0] : a.mid) + (query < 0 ? 0 : at) * D;
        if (query >= 0 && (!both || g == 0))
          (begins ? a.stats[0] : a.mid_stats)[at] = make_float2(m, l);
        // with both groups' parts each takes half of the numbers
        const int y0 = both ? g * (D / 2) : 0, y1 = both ? y0 + D / 2 : D;
#pragma unroll 1
        for (int y = y0; y < y1; y += 32) {
          float o[32], o2[32];
          tmem_ld32(o_addr + y, o);
          // (without a part of the other group: twice its own, other 0)
          tmem_ld32(lane_addr + 256 + (both ? g ^ 1 : g) * 128 + y, o2);
          tmem_wait_ld();
          tmem_tie32(o);
          tmem_tie32(o2);
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = o[x] * mine + o2[x] * other;
          if (query >= 0) {
#pragma unroll
            for (int x = 0; x < 32; x += 8) store8(to + y + x, o + x);
          }
        }
      }
      tc_fence_before();
      if (both) {
        mbar_arrive(&sh.read[g ^ 1]);
        pf_wait(&sh.read[g], told_phase, guard);
        told_phase ^= 1;
        if (__any_sync(0xffffffffu, guard->aborted())) break;
      }
    }
    if (row == 0) *reinterpret_cast<volatile int*>(&sh.guard.done[g]) = 1;
  } else if (warp < kMmaWarp) {
    setmaxnreg_dec<kPfLoadRegs>();
    // ---------------------------------------------------------------- values
    // From the codes in shared memory to bf16. (Read into registers from global memory, the
    // code of two tiles in flight was four times as long, and the instruction cache too small.)
    constexpr int kPerKey = D / 16;              // 16-byte chunks of a key's codes
    constexpr int kAtOnce = 32 / kPerKey;        // keys of a warp's step
    constexpr int kSteps = kPfTile * kPerKey / kPfLoad;
    constexpr int kKeyStep = kPfTile / kSteps;   // from step to step: a part, or two
    static_assert(kKeyStep % kPfPart == 0, "a lane's keys are in the same place of their parts");
    const int lw = warp - kPfSoftmax / 32;
    // a quarter of the warp writes two keys that are not 8 apart: no bank twice
    const int chunk = D == 128 ? (lane & 3) + 4 * (lane >> 3 & 1) : lane & 3;
    const int key0 = lw * kAtOnce + (D == 128 ? (lane >> 2 & 1) + 2 * (lane >> 4) : lane >> 2);
    // (a lane's keys are multiples of 8 apart: the swizzles are the same)
    const uint32_t from = pf_place8<D>(key0, chunk);
    const uint32_t place0 = pf_place(key0, 2 * chunk), place1 = pf_place(key0, 2 * chunk + 1);
    PfRing<RS> rr;
    PfRing<VS> vr;
    for (;; rr.next(), vr.next()) {
      bool came = pf_wait(&sh.raw_full[rr.at], rr.phase, guard);
      const int what = sh.raw_tile[rr.at];
      came = came && what >= 0 && pf_wait(&sh.v_empty[vr.at], vr.phase ^ 1, guard);
      if (!__all_sync(0xffffffffu, came)) break;
      const PfTile& t = sh.tile[what];
      const uint8_t* raw = raw_s + rr.at * kCode + from;
      uint8_t* to = sm + vr.at * kWide;
      const bool plain = t.plain_v;
      const int valid = t.valid;
#pragma unroll 2
      for (int i = 0; i < kSteps; ++i) {
        const int key = key0 + i * kKeyStep, part = key / kPfPart;
        uint4 v = *reinterpret_cast<const uint4*>(raw + i * kKeyStep * D);
        if (!(valid >> part & 1)) v = make_uint4(0u, 0u, 0u, 0u);  // not copied
        const float scale = t.vs[part];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t r[8];
        // a code that is no number (all ones but the sign) would become 480 below
        uint32_t none = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) none |= (w[y] & 0x7f7f7f7fu) + 0x01010101u;
        if (plain && !(none & 0x80808080u)) {
          // the product with scale * 2^120 is exact
          const uint32_t up = ((__float_as_uint(scale) >> 23) + 120 << 7) * 0x00010001u;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            r[2 * y] = mul_bf16x2(e4m3_in_bf16<0x9180u>(w[y]), up);
            r[2 * y + 1] = mul_bf16x2(e4m3_in_bf16<0xb3a2u>(w[y]), up);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float f[4];
            e4m3x4_to_f32(w[y], f);
#pragma unroll
            for (int z = 0; z < 4; ++z) {  // nor may a product overflow; a NaN stays
              f[z] *= scale;
              f[z] = f[z] > kMaxBf16 ? kMaxBf16 : f[z] < -kMaxBf16 ? -kMaxBf16 : f[z];
            }
            const __nv_bfloat162 v0 = __floats2bfloat162_rn(f[0], f[1]);
            const __nv_bfloat162 v1 = __floats2bfloat162_rn(f[2], f[3]);
            r[2 * y] = *reinterpret_cast<const uint32_t*>(&v0);
            r[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&v1);
          }
        }
        *reinterpret_cast<uint4*>(to + place0 + i * kKeyStep * 128) =
            make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(to + place1 + i * kKeyStep * 128) =
            make_uint4(r[4], r[5], r[6], r[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.raw_empty[rr.at]);
        mbar_arrive(&sh.v_full[vr.at]);
      }
    }
  } else {
    setmaxnreg_dec<kPfOtherRegs>();
    if (warp == kWalkWarp) {
    // ---------------------------------------------------------------- work list, queries
    const int64_t u_end = pf_share(plan, blockIdx.x + 1);
    int64_t u = pf_share(plan, blockIdx.x);
    int lo = 0, hi = plan.NG - 1;  // the last group that begins at or before u
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (plan.prefix[m] <= u) lo = m;
      else hi = m - 1;
    }
    int e = lo;
    // the piece that begins at u, and u past it; stop at the end
    auto describe = [&]() {
      PfItem it = {};
      it.stop = 1;
      while (u < u_end && e < plan.NG) {
        const int64_t base = plan.prefix[e], len = plan.prefix[e + 1] - base;
        if (u >= base + len) {
          ++e;
          continue;
        }
        const int64_t per_h = len / a.H;
        const PrefixGroup g = plan.groups[e];
        it.row = g.row;
        it.entry = g.entry;
        const int64_t nq = int64_t(g.count) * a.T * a.G, tiles = g.tiles;
        const int64_t in = u - base, h = per_h > 0 ? in / per_h : a.H, in_h = in - h * per_h;
        if (tiles <= 0 || nq <= 0 || h >= a.H || it.row < 0 || it.row >= a.B)
          break;  // not a plan that was made here
        const int64_t qb = in_h / pf_item_units(kPfTwoUnits, tiles);
        const int w = nq - qb * 256 > 128 ? kPfTwoUnits : kPfOneUnits;
        const int64_t at = in_h - qb * pf_item_units(kPfTwoUnits, tiles),
                      stop = min(pf_item_units(w, tiles), at + (u_end - u));
        it.h = int(h);
        it.two = w == kPfTwoUnits;
        it.q0 = int(qb * 256);
        it.nq = int(min(nq - qb * 256, int64_t(256)));
        it.t0 = pf_cut(at, w);
        it.t1 = pf_cut(stop, w);
        u += stop - at;
        if (it.t0 < it.t1) {
          it.stop = 0;
          break;
        }
      }
      return it;
    };
    // Items are described as far ahead as there are places, whatever their queries wait for.
    // The first item's queries are the softmax warps' to prepare.
    PfRing<kPfItems> ring, qitem;
    PfRing<kPfQueries> qring;
    int ahead = 0, m = 0;  // items whose queries are not there; M tile of the first of them
    int count = 0;         // M tiles before it
    bool ended = false, begun = false;
    // Between its work the warp watches: tiles have to be done.
    const volatile PfGuard* watch = &sh.guard;
    uint64_t since = global_ns();
    int seen = 0;
    while (!ended || ahead > 0 || !watch->done[0] || !watch->done[1]) {
      if (__any_sync(0xffffffffu, guard->aborted())) break;
      const int beats = watch->beat[0] + watch->beat[1];
      if (beats != seen) since = global_ns();
      seen = beats;
      if (!ended && ahead < kPfItems &&
          __all_sync(0xffffffffu, mbar_test_wait(&sh.item_empty[ring.at], ring.phase ^ 1))) {
        const PfItem it = describe();
        if (lane == 0) {
          sh.item[ring.at] = it;
          mbar_arrive(&sh.item_full[ring.at]);
        }
        __syncwarp();
        ring.next();
        ended = it.stop;
        if (!begun) {
          qitem.next();
          for (; !ended && count <= it.two; ++count) qring.next();
        } else if (!ended) {
          ++ahead;
        }
        begun = true;
        continue;
      }
      if (ahead > 0 &&
          __all_sync(0xffffffffu, mbar_test_wait(&sh.q_empty[qring.at], qring.phase ^ 1))) {
        const PfItem& it = sh.item[qitem.at];
        const int two = it.two;
        pf_prepare<D>(a, plan, it, m * kPfTile, q_s + qring.at * kWide,
                      sh.factor[count % kPfFactors], 0, 1);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&sh.q_full[qring.at], kPfSoftmax / 32);
        qring.next();
        ++count;
        if (++m > two) {
          m = 0;
          --ahead;
          qitem.next();
        }
        continue;
      }
      // nothing has a place yet
      __nanosleep(1000);
      if (global_ns() - since > a.wait_ns) {
        *reinterpret_cast<volatile int*>(&guard->abort) = 1;
        if (a.err) atomicOr(a.err, SPEC_DERR_TIMEOUT);
      }
    }
    } else if (warp == kFindWarp) {
    // ---------------------------------------------------------------- where the tiles are
    // Four tiles at a time, a lane a part: ids, then scales. Copies of K and V are started here, in
    // the order in which the products take them: those go through steps, in each of which first
    // group 0, then group 1 takes the output of its tile before (V), then the scores of the next
    // (K).
    PfRing<kPfItems> ring;
    PfRing<RS> rr;
    PfRing<KS> kr;
    // slots that have been copied to, and the phase of the last copy (V's from bit 16)
    uint32_t started = 0, started_phase = 0;
    bool ok = true, half = false;  // half: group 1 has not had its turn in the step
    int seq = 0, pend0 = -1, pend1 = -1;
    // V of a tile; -1: no more
    auto values = [&](int what) {
      const bool came = ok && pf_wait(&sh.raw_empty[rr.at], rr.phase ^ 1, guard);
      ok = __all_sync(0xffffffffu, came);
      if (!ok) return;
      if (what < 0) {
        if (lane == 0) {
          sh.raw_tile[rr.at] = what;
          mbar_arrive(&sh.raw_full[rr.at]);
        }
        return;
      }
      const PfTile& tile = sh.tile[what];
      if (lane == 0) {
        sh.raw_tile[rr.at] = what;
        mbar_arrive_expect_tx(&sh.raw_full[rr.at], __popc(tile.valid) * kPfPart * D);
      }
      __syncwarp();
      if (lane < kPfParts && tile.plane[lane] >= 0)
        tma_tile_3d(raw_s + rr.at * kCode + lane * kPfPart * D, &map, 0, tile.in_block[lane],
                    tile.plane[lane], &sh.raw_full[rr.at]);
      started |= 0x10000u << rr.at;
      started_phase = (started_phase & ~(0x10000u << rr.at)) | rr.phase << (16 + rr.at);
      rr.next();
    };
    auto values0 = [&]() {
      if (pend0 >= 0) values(pend0);
      pend0 = -1;
    };
    auto values1 = [&]() {
      if (pend1 >= 0) values(pend1);
      pend1 = -1;
      half = false;
    };
    while (ok && next_item(ring)) {
      const PfItem it = sh.item[ring.at];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[ring.at]);
      ring.next();
      const int row = it.row;
      for (int t = it.t0; t < it.t1 && ok;) {
        const int many = min(4, it.t1 - t);
        const int pos = t * kPfTile + (lane >> 3) * kPfTile + (lane & 7) * kPfPart;
        const bool on = lane >> 3 < many;
        const int j = pos / a.bs, in_block = pos - j * a.bs;
        int id = -1;
        if (on && j < a.MB) id = a.bt[int64_t(row) * a.MB + j];
        int plane = -1;
        float ks = 1.0f, vs = 1.0f;
        if (on) {
          if (id >= 0 && id < a.NB) {
            const float* at = a.scales + id * a.block_scales + it.h;
            ks = at[0];
            vs = at[a.H];
            plane = id * a.planes_per_block + a.plane0 + it.h;
            // values that are no numbers: zeros, and their keys are NaN
            if (!(fabsf(vs) <= FLT_MAX)) {
              vs = 0.0f;
              ks = __uint_as_float(0x7fc00000u);
            }
          } else {
            // keys that cannot be read: their queries' outputs become NaN
            ks = __uint_as_float(0x7fc00000u);
            if (a.err) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
          }
        }
        const uint32_t vu = __float_as_uint(vs);
        const uint32_t k_below = __ballot_sync(0xffffffffu, ks < 0.0f),
                       v_plain = __ballot_sync(0xffffffffu, (vu & 0x807fffffu) == 0 &&
                                                                vu >> 23 >= 27 && vu >> 23 <= 134);
#pragma unroll 1
        for (int x = 0; x < many && ok; ++x, ++t, ++seq) {
          const int g = it.two ? 0 : (t - it.t0) & 1, at = seq % NT;
          if (g == 0) {
            if (half) values1();
            values0();
          } else {
            values1();
          }
          // the test of a wait that runs out: these keys never come
          if (row == a.stall_row) ok = false;
          const bool came = ok && pf_wait(&sh.k_empty[kr.at], kr.phase ^ 1, guard);
          ok = __all_sync(0xffffffffu, came);
          if (!ok) break;
          const bool mine = lane >> 3 == x;
          const uint32_t valid = __ballot_sync(0xffffffffu, mine && plane >= 0);
          if (mine) {
            PfTile& tile = sh.tile[at];
            tile.plane[lane & 7] = plane < 0 ? -1 : plane + a.H;
            tile.in_block[lane & 7] = in_block;
            const bool below = k_below >> 8 * x & 255u;
            tile.ks[lane & 7] = below ? 1.0f : ks;
            tile.raw_ks[lane & 7] = ks;
            tile.vs[lane & 7] = vs;
            if ((lane & 7) == 0) {
              tile.valid = valid >> 8 * x & 255u;
              tile.below = below;
              tile.plain_v = (v_plain >> 8 * x & 255u) == 255u;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[kr.at], __popc(valid) * kPfPart * D);
          started |= 1u << kr.at;
          started_phase = (started_phase & ~(1u << kr.at)) | kr.phase << kr.at;
          __syncwarp();
          if (mine && plane >= 0)
            tma_tile_3d(k_s + kr.at * kCode + (lane & 7) * kPfPart * D, &map, 0, in_block, plane,
                        &sh.k_full[kr.at]);
          kr.next();
          if (g == 1) {
            pend1 = at;
          } else {
            pend0 = at;
            if (it.two) values1();
            else half = true;
          }
        }
      }
    }
    if (half) values1();
    values0();
    values1();
    values(-1);
    // a wait has run out: copies in flight end before the CTA does
    if (__any_sync(0xffffffffu, guard->aborted())) {
      for (int i = 0; i < KS; ++i)
        if (started >> i & 1u) mbar_wait(&sh.k_full[i], started_phase >> i & 1u);
      for (int i = 0; i < RS; ++i)
        if (started >> (16 + i) & 1u) mbar_wait(&sh.raw_full[i], started_phase >> (16 + i) & 1u);
    }
    } else {
    // ---------------------------------------------------------------- products
    // A warp a group: the output of a tile, then the next scores, which take the place of that
    // tile's probabilities. They take turns, so that one group's products run while the other's
    // softmax does; as issuing lasts as long as the products, one warp for both would leave the
    // tensor cores idle while it waits and prepares. All waits of a turn are made at once, a
    // lane each. Tiles that only the other group takes are waited for and released too, so that
    // no warp falls two rounds behind in a ring, where the parity of its waits would mislead it.
    // The whole warp goes through the loops, so that what the products need is known to be
    // uniform; one lane issues them.
    constexpr uint32_t kSwz = D == 128 ? 2 : 4;  // K and queries: 128- or 64-byte swizzle
    constexpr uint32_t idesc_s = tc_idesc(0, 0, 0, 0, kPfTile, kPfTile);
    constexpr uint32_t idesc_o = tc_idesc(1, 1, 0, 1, kPfTile, D);
    auto uniform = [](uint32_t x) { return __reduce_max_sync(0xffffffffu, x); };
    const int g = uniform(warp) - kMmaWarp;
    const uint32_t s_at = uniform(tmem) + g * 128, o_at = s_at + 256;
    const uint64_t k0 = tc_desc(smem_u32(k_s), 16, 8 * D, kSwz);
    const uint64_t v0 = tc_desc(smem_u32(sm), kPfTile * 128, 1024, 2);
    const uint32_t k_hi = uint32_t(k0 >> 32), v_hi = uint32_t(v0 >> 32), k_lo = uint32_t(k0),
                   v_lo = uint32_t(v0), q_lo = uint32_t(tc_desc(smem_u32(q_s), 16, 8 * D, kSwz));
    PfRing<kPfItems> ring;
    PfRing<kPfQueries> qring;
    PfRing<KS> kr;
    PfRing<VS> vr;
    PfRing<kPfTurns> turn;  // group 1: the one of this step; group 0: of the step before
    uint32_t p_phase = 0;
    // An output that waits, whether it is of its item's first and last tile, and of a V tile
    // that both take. The other group's V and K that are to be released.
    bool pending = false, first = false, last = false, shared = false, begun = false;
    bool pend0 = false, pend1 = false, other_v = false, other_k = false;
    int s_turn = 0;  // step, round and round
    bool ok = true;  // no wait has run out
    // steps of items, and one after the last for the outputs that wait
    for (bool more = true; more && ok;) {
      ok = __all_sync(0xffffffffu, pf_wait(&sh.item_full[ring.at], ring.phase, guard));
      if (!ok) break;
      const PfItem& it = sh.item[ring.at];
      more = !uniform(it.stop);
      const int two = more ? uniform(it.two) : 0, tiles = more ? uniform(it.t1 - it.t0) : 0;
      __syncwarp();
      if (more && lane == 0) mbar_arrive(&sh.item_empty[ring.at]);
      ring.next();
      const PfRing<kPfQueries> q0 = qring;
      if (more) qring.next();
      const PfRing<kPfQueries> q1 = two ? qring : q0;
      if (two) qring.next();
      const PfRing<kPfQueries> q = g ? q1 : q0, q_other = g ? q0 : q1;
      const int by = two ? 1 : 2, steps = !more ? 1 : (tiles + by - 1) / by;
      int x = two ? 0 : g;  // this group's next tile of the item
#pragma unroll 1
      for (int s = 0; s < steps && ok; ++s, x += by) {
        if (g == 1) {  // group 0's of this step come before its own
          other_v = pend0 && !shared;
          other_k = more && !two;
        }
        const PfRing<VS> v_other = vr;
        if (other_v) vr.next();
        const PfRing<KS> k_other = kr;
        if (other_k) kr.next();
        const bool on = x < tiles, ends = x + by >= tiles;
        // The output and the scores are issued together, but an item's first scores wait for its
        // queries, and the output before them does not wait for that.
        bool out = pending, waits = begun || g == 1;  // for its turn
#pragma unroll 1
        for (int r = out && s == 0 ? 0 : 1; r < 2 && ok; ++r) {
          const bool now = r == 1, score = now && on;
          {
            uint64_t* bar = &sh.p_full[g];
            uint32_t phase = p_phase;
            bool need = out;
            if (lane == 1) bar = &sh.v_full[vr.at], phase = vr.phase;
            if (lane == 2) bar = &sh.k_full[kr.at], phase = kr.phase, need = score;
            if (lane == 3) bar = &sh.q_full[q.at], phase = q.phase, need = now && more && s == 0;
            if (lane == 4)
              bar = &sh.q_full[q_other.at], phase = q_other.phase, need = now && two && s + 1 == steps;
            if (lane == 5) bar = &sh.v_full[v_other.at], phase = v_other.phase, need = now && other_v;
            if (lane == 6) bar = &sh.k_full[k_other.at], phase = k_other.phase, need = now && other_k;
            if (lane == 7) bar = &sh.turn[g ^ 1][turn.at], phase = turn.phase, need = waits;
            need = need && lane < 8;
            ok = __all_sync(0xffffffffu, !need || pf_wait(bar, phase, guard));
          }
          if (!ok) break;
          tc_fence_after();
          const uint32_t v_desc = v_lo + vr.at * (kWide / 16), k_desc = k_lo + kr.at * (kCode / 16),
                         q_desc = q_lo + q.at * (kWide / 16);
          if (elect_one()) {
            if (out) {
#pragma unroll
              for (int y = 0; y < kPfTile / 16; ++y)
                pf_mma_o(o_at, s_at + 8 * y, v_desc + 128 * y, v_hi, idesc_o, y > 0 || !first);
            }
            if (score) {
              // both terms of the queries into one sum
#pragma unroll
              for (int z = 0; z < D / 32; ++z) {
                pf_mma_s(s_at, q_desc + 2 * z, k_desc + 2 * z, k_hi, idesc_s, z > 0);
                pf_mma_s(s_at, q_desc + kCode / 16 + 2 * z, k_desc + 2 * z, k_hi, idesc_s, true);
              }
              tc_commit(&sh.s_full[g]);
            }
            if (now) mbar_arrive(&sh.turn[g][s_turn]);
            if (out) {
              tc_commit(&sh.v_empty[vr.at]);
              if (last) tc_commit(&sh.o_full[g]);
            }
            if (score) {
              tc_commit(&sh.k_empty[kr.at]);
              if (ends) tc_commit(&sh.q_empty[q.at]);  // the item's last scores of these queries
            }
            if (now) {
              if (other_v) mbar_arrive(&sh.v_empty[v_other.at]);
              if (other_k) mbar_arrive(&sh.k_empty[k_other.at]);
              if (two && s + 1 == steps) mbar_arrive(&sh.q_empty[q_other.at]);
              if (!two && more && s == 0 && g >= tiles) mbar_arrive(&sh.q_empty[q.at]);
            }
          }
          __syncwarp();
          if (out) {
            p_phase ^= 1;
            vr.next();
          }
          if (score) kr.next();
          out = waits = false;
        }
        if (g == 1 || begun) turn.next();
        if (++s_turn == kPfTurns) s_turn = 0;
        if (g == 0) {  // group 1's of this step come after its own
          other_v = pend1 && !shared;
          other_k = !two && 2 * s + 1 < tiles;
        }
        pend0 = more;
        pend1 = two || 2 * s + 1 < tiles;
        pending = on;
        first = s == 0;
        last = ends;
        shared = two;
        begun = true;
      }
    }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (sh.guard.abort) {
    // What has been issued ends before the CTA's memory is another's. A commit stands for the
    // products of its own thread: it has to come from the lane that issued them.
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      if (elect_one()) tc_commit(&sh.drained);
      __syncwarp();
      mbar_wait(&sh.drained, 0);
      __syncwarp();  // the warp frees the TMEM as one
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
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

template <int D>
int launch_shape(const PfArgs& a, const CUtensorMap& map, int ctas, cudaStream_t st) {
  auto kern = kv_prefix_attention_kernel<D>;
  constexpr size_t smem = PfShape<D>::kBytes;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kern, smem, done) != SPEC_OK) return SPEC_ECUDA;
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(kPfThreads), smem, st, a, map);
}

}  // namespace

int launch_pf_attention(const PfArgs& a, const void* pool_base, int64_t planes, int ctas,
                        void* stream) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return SPEC_ECUDA;
  CUtensorMap map;
  const cuuint64_t dims[3] = {cuuint64_t(a.D), cuuint64_t(a.bs), cuuint64_t(planes)};
  const cuuint64_t strides[2] = {cuuint64_t(a.D), cuuint64_t(a.bs) * a.D};
  const cuuint32_t box[3] = {cuuint32_t(a.D), kPfPart, 1};
  const cuuint32_t step[3] = {1, 1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool_base), dims, strides, box,
          step, CU_TENSOR_MAP_INTERLEAVE_NONE,
          a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SPEC_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.D == 128 ? launch_shape<128>(a, map, ctas, st) : launch_shape<64>(a, map, ctas, st);
}

}  // namespace sv
