// The prefix attention's products and softmax (kv_prefix.cuh says what is computed and
// how the work is split).
//
// With the queries of many rows there are enough of them to be the M operand:
//   S [128 queries x 128 keys]  = Q [128 x D] * K^T          bf16 x bf16, fp32 sums in TMEM
//   O [128 queries x D]        += P [128 x 128] * V          P bf16 in TMEM, V bf16
// A thread owns a query: no maximum or sum crosses lanes. Two M tiles per CTA take turns, so
// that the tensor core works for one while the other's softmax runs: with more than 128
// queries they are two halves of the block and share each key tile, else both hold the same
// queries and take the key tiles by turns, each with a part of its own, added at the end.
//
// The cached codes are read by ordinary loads, widened to bf16 on the way to shared memory:
// a code is exact in bf16 (its exponent and fraction moved to their place, then one product
// with scale * 2^120, exact for the powers of two that appending leaves; other scales take a
// path that multiplies in fp32 and rounds once to bf16). A copy by TMA would pass the codes
// through shared memory once more, whose bandwidth the products need: of its 128 bytes a
// cycle S takes 128 and O 64 while each runs.
// P is rounded to bf16 (2^-9 relative, as the output); the sums l take it in fp32 before.
//   Softmax: a row's reference is the largest z_j so far, moved only when a later one
// exceeds it by 2^8; then O and l are rescaled.
//
// Roles: two groups of 4 softmax warps, 4 loading warps, a warp that issues the products,
// and one that walks the work list and copies the queries: 14 warps, so that no quarter of
// the SM has more than 4 and a thread may have 128 registers. One CTA per SM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kv_prefix.cuh"
#include "launch_util.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace sv {

constexpr int kPfSoftmax = 256, kPfLoad = 128;
constexpr int kPfThreads = kPfSoftmax + kPfLoad + 64;
constexpr int kPfItems = 4;     // items described at a time
constexpr int kPfQueries = 3;   // M tiles of queries held at a time
constexpr float kPfSlack = 8.0f;  // binades by which keys may exceed the reference

struct PfGuard {
  uint64_t limit_ns;
  int abort;
  __device__ __forceinline__ bool aborted() const {
    return *reinterpret_cast<const volatile int*>(&abort) != 0;
  }
};

// One piece of an item.
struct PfItem {
  int stop;       // no more items
  int two;        // two M tiles (else one, and its key tiles by turns)
  int row;        // whose table the keys come from
  int h;
  int t0, t1;     // tiles of the item
  int tile0;      // the item's first tile in the row
  int L, n, end;  // own keys: committed, new, end. A prefix: all keys are seen, end past them
  int own;        // 0 prefix, 1 own keys
  int q0, nq;     // first query of the block in its entry, queries of the block
  int entry;      // prefix: the group's first member
};

struct PfShared {
  PfItem item[kPfItems];
  float2 part[2][kPfTile];  // what one group tells the other at the end of an item
  uint64_t item_full[kPfItems], item_empty[kPfItems];
  uint64_t q_full[kPfQueries], q_empty[kPfQueries];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2], p_full[2], o_full[2], told[2], read[2], drained;
  uint32_t tmem;
  PfGuard guard;
};

template <int D>
struct PfShape {
  static constexpr int kTileBytes = kPfTile * D * 2;  // K, V or an M tile of queries
  static constexpr int kSlots = D == 128 ? 4 : 8;
  static constexpr size_t kBytes = size_t(kSlots + kPfQueries) * kTileBytes + sizeof(PfShared);
  static_assert(kBytes <= 227 * 1024, "one CTA per SM");
};

// Bounded waits, as in the other attention kernel: once one has run out, all return at once
// and every role leaves its loop; the error bit is set.
__device__ __noinline__ void pf_wait_long(uint64_t* bar, uint32_t parity, PfGuard* guard,
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
__device__ __forceinline__ void pf_wait(uint64_t* bar, uint32_t parity, PfGuard* guard,
                                        int32_t* err) {
  if (!mbar_try_wait(bar, parity, kSuspendNs)) pf_wait_long(bar, parity, guard, err);
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

// Where an M tile, K or V holds 16-byte chunk c (of D / 8) of row r: halves of 64 numbers,
// rows of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t pf_place(int r, int c) {
  return uint32_t((c >> 3) * (kPfTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The query of index qi of an entry: its row of q and out ([B, T, H * G]), or -1; t: its query.
__device__ __forceinline__ int64_t pf_query(const PfArgs& a, const PfPlan& p, const PfItem& it,
                                            int x, int& t) {
  t = 0;
  if (x >= it.nq) return -1;
  const int R = a.T * a.G, qi = it.q0 + x;
  int b = it.row, r = qi;
  if (!it.own) {
    const int e = qi / R;
    r = qi - e * R;
    b = it.entry + e < p.NE ? p.members[it.entry + e] : -1;
    if (b < 0 || b >= a.B) return -1;
  }
  t = r / a.G;
  return (int64_t(b) * a.T + t) * a.H * a.G + it.h * a.G + (r - t * a.G);
}

// Sixteen codes, where the call stands (ahead of their use), not kept in L1.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// D[tmem] (+)= A B in bf16, K = 16; one thread issues. A in shared memory or in TMEM.
__device__ __forceinline__ void tc_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                               bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}

// ------------------------------------------------------------------ the order of the tiles
// The products go through steps; in each, first group 0, then group 1, takes the output of its
// tile before (V), then the scores of the next (K). The loading warps follow the same order:
// phases 0 to 3 of a step are V and K of group 0, V and K of group 1.
struct PfTile {
  int row, h, p0, end, own;  // keys [p0, p0 + 128) of the row's table, those past `end` zero
  bool v;
};

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) kv_prefix_attention_kernel(const PfArgs a) {
  using S = PfShape<D>;
  constexpr int NS = S::kSlots, kTile = S::kTileBytes;
  constexpr int kMmaWarp = (kPfSoftmax + kPfLoad) / 32, kWalkWarp = kMmaWarp + 1;
  extern __shared__ __align__(1024) uint8_t sm[];  // ring of K and V, queries, the rest
  uint8_t* q_s = sm + NS * kTile;
  PfShared& sh = *reinterpret_cast<PfShared*>(q_s + kPfQueries * kTile);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < kPfItems; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_empty[i], (kPfSoftmax + kPfLoad) / 32 + 1);
    }
    for (int i = 0; i < kPfQueries; ++i) {
      mbar_init(&sh.q_full[i], 32);
      mbar_init(&sh.q_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.kv_full[i], kPfLoad / 32);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.told[i], 128);
      mbar_init(&sh.read[i], 128);
    }
    mbar_init(&sh.drained, 1);
    sh.guard.abort = 0;
    sh.guard.limit_ns = a.wait_ns;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  const PfPlan plan = pf_plan(a, gridDim.x);
  const bool work = int(blockIdx.x) < plan.nc;
  PfGuard* guard = &sh.guard;

  // The next item, as the other roles take it; false: no more.
  auto next_item = [&](PfRing<kPfItems>& ring, PfItem& it) {
    pf_wait(&sh.item_full[ring.at], ring.phase, guard, a.err);
    if (__any_sync(0xffffffffu, guard->aborted())) return false;
    it = sh.item[ring.at];
    return it.stop == 0;
  };

  if (work && warp == kWalkWarp) {
    // ---------------------------------------------------------------- work list, queries
    const int64_t u_end = pf_share(plan, blockIdx.x + 1);
    int64_t u = pf_share(plan, blockIdx.x);
    const int entries = plan.NG + a.B;
    int lo = 0, hi = entries - 1;  // the last entry that begins at or before u
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (plan.prefix[m] <= u) lo = m;
      else hi = m - 1;
    }
    int e = lo;
    PfRing<kPfItems> ring;
    PfRing<kPfQueries> qring;
    for (;;) {
      PfItem it = {};
      it.stop = 1;
      while (u < u_end && e < entries) {
        const int64_t base = plan.prefix[e], len = plan.prefix[e + 1] - base;
        if (u >= base + len) {
          ++e;
          continue;
        }
        int64_t nq;
        int tiles;
        if (e < plan.NG) {
          const PfGroup g = plan.groups[e];
          it.row = g.row;
          it.entry = g.entry;
          nq = int64_t(g.count) * a.T * a.G;
          tiles = g.tiles;
          it.own = 0;
          it.tile0 = 0;
          it.L = it.end = tiles * kPfTile;
          it.n = 0;
        } else {
          const PfRow r = plan.rows[e - plan.NG];
          it.row = e - plan.NG;
          nq = int64_t(r.n) * a.G;
          tiles = r.tiles;
          it.own = 1;
          it.tile0 = r.skip;
          it.L = r.L;
          it.n = r.n;
          it.end = r.L + r.n;
        }
        const int64_t per_h = pf_units(nq, tiles);
        const int64_t in = u - base, h = per_h > 0 ? in / per_h : a.H, in_h = in - h * per_h;
        if (tiles <= 0 || nq <= 0 || h >= a.H || it.row < 0 || it.row >= a.B)
          break;  // not a plan that was made here
        const int64_t qb = in_h / (2 * int64_t(tiles));
        const int w = nq - qb * 256 > 128 ? 2 : 1;
        const int64_t at = in_h - qb * 2 * tiles, stop = min(int64_t(w) * tiles, at + (u_end - u));
        it.h = int(h);
        it.two = w == 2;
        it.q0 = int(qb * 256);
        it.nq = int(min(nq - qb * 256, int64_t(256)));
        it.t0 = int((at + w - 1) / w);
        it.t1 = int((stop + w - 1) / w);
        u += stop - at;
        if (it.t0 < it.t1) {
          it.stop = 0;
          break;
        }
      }
      pf_wait(&sh.item_empty[ring.at], ring.phase ^ 1, guard, a.err);
      if (__any_sync(0xffffffffu, guard->aborted())) break;
      if (lane == 0) {
        sh.item[ring.at] = it;
        mbar_arrive(&sh.item_full[ring.at]);
      }
      __syncwarp();
      ring.next();
      if (it.stop) break;
      for (int m = 0; m <= it.two; ++m) {
        pf_wait(&sh.q_empty[qring.at], qring.phase ^ 1, guard, a.err);
        if (__any_sync(0xffffffffu, guard->aborted())) break;
        uint8_t* to = q_s + qring.at * kTile;
        int64_t mine[kPfTile / 32];  // rows lane, lane + 32, ...
#pragma unroll
        for (int i = 0; i < kPfTile / 32; ++i) {
          int t;
          mine[i] = pf_query(a, plan, it, m * kPfTile + 32 * i + lane, t);
        }
        constexpr int kChunks = D / 8;  // of a row
#pragma unroll
        for (int i = 0; i < kPfTile / 32; ++i)
#pragma unroll 4
          for (int x = 0; x < kChunks; ++x) {
            const int c = x * 32 + lane, r = c / kChunks;  // r: of these 32 rows
            const int64_t row = __shfl_sync(0xffffffffu, mine[i], r);
            cp_async16(to + pf_place(32 * i + r, c % kChunks),
                       static_cast<const __nv_bfloat16*>(a.q) + (row < 0 ? 0 : row) * D +
                           c % kChunks * 8,
                       row >= 0);
          }
        cp_async_wait_all();
        fence_async_smem();
        mbar_arrive(&sh.q_full[qring.at]);
        qring.next();
      }
    }
  } else if (work && warp == kMmaWarp) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t idesc_s = tc_idesc(1, 1, 0, 0, kPfTile, kPfTile);
      constexpr uint32_t idesc_o = tc_idesc(1, 1, 0, 1, kPfTile, D);
      const uint64_t kv0 = tc_desc(smem_u32(sm), kPfTile * 128, 1024, 2);
      const uint64_t q0 = tc_desc(smem_u32(q_s), kPfTile * 128, 1024, 2);
      PfRing<kPfItems> ring;
      PfRing<kPfQueries> qring;
      PfRing<NS> kv;
      uint32_t p_phase[2] = {0, 0};
      bool pending[2] = {false, false}, first[2] = {}, last[2] = {}, shared[2] = {};
      int v_slot = 0;  // of a V tile that both groups take
      auto output = [&](int g) {
        if (!pending[g]) return;
        pending[g] = false;
        int slot = v_slot;
        if (!(shared[g] && g == 1)) {
          slot = v_slot = kv.at;
          pf_wait(&sh.kv_full[kv.at], kv.phase, guard, a.err);
          kv.next();
        }
        pf_wait(&sh.p_full[g], p_phase[g], guard, a.err);
        p_phase[g] ^= 1;
        if (guard->aborted()) return;
        tc_fence_after();
        const uint64_t v = kv0 + slot * (kTile / 16);
#pragma unroll
        for (int x = 0; x < kPfTile / 16; ++x)
          tc_mma_bf16_ts(tmem + 256 + g * 128, tmem + g * 128 + 8 * x, v + x * 128, idesc_o,
                         !(first[g] && x == 0));
        if (!(shared[g] && g == 0)) tc_commit(&sh.kv_empty[slot]);
        if (last[g]) tc_commit(&sh.o_full[g]);
      };
      for (;;) {
        pf_wait(&sh.item_full[ring.at], ring.phase, guard, a.err);
        if (guard->aborted()) break;
        const PfItem& it = sh.item[ring.at];
        if (it.stop) break;
        const int two = it.two, tiles = it.t1 - it.t0;
        mbar_arrive(&sh.item_empty[ring.at]);
        ring.next();
        const int steps = two ? tiles : (tiles + 1) / 2;
        int qs[2];
        uint32_t qp[2];
        qs[0] = qs[1] = qring.at;
        qp[0] = qp[1] = qring.phase;
        qring.next();
        if (two) {
          qs[1] = qring.at;
          qp[1] = qring.phase;
          qring.next();
        }
        int k_slot = 0;
        for (int s = 0; s < steps; ++s) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            output(g);
            const bool on = two || 2 * s + g < tiles;
            if (!on || guard->aborted()) continue;
            if (s == 0 && (two || g == 0)) pf_wait(&sh.q_full[qs[g]], qp[g], guard, a.err);
            if (!(two && g == 1)) {
              k_slot = kv.at;
              pf_wait(&sh.kv_full[kv.at], kv.phase, guard, a.err);
              kv.next();
            }
            if (guard->aborted()) continue;
            tc_fence_after();
            const uint64_t k = kv0 + k_slot * (kTile / 16), q = q0 + qs[g] * (kTile / 16);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const int at = (x & 3) * 2 + (x >> 2) * (kPfTile * 128 / 16);
              tc_mma_bf16(tmem + g * 128, q + at, k + at, idesc_s, x > 0);
            }
            if (!(two && g == 0)) tc_commit(&sh.kv_empty[k_slot]);
            tc_commit(&sh.s_full[g]);
            pending[g] = true;
            first[g] = s == 0;
            shared[g] = two;
            last[g] = two ? s + 1 == steps : 2 * (s + 1) + g >= tiles;
            // the item's last scores of these queries
            if (two ? s + 1 == steps : 2 * s + g + 1 == tiles) tc_commit(&sh.q_empty[qs[g]]);
          }
          if (guard->aborted()) break;
        }
      }
      output(0);
      output(1);
    }
    __syncwarp();
  } else if (work && warp < kPfSoftmax / 32) {
    // ---------------------------------------------------------------- softmax
    const int g = warp >> 2, row = tid & 127;
    const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + g * 128;
    PfRing<kPfItems> ring;
    uint32_t s_phase = 0, o_phase = 0, told_phase = 0;
    PfItem it;
    while (next_item(ring, it)) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_empty[ring.at]);
      ring.next();
      const int tiles = it.t1 - it.t0;
      const int turns = it.two ? tiles : (tiles + 1 - g) / 2;
      if (turns == 0) continue;
      int t;
      const int64_t query = pf_query(a, plan, it, (it.two ? g * kPfTile : 0) + row, t);
      // the new tokens that the query sees, as bits
      uint32_t bits = 0;
      if (it.own && query >= 0) {
        bits = a.tree ? a.tree[int64_t(it.row) * a.T + t] : (2u << t) - 1u;
        if (it.n < 32) bits &= (1u << it.n) - 1u;
      }
      const bool live = __any_sync(0xffffffffu, query >= 0);
      const float c = a.scale_log2;
      float ref = -INFINITY, l = 0.0f;  // ref: of the scores before they are scaled
      bool stop = false;
#pragma unroll 1
      for (int i = 0; i < turns; ++i) {
        const int p0 = (it.tile0 + it.t0 + (it.two ? i : 2 * i + g)) * kPfTile;
        pf_wait(&sh.s_full[g], s_phase, guard, a.err);
        s_phase ^= 1;
        stop = __any_sync(0xffffffffu, guard->aborted());
        if (stop) break;
        tc_fence_after();
        if (live) {
          const bool masked = p0 + kPfTile > it.L;
          auto hide = [&](float* z, int at) {  // of the 32 keys from position `at`
            const int d = at - it.L;
            const uint32_t m = d <= -32 ? ~0u : d < 0 ? (bits << -d) | ((1u << -d) - 1u)
                               : d < 32 ? bits >> d : 0u;
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(m >> x & 1u)) z[x] = -INFINITY;
          };
          float top = -INFINITY;
#pragma unroll
          for (int y = 0; y < 4; y += 2) {
            float z[64];
            tmem_ld32(s_addr + 32 * y, z);
            tmem_ld32(s_addr + 32 * y + 32, z + 32);
            tmem_wait_ld();
            if (masked) {
              hide(z, p0 + 32 * y);
              hide(z + 32, p0 + 32 * y + 32);
            }
            float m[4] = {top, z[0], z[1], z[2]};
#pragma unroll
            for (int x = 3; x < 64; x += 1) m[x & 3] = fmaxf(m[x & 3], z[x]);
            top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
          }
          if (__any_sync(0xffffffffu, (top - ref) * c > kPfSlack)) {
            // -inf - -inf is NaN: not greater, and the reference stays unset
            const float to = fmaxf(ref, top);
            const float by = to == -INFINITY ? 1.0f : ex2_approx((ref - to) * c);
            l *= by;
            ref = to;
            if (i > 0) {
              // the output before this tile is done: its products were issued before the scores
#pragma unroll 1
              for (int y = 0; y < D; y += 32) {
                float o[32];
                tmem_ld32(lane_addr + 256 + g * 128 + y, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= by;
                tmem_st16(lane_addr + 256 + g * 128 + y, reinterpret_cast<uint32_t*>(o));
                tmem_st16(lane_addr + 256 + g * 128 + y + 16, reinterpret_cast<uint32_t*>(o) + 16);
              }
            }
          }
          const float minus = ref == -INFINITY ? 0.0f : -ref * c;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float z[32];
            uint32_t w[16];
            tmem_ld32(s_addr + 32 * y, z);
            tmem_wait_ld();
            if (masked) hide(z, p0 + 32 * y);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float e0 = ex2_approx(fmaf(z[x], c, minus));
              const float e1 = ex2_approx(fmaf(z[x + 1], c, minus));
              sum[x & 3] += e0;
              sum[(x & 3) + 1] += e1;
              const __nv_bfloat162 v = __floats2bfloat162_rn(e0, e1);
              w[x / 2] = *reinterpret_cast<const uint32_t*>(&v);
            }
            tmem_st16(s_addr + 16 * y, w);  // over scores that have been read
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&sh.p_full[g]);
      }
      if (stop) break;
      // ------------------------------------------------------------ the piece's end
      pf_wait(&sh.o_full[g], o_phase, guard, a.err);
      o_phase ^= 1;
      const bool both = !it.two && tiles > 1;
      float m = ref == -INFINITY ? -INFINITY : ref * c;
      float mine = 1.0f, other = 0.0f;
      if (both) {
        sh.part[g][row] = make_float2(m, l);
        mbar_arrive(&sh.told[g]);
        pf_wait(&sh.told[g ^ 1], told_phase, guard, a.err);
        const float2 st = sh.part[g ^ 1][row];
        const float mn = fmaxf(m, st.x), base = mn == -INFINITY ? 0.0f : mn;
        mine = ex2_approx(m - base);
        other = ex2_approx(st.x - base);
        l = l * mine + st.y * other;
        m = mn;
      }
      if (__any_sync(0xffffffffu, guard->aborted())) break;
      tc_fence_after();
      if (live) {
        const bool begins = it.t0 == 0;
        const int64_t at = begins ? query
                                  : int64_t(blockIdx.x) * 256 + (it.two ? g * kPfTile : 0) + row;
        float* to = (begins ? a.parts[it.own] : a.mid) + (query < 0 ? 0 : at) * D;
        if (query >= 0 && (!both || g == 0))
          (begins ? a.stats[it.own] : a.mid_stats)[at] = make_float2(m, l);
        // with both groups' parts each takes half of the numbers
        const int y0 = both ? g * (D / 2) : 0, y1 = both ? y0 + D / 2 : D;
#pragma unroll 1
        for (int y = y0; y < y1; y += 32) {
          float o[32];
          tmem_ld32(lane_addr + 256 + g * 128 + y, o);
          if (both) {
            float o2[32];
            tmem_ld32(lane_addr + 256 + (g ^ 1) * 128 + y, o2);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = o[x] * mine + o2[x] * other;
          } else {
            tmem_wait_ld();
          }
          if (query >= 0) {
#pragma unroll
            for (int x = 0; x < 32; x += 4)
              *reinterpret_cast<float4*>(to + y + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
      }
      tc_fence_before();
      if (both) {
        mbar_arrive(&sh.read[g ^ 1]);
        pf_wait(&sh.read[g], told_phase, guard, a.err);
        told_phase ^= 1;
        if (__any_sync(0xffffffffu, guard->aborted())) break;
      }
    }
  } else if (work && warp < (kPfSoftmax + kPfLoad) / 32) {
    // ---------------------------------------------------------------- keys and values
    constexpr int kPerKey = D / 16;              // 16-byte chunks of a key's codes
    constexpr int kAtOnce = 32 / kPerKey;        // keys of a warp's load
    constexpr int kLoads = kPfTile * kPerKey / kPfLoad;
    constexpr int kPfAhead = D == 128 ? 2 : 4;   // tiles in flight
    const int lw = warp - kPfSoftmax / 32;
    // a quarter of the warp writes two keys that are not 8 apart: no bank twice
    const int chunk = D == 128 ? (lane & 3) + 4 * (lane >> 3 & 1) : lane & 3;
    const int sub = D == 128 ? (lane >> 2 & 1) + 2 * (lane >> 4) : lane >> 2;
    // the key of load i and place s of it; each lane finds one key's address
    static_assert(kLoads * kAtOnce == 32, "a warp's keys of a tile");
    auto key_of = [&](int i, int s) { return i * (kPfTile / kLoads) + lw * kAtOnce + s; };
    const int found = key_of(lane / kAtOnce, lane % kAtOnce);

    PfRing<kPfItems> ring;
    PfItem it;
    bool have = next_item(ring, it), stalled = false;
    int step = 0, phase = 0;
    PfTile pend0 = {}, pend1 = {};
    bool pending0 = false, pending1 = false;  // group 1 shares a tile with group 0: not pending
    // the tiles in their order; false: no more
    auto advance = [&](PfTile& out) {
      for (;;) {
        const int at = phase;
        if (at == 0) {
          ++phase;
          if (pending0) {
            pending0 = false;
            out = pend0;
            out.v = true;
            return true;
          }
          continue;
        }
        if (at == 2) {
          ++phase;
          if (pending1) {
            pending1 = false;
            out = pend1;
            out.v = true;
            return true;
          }
          continue;
        }
        if (!have) {
          if (at == 3) return false;
          ++phase;
          continue;
        }
        const int tiles = it.t1 - it.t0;
        const int x = it.two ? step : 2 * step + (at >> 1);
        const bool on = it.two ? at == 1 : x < tiles;
        if (on) {
          out.row = it.row;
          out.h = it.h;
          out.p0 = (it.tile0 + it.t0 + x) * kPfTile;
          out.end = it.end;
          out.own = it.own;
          out.v = false;
          if (at == 1) {
            pend0 = out;
            pending0 = true;
          } else {
            pend1 = out;
            pending1 = true;
          }
        }
        if (++phase == 4) {
          phase = 0;
          if (++step == (it.two ? tiles : (tiles + 1) / 2)) {
            step = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.item_empty[ring.at]);
            ring.next();
            have = next_item(ring, it);
          }
        }
        if (on) return true;
      }
    };

    PfTile tile[kPfAhead];
    bool full[kPfAhead];
    uint4 code[kPfAhead][kLoads];
    float scale[kPfAhead];  // of the key that this lane finds
    // where the codes are: found by one lane a key, passed to those that load it
    auto issue = [&](int x) {
      const PfTile& t = tile[x];
      const int pos = t.p0 + found;
      int64_t from = -1;
      scale[x] = 1.0f;
      if (pos < t.end) {
        const int j = pos / a.bs;
        const int id = j < a.MB ? a.bt[int64_t(t.row) * a.MB + j] : -1;
        const int unit = (t.v ? a.H : 0) + t.h;
        if (id >= 0 && id < a.NB) {
          scale[x] = a.scales[id * a.block_scales + unit];
          from = id * a.block_bytes + (int64_t(unit) * a.bs + (pos - j * a.bs)) * D;
        } else {
          // a key that cannot be read: its queries' outputs become NaN
          if (!t.v) scale[x] = __uint_as_float(0x7fc00000u);
          if (a.err) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, from, i * kAtOnce + sub);
        code[x][i] = make_uint4(0u, 0u, 0u, 0u);
        if (at >= 0) code[x][i] = load_codes(a.pool + at + chunk * 16);
      }
    };
    PfRing<NS> kv;
    auto widen = [&](int x) {
      pf_wait(&sh.kv_empty[kv.at], kv.phase ^ 1, guard, a.err);
      uint8_t* to = sm + kv.at * kTile;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int key = key_of(i, sub);
        const float s = __shfl_sync(0xffffffffu, scale[x], i * kAtOnce + sub);
        const uint32_t bits = __float_as_uint(s), exponent = bits >> 23;
        const uint32_t w[4] = {code[x][i].x, code[x][i].y, code[x][i].z, code[x][i].w};
        uint32_t r[8];
        if ((bits & 0x807fffffu) == 0 && exponent >= 27 && exponent <= 134) {
          // 2^-100 .. 2^7: the product with scale * 2^120 is exact
          const uint32_t up = ((exponent + 120) << 7) * 0x00010001u;
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
            const __nv_bfloat162 v0 = __floats2bfloat162_rn(f[0] * s, f[1] * s);
            const __nv_bfloat162 v1 = __floats2bfloat162_rn(f[2] * s, f[3] * s);
            r[2 * y] = *reinterpret_cast<const uint32_t*>(&v0);
            r[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&v1);
          }
        }
        *reinterpret_cast<uint4*>(to + pf_place(key, 2 * chunk)) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4*>(to + pf_place(key, 2 * chunk + 1)) =
            make_uint4(r[4], r[5], r[6], r[7]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.kv_full[kv.at]);
      kv.next();
    };
#pragma unroll
    for (int x = 0; x < kPfAhead; ++x) {
      full[x] = (x == 0 || full[x > 0 ? x - 1 : 0]) && advance(tile[x]);
      if (full[x]) issue(x);
    }
    for (bool more = true; more;) {
#pragma unroll
      for (int x = 0; x < kPfAhead; ++x) {
        if (!more) continue;
        more = full[x];
        if (!more) continue;
        stalled = stalled || (tile[x].own && tile[x].v && tile[x].row == a.stall_row);
        if (stalled || __any_sync(0xffffffffu, guard->aborted())) {
          more = false;
          continue;
        }
        widen(x);
        full[x] = full[(x + kPfAhead - 1) % kPfAhead] && advance(tile[x]);
        if (full[x]) issue(x);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (sh.guard.abort) {
    // what has been issued ends before the CTA's memory is another's
    if (warp == kMmaWarp) {
      if (lane == 0) tc_commit(&sh.drained);
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

template <int D>
int launch_shape(const PfArgs& a, int ctas, cudaStream_t st) {
  auto kern = kv_prefix_attention_kernel<D>;
  constexpr size_t smem = PfShape<D>::kBytes;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kern, smem, done) != SPEC_OK) return SPEC_ECUDA;
  return launch_pdl(kern, dim3(unsigned(ctas)), dim3(kPfThreads), smem, st, a);
}

}  // namespace

int launch_pf_attention(const PfArgs& a, int ctas, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.D == 128 ? launch_shape<128>(a, ctas, st) : launch_shape<64>(a, ctas, st);
}

}  // namespace sv
