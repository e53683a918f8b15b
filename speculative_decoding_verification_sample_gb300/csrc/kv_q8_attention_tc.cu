// Attention over the 8-bit paged cache on the tensor cores (see q8_attn.cuh for
// what is computed and how the work is split).
//
// The cached codes go from TMA straight into tcgen05.mma: nothing converts them.
// Both products are taken with the cache as the M operand, so that the few
// query rows of a verification step fill the small N side:
//   S^T [128 keys x 2 NR]  = K  [128 x D]   * (Qhi | Qlo)^T       e4m3 x e4m3
//   O^T [D x NO]          += V^T [D x 128]  * (P0 + P1 + P2)^T    e4m3 x e5m2
// K is read along D, V along its other side (D is contiguous), both through the
// swizzle that TMA wrote. A block scale belongs to a key, that is to a TMEM lane
// of S^T, so scaling costs one product for K's and is folded into the
// probabilities for V's.
//   Queries: each row is scaled by a power of two to [128, 256) and split into two
// e4m3 terms (4 + 4 bits: a bf16 number exactly, down to 2^-10 of the row's
// largest). Probabilities: p is rounded once to 9 bits (2^-9 relative) and split
// into three e5m2 terms of at most 3 bits, exactly; e5m2 is the upper byte of
// fp16, so a term is a byte of the fp16 number and the rest one subtraction.
// 9 bits leave the bf16 output's own rounding the larger error; e5m2's 32
// binades hold what a key contributes (probability times V scale) down to 2^-22 of
// the row's reference.
//   Softmax: a row's reference m is the largest z_j + log2(V scale of j) (rounded up
// to a binade) of the first tile, and is only moved when a later one exceeds it by
// 8: then O and l are rescaled once; otherwise a tile costs no reduction over its
// keys. l stays per thread (one key of every tile) until the item ends.
//
// Roles: warps 0-3 softmax (thread = key of the tile), warp 4 TMA, warp 5 MMA.
// K and V tiles share one ring of slots, released separately. Two CTAs per SM
// hide each other's latencies.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <mutex>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8_attn.cuh"
#include "tc.cuh"

namespace sv {

constexpr int kTcSoftmax = 128;             // threads of the softmax warps
constexpr int kTcThreads = kTcSoftmax + 64;
constexpr int kTcScaleRing = 8;             // tiles whose scales are held
constexpr int kTcMaxPages = 16;             // blocks of one tile
constexpr float kTcUnset = -1e30f;          // reference of a row that has seen no key
constexpr float kTcSlack = 8.0f;            // binades by which keys may exceed the reference
constexpr float kTcLift = 64.0f;            // 1 enters as 2^6: 2^6 2^8 < 2^16, e5m2's range
constexpr int kTcSmem = 107 * 1024;         // dynamic, of one CTA: two per SM

template <int NR, int D>
struct TcShape {
  static constexpr int NO = (NR + 15) / 16 * 16;
  static constexpr int kSlot = kAttnTile * D;
  static constexpr int kQ = 2 * NR * D;
  static constexpr int kP = 3 * NO * kAttnTile;
  static constexpr int kFit = (kTcSmem - kQ - kP - 1024) / kSlot;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static constexpr int kSBufs = 4 * NR + NO <= 256 ? 2 : 1;
  static constexpr int kCols = kSBufs * 2 * NR + NO;
  static constexpr int kAlloc = kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
  static constexpr size_t kBytes = size_t(kSlots) * kSlot + kQ + kP + 1024;
  static_assert(kCols <= 256 && kSlots >= 3, "two CTAs per SM");
};

template <int NR>
struct TcShared {
  uint64_t full[8], empty[8], s_full[2], s_empty[2], p_full, pv_done, q_full;
  uint32_t tmem;
  int abort;
  float ks[kTcScaleRing][kTcMaxPages], vs[kTcScaleRing][kTcMaxPages];
  float row_c[NR];     // query row's scale * softmax_scale * log2(e)
  float row_m[NR];     // reference of the exponentials
  float row_a[NR];     // rescale factor, then that of the output
  int row_t[NR];       // query (T for rows that do not exist)
  uint32_t row_mask[NR];
  float part[4][NR];   // the warps' maxima, then sums
  int part_v[4];
};

// Bounded wait. Once one has given up, every wait returns at once: the roles
// run out their loops (the barriers among the softmax threads stay matched),
// the error bit is set and the outputs are not to be used.
__device__ __forceinline__ void tc_wait(uint64_t* bar, uint32_t parity, int* abort, int32_t* err) {
  if (mbar_try_wait(bar, parity, kSuspendNs)) return;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (*reinterpret_cast<volatile int*>(abort)) return;
    if (mbar_try_wait(bar, parity, kSuspendNs)) return;
    if (global_ns() - t0 > kWaitNs) break;
  }
  *reinterpret_cast<volatile int*>(abort) = 1;
  if (err) atomicOr(err, SPEC_DERR_TIMEOUT);
}

__device__ __forceinline__ void bar_softmax() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}
__device__ __forceinline__ bool bar_softmax_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(x))
      : "memory");
  return r != 0;
}

// The smallest e in [-100, 100] with |x| <= 2^e (100 for larger ones).
__device__ __forceinline__ int scale_binade(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  const int e = int(u >> 23) - 127 + ((u & 0x7fffffu) != 0);
  return max(-100, min(100, e));
}

// Maximum over the warp of floats without NaN: as integers in float order.
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  i ^= (i >> 31) & 0x7fffffff;
  return __int_as_float(i);
}

template <int NR, int D>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_tc_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap map) {
  using S = TcShape<NR, D>;
  constexpr int NS = S::kSlots, NO = S::NO, NB = S::kSBufs;
  constexpr uint32_t kSwz = D == 128 ? 2 : 4;  // TMA and operands: 128- or 64-byte swizzle
  extern __shared__ uint8_t raw_smem[];
  __shared__ TcShared<NR> sh;
  __shared__ int64_t prefix[kTcThreads + 1];
  uint8_t* sm = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  uint8_t* q_s = sm + NS * S::kSlot;
  uint8_t* p_s = q_s + S::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, nc = gridDim.x;

  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sh.full[i], 1 + 32);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.s_empty[i], kTcSoftmax);
    }
    mbar_init(&sh.p_full, kTcSoftmax);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.q_full, kTcSoftmax);
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(&sh.tmem, S::kAlloc);
    tmem_relinquish();
    if (lane == 0) tma_prefetch_map(&map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  write_empty_rows<__nv_bfloat16>(a, c, nc);
  const AttnPlan plan = attn_plan(a, prefix, nc, c);
  const bool work = plan.u0 < plan.u1;
  Segment g;
  if (work) g = find_segment(a, prefix, plan.u0, plan.u1);
  if (tid == 0) write_join(a, plan, work ? &g : nullptr, c);
  const int bs = min(a.bs, kAttnTile);      // rows of one copy
  const int pages = kAttnTile / bs;

  if (work && warp == 4) {
    // ---------------------------------------------------------------- TMA
    int i = 0, j = 0;  // ring position, tile
    int id = -1;
    auto page_id = [&](const Segment& s, int k) {
      const int pos = tile_start(s.s, k) + lane * bs;
      return lane < pages && needed(s.s, pos, bs) ? a.bt[int64_t(s.b) * a.MB + pos / a.bs] : -2;
    };
    id = page_id(g, g.t0);
    for (;;) {
      for (int k = g.t0; k < g.t1; ++k, ++j) {
        const int cur = id;
        const int pos = tile_start(g.s, k) + lane * bs;
        if (k + 1 < g.t1) id = page_id(g, k + 1);  // in flight while this tile's slots are awaited
        const bool ok = cur >= 0 && cur < a.NB;
        if (cur != -2 && !ok && a.err) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * uint32_t(bs) * D;
        const int c1 = pos % a.bs;
        const int plane = ok ? cur * a.planes_per_block + a.plane0 + g.h : 0;
#pragma unroll
        for (int v = 0; v < 2; ++v, ++i) {
          const int slot = i % NS;
          tc_wait(&sh.empty[slot], ((i / NS) & 1) ^ 1, &sh.abort, a.err);
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
          __syncwarp();
          if (ok)
            tma_tile_3d(sm + slot * S::kSlot + lane * bs * D, &map, 0, c1, plane + v * a.H,
                        &sh.full[slot]);
          bool copying = false;
          if (v == 1 && lane < pages) {
            float* ks = &sh.ks[j % kTcScaleRing][lane];
            float* vs = &sh.vs[j % kTcScaleRing][lane];
            if (ok) {
              const float* sp = a.scales + cur * a.block_scales + g.h;
              cp_async4(ks, sp);
              cp_async4(vs, sp + a.H);
              copying = true;
            } else {
              // a block that cannot be read: NaN scores; one that is not needed: zeros
              *ks = cur == -2 ? 0.0f : __uint_as_float(0x7fc00000u);
              *vs = 0.0f;
            }
          }
          if (copying) cp_async_arrive(&sh.full[slot]);
          else mbar_arrive(&sh.full[slot]);
        }
      }
      if (g.u + (g.t1 - g.t0) >= plan.u1) break;
      next_segment(a, g, plan.u1);
      id = page_id(g, g.t0);
    }
    // the copies land before the CTA may leave
    for (int x = max(0, i - NS); x < i; ++x)
      tc_wait(&sh.full[x % NS], (x / NS) & 1, &sh.abort, a.err);
  } else if (work && warp == 5) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      constexpr uint32_t idesc_s = tc_idesc(0, 0, 0, 0, 128, 2 * NR);
      constexpr uint32_t idesc_o = tc_idesc(0, 1, 1, 1, 128, NO);
      const uint32_t ring = smem_u32(sm);
      const uint64_t q_desc = tc_desc(smem_u32(q_s), 16, 8 * D, kSwz);
      const uint64_t p_desc = tc_desc(smem_u32(p_s), 128, 2048, 0);
      int j = 0, seg = 0;
      auto scores = [&](int t, bool first) {
        const int i = 2 * t, slot = i % NS, buf = t % NB;
        if (first) tc_wait(&sh.q_full, seg & 1, &sh.abort, a.err);
        tc_wait(&sh.full[slot], (i / NS) & 1, &sh.abort, a.err);
        tc_wait(&sh.s_empty[buf], ((t / NB) & 1) ^ 1, &sh.abort, a.err);
        tc_fence_after();
        const uint64_t k_desc = tc_desc(ring + slot * S::kSlot, 16, 8 * D, kSwz);
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
          tc_mma_f8(tmem + buf * 2 * NR, k_desc + 2 * x, q_desc + 2 * x, idesc_s, x > 0);
        tc_commit(&sh.empty[slot]);
        tc_commit(&sh.s_full[buf]);
      };
      auto outputs = [&](int t, bool first) {
        const int i = 2 * t + 1, slot = i % NS;
        tc_wait(&sh.full[slot], (i / NS) & 1, &sh.abort, a.err);
        tc_wait(&sh.p_full, t & 1, &sh.abort, a.err);
        tc_fence_after();
        // V as stored: D contiguous, groups of 8 keys 8 D bytes apart. With D = 64 the
        // second half of M repeats the first (offset 0) and is ignored.
        const uint64_t v_desc = tc_desc(ring + slot * S::kSlot, 0, 8 * D, kSwz);
#pragma unroll
        for (int x = 0; x < kAttnTile / 32; ++x)
#pragma unroll
          for (int m = 0; m < 3; ++m)
            tc_mma_f8(tmem + NB * 2 * NR, v_desc + x * (32 * D / 16),
                      p_desc + (m * NO * kAttnTile + x * 512) / 16, idesc_o,
                      !(first && x == 0 && m == 0));
        tc_commit(&sh.empty[slot]);
        tc_commit(&sh.pv_done);
      };
      for (;;) {
        scores(j, true);
        for (int k = g.t0; k < g.t1; ++k, ++j) {
          if (k + 1 < g.t1) scores(j + 1, false);
          outputs(j, k == g.t0);
        }
        ++seg;
        if (g.u + (g.t1 - g.t0) >= plan.u1) break;
        next_segment(a, g, plan.u1);
      }
    }
    __syncwarp();
  } else if (work) {
    // ---------------------------------------------------------------- softmax
    const uint32_t lane_addr = tmem + (uint32_t(warp * 32) << 16);
    const uint32_t o_addr = lane_addr + NB * 2 * NR;
    int j = 0;
    for (;;) {
      // queries of this item -> two e4m3 terms each
      bar_softmax();  // the previous item's rows are done with
      constexpr int kPerRow = D / 8;  // threads of a row, eight numbers each
#pragma unroll 1
      for (int r0 = 0; r0 < NR; r0 += kTcSoftmax / kPerRow) {
        const int r = r0 + tid / kPerRow, d8 = tid % kPerRow;
        if (r < NR) {
          const int row = g.rb * a.rows_per_block + r;
          const bool live = r < a.rows_per_block && row < a.R;
          const int t = live ? row / a.G : a.T;
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (live)
            w = *reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) +
                ((int64_t(g.b) * a.T + t) * a.H * a.G + g.h * a.G + (row - t * a.G)) * D + d8 * 8);
          float f[8];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
          uint32_t top = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            f[2 * x] = __uint_as_float(u[x] << 16);
            f[2 * x + 1] = __uint_as_float(u[x] & 0xffff0000u);
            top = max(top, max((u[x] << 16) & 0x7fffffffu, u[x] & 0x7fff0000u));
          }
#pragma unroll
          for (int o = kPerRow / 2; o > 0; o >>= 1)
            top = max(top, __shfl_xor_sync(__activemask(), top, o));
          // |x| 2^-e in [128, 256) at the largest; e also stays in range for bf16 subnormals
          const int e = max(int(top >> 23) - 127 - 7, -110);
          const float down = q8_pow2(-e > 120 ? 120 : -e);
          const float up = q8_pow2(e);
          float lo[8];
          uint32_t hw[2], lw[2];
#pragma unroll
          for (int x = 0; x < 8; ++x) f[x] *= down;
          hw[0] = f32x4_to_e4m3(f[0], f[1], f[2], f[3]);
          hw[1] = f32x4_to_e4m3(f[4], f[5], f[6], f[7]);
          e4m3x4_to_f32(hw[0], lo);
          e4m3x4_to_f32(hw[1], lo + 4);
#pragma unroll
          for (int x = 0; x < 8; ++x) lo[x] = f[x] - lo[x];
          lw[0] = f32x4_to_e4m3(lo[0], lo[1], lo[2], lo[3]);
          lw[1] = f32x4_to_e4m3(lo[4], lo[5], lo[6], lo[7]);
          auto put = [&](int rr, const uint32_t* x) {
            const int sw = D == 128 ? rr & 7 : (rr >> 1) & 3;
            const int chunk = (d8 >> 1) ^ sw;
            *reinterpret_cast<uint2*>(q_s + rr * D + chunk * 16 + (d8 & 1) * 8) =
                make_uint2(x[0], x[1]);
          };
          put(r, hw);
          put(NR + r, lw);
          if (d8 == 0) {
            // a row with an infinity or a NaN: its scores are NaN
            sh.row_c[r] = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : up * a.scale_log2;
            sh.row_m[r] = live ? kTcUnset : 0.0f;
            sh.row_t[r] = t;
            sh.row_mask[r] = a.tree && live ? a.tree[int64_t(g.b) * a.T + t] : 0u;
          }
        }
      }
      fence_async_smem();
      mbar_arrive(&sh.q_full);
      bar_softmax();
      float l[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) l[r] = 0.0f;
      int vref = 0;

      for (int k = g.t0; k < g.t1; ++k, ++j) {
        const int p0 = tile_start(g.s, k), pos = p0 + tid;
        const int buf = j % NB, vi = 2 * j + 1, vslot = vi % NS;
        tc_wait(&sh.s_full[buf], (j / NB) & 1, &sh.abort, a.err);
        tc_wait(&sh.full[vslot], (vi / NS) & 1, &sh.abort, a.err);
        tc_fence_after();
        const float vs = sh.vs[j % kTcScaleRing][tid / bs];
        const float ks =
            fabsf(vs) <= FLT_MAX ? sh.ks[j % kTcScaleRing][tid / bs] : __uint_as_float(0x7fc00000u);
        float z[NR];
#pragma unroll
        for (int r = 0; r < NR; r += 8) {
          float lo[8];
          tmem_ld8(lane_addr + buf * 2 * NR + r, z + r);
          tmem_ld8(lane_addr + buf * 2 * NR + NR + r, lo);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 8; ++x) z[r + x] += lo[x];
        }
        tc_fence_before();
        mbar_arrive(&sh.s_empty[buf]);
#pragma unroll
        for (int r = 0; r < NR; ++r) z[r] = z[r] * ks * sh.row_c[r];
        bool keep = ks == ks;  // does the token's V row enter the product?
        if (!tile_open(a, g.s, p0)) {
          keep = keep && needed(g.s, pos, 1);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (!sees(a, g.s, sh.row_mask[r], sh.row_t[r], pos)) z[r] = -INFINITY;
        }
        if (!keep) {
          // what lies there is not a number of this row (and 0 * NaN is NaN)
          uint4* v = reinterpret_cast<uint4*>(sm + vslot * S::kSlot + tid * D);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) v[x] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (k == g.t0) {
          // V scales are taken relative to this tile's largest, a power of two
          const int x = __reduce_max_sync(0xffffffffu, scale_binade(vs));
          if (lane == 0) sh.part_v[warp] = x;
          bar_softmax();
          vref = max(max(sh.part_v[0], sh.part_v[1]), max(sh.part_v[2], sh.part_v[3]));
        }
        const float vr = vs * q8_pow2(-vref);
        const float lv = float(scale_binade(vr));  // vr <= 2^lv
        bool over = k == g.t0;
#pragma unroll
        for (int r = 0; r < NR; ++r) over = over || z[r] - sh.row_m[r] > kTcSlack - lv;
        if (bar_softmax_or(over)) {
          // move the references to this tile's maxima
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float x = warp_max(z[r] == z[r] ? z[r] + lv : -INFINITY);
            if (lane == (r & 31)) sh.part[warp][r] = x;
          }
          bar_softmax();
          for (int r = tid; r < NR; r += kTcSoftmax) {
            const float old = sh.row_m[r];
            const float m = fmaxf(fmaxf(fmaxf(sh.part[0][r], sh.part[1][r]),
                                        fmaxf(sh.part[2][r], sh.part[3][r])), old);
            sh.row_m[r] = m;
            sh.row_a[r] = ex2_approx(old - m);
          }
          bar_softmax();
#pragma unroll
          for (int r = 0; r < NR; ++r) l[r] *= sh.row_a[r];
          if (k > g.t0) {
            tc_wait(&sh.pv_done, (j - 1) & 1, &sh.abort, a.err);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < NR; r += 8) {
              float o[8];
              tmem_ld8(o_addr + r, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 8; ++x) o[x] *= sh.row_a[r + x];
              tmem_st8(o_addr + r, o);
            }
            tmem_wait_st();
          }
        }
        if (j > 0) tc_wait(&sh.pv_done, (j - 1) & 1, &sh.abort, a.err);  // P may be replaced
        const float lift = vr * kTcLift;
#pragma unroll
        for (int r0 = 0; r0 < NR; r0 += 16) {
          uint32_t t0[4], t1[4], t2[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = r0 + 4 * x;
            if (r < NR) {
              uint32_t h[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float p[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const int rr = r + 2 * y + w;
                  p[w] = ex2_approx(z[rr] - sh.row_m[rr]);
                  l[rr] += p[w];
                  p[w] *= lift;
                }
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[y]) : "f"(p[1]), "f"(p[0]));
                h[y] = (h[y] + 0x00020002u) & 0xfffcfffcu;  // 9 bits, half up
              }
              auto rest = [](uint32_t v) {
                uint32_t o;
                asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(v), "r"(v & 0xff00ff00u));
                return o;
              };
              t0[x] = __byte_perm(h[0], h[1], 0x7531);
              h[0] = rest(h[0]);
              h[1] = rest(h[1]);
              t1[x] = __byte_perm(h[0], h[1], 0x7531);
              h[0] = rest(h[0]);
              h[1] = rest(h[1]);
              t2[x] = __byte_perm(h[0], h[1], 0x7531);
            }
          }
          uint8_t* d = p_s + (r0 / 16) * 2048 + tid * 16;
          auto put = [&](uint8_t* to, const uint32_t* t) {
            if (r0 + 16 <= NR) *reinterpret_cast<uint4*>(to) = make_uint4(t[0], t[1], t[2], t[3]);
            else *reinterpret_cast<uint2*>(to) = make_uint2(t[0], t[1]);
          };
          put(d, t0);
          put(d + NO * kAttnTile, t1);
          put(d + 2 * NO * kAttnTile, t2);
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sh.p_full);
      }

      // ------------------------------------------------------------ the item's end
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float x = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == (r & 31)) sh.part[warp][r] = x;
      }
      bar_softmax();
      const bool whole = g.t0 == 0 && g.t1 == g.s.tiles;
      const int64_t slot = 2 * c + (g.u == plan.u0 ? 0 : 1);
      const int rows = min(a.rows_per_block, a.R - g.rb * a.rows_per_block);
      for (int r = tid; r < NR; r += kTcSoftmax) {
        const float sum = sh.part[0][r] + sh.part[1][r] + sh.part[2][r] + sh.part[3][r];
        // A part is left with its sum in [1, 2): references of parts differ by their V
        // scales, so a sum by itself may be as far from 1 as those.
        const int e = sum > 0.0f && sum <= FLT_MAX ? int(__float_as_uint(sum) >> 23) - 127 : 0;
        sh.row_a[r] = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : q8_pow2(-e);
        if (!whole && r < rows)
          a.stats[slot * a.rows_per_block + r] =
              make_float2(sum == 0.0f ? -INFINITY : sh.row_m[r] + float(e), sum * q8_pow2(-e));
      }
      bar_softmax();
      tc_wait(&sh.pv_done, (j - 1) & 1, &sh.abort, a.err);
      tc_fence_after();
      const float unlift = q8_pow2(vref) / kTcLift;
#pragma unroll 1
      for (int r0 = 0; r0 < NR; r0 += 8) {
        float o[8];
        tmem_ld8(o_addr + r0, o);
        tmem_wait_ld();
        if (D == 128 || tid < D) {
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int r = r0 + x;
            if (r < rows) {
              const float v = o[x] * sh.row_a[r] * unlift;
              if (whole) {
                const int row = g.rb * a.rows_per_block + r, t = sh.row_t[r];
                static_cast<__nv_bfloat16*>(
                    a.out)[((int64_t(g.b) * a.T + t) * a.H * a.G + g.h * a.G + (row - t * a.G)) * D +
                           tid] = __float2bfloat16(v);
              } else {
                a.parts[(slot * a.rows_per_block + r) * D + tid] = v;
              }
            }
          }
        }
      }
      tc_fence_before();  // the next item's products overwrite O after its q_full and p_full
      if (g.u + (g.t1 - g.t0) >= plan.u1) break;
      next_segment(a, g, plan.u1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, S::kAlloc);
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
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) !=
      cudaSuccess)
    return SPEC_ECUDA;
  return launch_pdl(kern, dim3(nc), dim3(kTcThreads), smem, st, a, map);
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
