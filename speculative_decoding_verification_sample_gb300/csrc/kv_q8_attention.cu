// Attention over the 8-bit paged cache: the kernel for every head size and
// block size, and the kernel that joins the parts of split items.
//
// attn_any_kernel runs on the CUDA cores in fp32 and takes what the tensor
// kernel does not: fp32 queries, head sizes other than 64 and 128, block sizes
// that neither divide 128 nor are multiples of it. 32 query rows by 32 keys at
// a time from shared memory, one pass with the running maximum and sum; 8
// threads share a row. Bound by the multiply-adds of the CUDA cores: 12.3 ms for 256 rows of
// 512-4096 tokens, 5 queries of 32 heads, where the tensor kernel takes 0.21 ms.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8_attn.cuh"

namespace sv {

constexpr int kAnyThreads = 256;
constexpr int kAnyRows = 32, kAnyKeys = 32, kAnyMaxD = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__global__ void __launch_bounds__(kAnyThreads) attn_any_kernel(const AttnArgs a) {
  extern __shared__ float sm[];
  __shared__ int64_t prefix[kAnyThreads + 1], warp_sum[kAnyThreads / 32];
  const int ld = a.D + 1;
  float* qs = sm;                    // [32][D]
  float* ks = qs + kAnyRows * a.D;   // [32][D + 1]
  float* vs = ks + kAnyKeys * ld;    // [32][D]
  float* ps = vs + kAnyKeys * a.D;   // [32][33]
  const int tid = threadIdx.x, c = blockIdx.x, nc = gridDim.x;
  const int r = tid >> 3, part = tid & 7;
  pdl_trigger();
  pdl_wait();
  write_empty_rows<T>(a, c, nc, tid, kAnyThreads);
  const AttnPlan plan = attn_plan(a, prefix, warp_sum, nc, c);
  if (plan.u0 >= plan.u1) {
    if (tid == 0) write_join(a, plan, nullptr, c);
    return;
  }
  Segment g = find_segment(a, prefix, plan.u0, plan.u1);
  if (tid == 0) write_join(a, plan, &g, c);
  for (;;) {
    const int row = g.rb * kAnyRows + r;  // query row of this thread
    const int t = row / a.G, head = g.h * a.G + row % a.G;
    const bool live = row < a.R;
    __syncthreads();
    for (int i = tid; i < kAnyRows * a.D; i += kAnyThreads) {
      const int rr = g.rb * kAnyRows + i / a.D, d = i % a.D;
      float x = 0.0f;
      if (rr < a.R) {
        const int64_t o = ((int64_t(g.b) * a.T + rr / a.G) * a.H * a.G + g.h * a.G + rr % a.G) * a.D;
        x = to_f32(static_cast<const T*>(a.q)[o + d]) * a.scale_log2;
      }
      qs[i] = x;
    }
    const uint32_t tmask = a.tree && live ? a.tree[int64_t(g.b) * a.T + t] : 0u;
    float m = -INFINITY, l = 0.0f, acc[kAnyMaxD / 8];
#pragma unroll
    for (int i = 0; i < kAnyMaxD / 8; ++i) acc[i] = 0.0f;
    for (int k = g.t0; k < g.t1; ++k) {
      const int p0 = tile_start(g.s, k);
      for (int p = p0; p < min(p0 + kAttnTile, g.s.end); p += kAnyKeys) {
        __syncthreads();
        // 32 keys and values: 16 codes a load
        const int gpt = a.D >> 4;
        for (int i = tid; i < 2 * kAnyKeys * gpt; i += kAnyThreads) {
          const int plane = i / (kAnyKeys * gpt), x = i % (kAnyKeys * gpt);
          const int j = x / gpt, d0 = (x % gpt) * 16, pos = p + j;
          float f[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) f[q] = 0.0f;
          if (needed(g.s, pos, 1)) {
            const int id = a.bt[int64_t(g.b) * a.MB + pos / a.bs];
            if (id >= 0 && id < a.NB) {
              const int64_t unit = int64_t(plane) * a.H + g.h;
              const float s = a.scales[id * a.block_scales + unit];
              const uint4 w = *reinterpret_cast<const uint4*>(
                  a.pool + id * a.block_bytes + (unit * a.bs + pos % a.bs) * a.D + d0);
              e4m3x4_to_f32(w.x, f);
              e4m3x4_to_f32(w.y, f + 4);
              e4m3x4_to_f32(w.z, f + 8);
              e4m3x4_to_f32(w.w, f + 12);
#pragma unroll
              for (int q = 0; q < 16; ++q) f[q] *= s;
            } else {
              // a key that cannot be read: its queries' outputs become NaN
              if (plane == 0)
#pragma unroll
                for (int q = 0; q < 16; ++q) f[q] = __uint_as_float(0x7fc00000u);
              if (a.err) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
            }
          }
          float* o = plane ? vs + j * a.D + d0 : ks + j * ld + d0;
#pragma unroll
          for (int q = 0; q < 16; ++q) o[q] = f[q];
        }
        __syncthreads();
        float z[4];
        float zm = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = part + 8 * i;
          z[i] = -INFINITY;
          if (live && sees(a, g.s, tmask, t, p + j)) {
            float dot = 0.0f;
            for (int d = 0; d < a.D; ++d) dot = fmaf(qs[r * a.D + d], ks[j * ld + d], dot);
            z[i] = dot;
          }
          zm = z[i] != z[i] ? z[i] : fmaxf(zm, z[i]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const float y = __shfl_xor_sync(0xffffffffu, zm, o);
          zm = fmaxf(zm, y);  // a NaN score makes l and the outputs NaN by itself
        }
        const float mn = fmaxf(m, zm);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float alpha = ex2_approx(m - base);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = ex2_approx(z[i] - base);
          ps[r * 33 + part + 8 * i] = e;
          sum += e;
        }
        l = l * alpha + sum;
        m = mn;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kAnyMaxD / 8; ++i) acc[i] *= alpha;
        for (int j = 0; j < kAnyKeys; ++j) {
          const float e = ps[r * 33 + j];
          if (e == 0.0f) continue;  // a key that the row does not see
#pragma unroll
          for (int i = 0; i < kAnyMaxD / 8; ++i)
            if (part + 8 * i < a.D) acc[i] = fmaf(e, vs[j * a.D + part + 8 * i], acc[i]);
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const bool whole = g.t0 == 0 && g.t1 == g.s.tiles;
    if (live) {
      if (whole) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        T* o = static_cast<T*>(a.out) +
               ((int64_t(g.b) * a.T + t) * a.H * a.G + head) * a.D;
#pragma unroll
        for (int i = 0; i < kAnyMaxD / 8; ++i)
          if (part + 8 * i < a.D) o[part + 8 * i] = T(acc[i] * inv);
      } else {
        const int64_t slot = 2 * c + (g.u == plan.u0 ? 0 : 1);
        float* o = a.parts + (slot * kAnyRows + r) * a.D;
#pragma unroll
        for (int i = 0; i < kAnyMaxD / 8; ++i)
          if (part + 8 * i < a.D) o[part + 8 * i] = acc[i];
        if (part == 0) a.stats[slot * kAnyRows + r] = make_float2(m, l);
      }
    }
    if (g.u + (g.t1 - g.t0) >= plan.u1) break;
    next_segment(a, g, plan.u1);
  }
}

// ------------------------------------------------------------------ joining
// CTA (c, y) joins rows 4 y .. 4 y + 3 of the item that ends in CTA c of the
// attention kernel, two warps a row (even and odd parts), each warp's lanes
// over the head's numbers, four a lane. Bound by the latency of its dependent reads
// (which parts, their statistics, their numbers), most of which lie in L2.
constexpr int kJoinThreads = 256, kJoinRows = 4;

__device__ __forceinline__ void store4(float* o, float4 v) { *reinterpret_cast<float4*>(o) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* o, float4 v) {
  __nv_bfloat162 x[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(x);
}

template <class T>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a) {
  __shared__ float4 acc_s[kJoinRows][kAnyMaxD / 4];
  __shared__ float2 st_s[kJoinRows];
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x;
  const int4 j = a.joins[c];
  if (j.x < 0) return;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, rr = w >> 1, half = w & 1;
  const int r = blockIdx.y * kJoinRows + rr, row = j.z * a.rows_per_block + r;
  const bool live = r < a.rows_per_block && row < a.R;
  const int c0 = j.w & ~(1 << 30), slot0 = j.w >> 30 & 1;
  const int np = c - c0 + 1;
  constexpr int kPer = kAnyMaxD / 128;
  const int quads = a.D / 4;
  float m = -INFINITY, l = 0.0f;
  float4 acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float pm, float pl, const float4* o) {
    const float mn = fmaxf(m, pm), base = mn == -INFINITY ? 0.0f : mn;
    const float x = ex2_approx(m - base), y = ex2_approx(pm - base);
    l = l * x + pl * y;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < quads) {
        const float4 v = o[32 * i];
        acc[i].x = acc[i].x * x + v.x * y;
        acc[i].y = acc[i].y * x + v.y * y;
        acc[i].z = acc[i].z * x + v.z * y;
        acc[i].w = acc[i].w * x + v.w * y;
      }
    m = mn;
  };
  if (live) {
#pragma unroll 2
    for (int k = half; k < np; k += 2) {
      const int64_t part =
          (2 * int64_t(c0 + k) + (k == 0 ? slot0 : 0)) * a.rows_per_block + r;
      const float2 st = a.stats[part];
      add(st.x, st.y, reinterpret_cast<const float4*>(a.parts + part * a.D) + lane);
    }
    if (half == 1) {
      st_s[rr] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < quads) acc_s[rr][lane + 32 * i] = acc[i];
    }
  }
  __syncthreads();
  if (!live || half == 1) return;
  add(st_s[rr].x, st_s[rr].y, &acc_s[rr][lane]);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  T* o = static_cast<T*>(a.out) +
         ((int64_t(j.x) * a.T + row / a.G) * a.H * a.G + j.y * a.G + row % a.G) * a.D + 4 * lane;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < quads)
      store4(o + 128 * i, make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
}

int launch_attn_join(const AttnArgs& a, int nc, int dtype, void* stream) {
  const dim3 grid(nc, (min(a.rows_per_block, a.R) + kJoinRows - 1) / kJoinRows);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SPEC_F32
             ? launch_pdl(attn_join_kernel<float>, grid, dim3(kJoinThreads), 0, st, a)
             : launch_pdl(attn_join_kernel<__nv_bfloat16>, grid, dim3(kJoinThreads), 0, st, a);
}

// ------------------------------------------------------------------ host
namespace {

constexpr int kAttnMaxCtas = 512;  // bound of the work split, for the workspace

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

size_t any_smem(int D) {
  return sizeof(float) * (size_t(kAnyRows) * D + kAnyKeys * (D + 1) + size_t(kAnyKeys) * D +
                          kAnyRows * 33);
}

template <class T>
int launch_any(const AttnArgs& a, int nc, void* stream) {
  static std::atomic<uint64_t> done{0};
  if (allow_smem(attn_any_kernel<T>, any_smem(kAnyMaxD), done) != SPEC_OK) return SPEC_ECUDA;
  return launch_pdl(attn_any_kernel<T>, dim3(nc), dim3(kAnyThreads), any_smem(a.D),
                    static_cast<cudaStream_t>(stream), a);
}

// Failure-detection test knobs, as the verification kernels have them, read at every launch:
// SPECVERIFY_STALL_ROW=b withholds the V tiles of batch row b, so that the tensor-core
// kernel's waits run out; SPECVERIFY_IDLE_NS shortens their limit.
void set_test_knobs(AttnArgs& a) {
  a.wait_ns = kWaitNs;
  a.stall_row = -1;
  const char* row = std::getenv("SPECVERIFY_STALL_ROW");
  if (!row) return;
  const long b = std::strtol(row, nullptr, 10);
  if (b >= 0 && b < a.B) a.stall_row = int(b);
  if (const char* ns = std::getenv("SPECVERIFY_IDLE_NS")) {
    const long long v = std::strtoll(ns, nullptr, 10);
    if (v > 0 && uint64_t(v) < kWaitNs) a.wait_ns = uint64_t(v);
  }
}

}  // namespace

// Enough for either kernel on any part of this family: at most kAttnMaxCtas
// CTAs, two parts each, at most 64 rows of a part.
size_t kv_q8_attention_workspace(int T, int G, int D) {
  const size_t rows = size_t(T) * G < 64 ? size_t(T) * G : 64;
  const size_t pad = rows < size_t(kAnyRows) ? size_t(kAnyRows) : 64;
  return up256(2 * kAttnMaxCtas * pad * D * sizeof(float)) +
         up256(2 * kAttnMaxCtas * pad * sizeof(float2)) + up256(kAttnMaxCtas * sizeof(int4));
}

int launch_kv_q8_attention(const Q8AttnLaunch& k) {
  AttnArgs a;
  const int64_t layer_bytes = int64_t(2) * k.H * k.bs * k.D;
  a.q = k.q;
  a.pool = static_cast<const uint8_t*>(k.pool) + k.layer * layer_bytes;
  a.scales = k.scales + int64_t(k.layer) * 2 * k.H;
  a.bt = k.block_table;
  a.sl = k.seq_lens;
  a.nn = k.num_new;
  a.tree = k.tree_mask;
  a.out = k.out;
  a.scale_log2 = float(double(k.softmax_scale) * 1.4426950408889634);
  a.window = k.window;
  a.sinks = k.sinks;
  a.NB = k.num_blocks;
  a.H = k.H;
  a.G = k.G;
  a.D = k.D;
  a.bs = k.bs;
  a.B = k.B;
  a.T = k.T;
  a.MB = k.max_blocks;
  a.block_bytes = k.num_layers * layer_bytes;
  a.block_scales = int64_t(k.num_layers) * 2 * k.H;
  a.R = k.T * k.G;
  a.err = k.err;
  set_test_knobs(a);
  a.plane0 = k.layer * 2 * k.H;
  a.planes_per_block = k.num_layers * 2 * k.H;
  const int sms = sm_count();
  if (sms == 0) return SPEC_ECUDA;
  const int64_t planes = int64_t(k.num_blocks) * a.planes_per_block;
  const bool tc = attn_tc_takes(k.dtype, k.D, k.bs, planes);
  a.rows_per_block = tc ? attn_tc_rows(a.R) : kAnyRows;
  a.RB = (a.R + a.rows_per_block - 1) / a.rows_per_block;
  uint8_t* ws = static_cast<uint8_t*>(k.workspace);
  a.parts = reinterpret_cast<float*>(ws);
  ws += up256(size_t(2) * kAttnMaxCtas * a.rows_per_block * k.D * sizeof(float));
  a.stats = reinterpret_cast<float2*>(ws);
  ws += up256(size_t(2) * kAttnMaxCtas * a.rows_per_block * sizeof(float2));
  a.joins = reinterpret_cast<int4*>(ws);
  int nc = 2 * sms < kAttnMaxCtas ? 2 * sms : kAttnMaxCtas;
  if (tc) {
    const int st = launch_attn_tc(a, k.pool, planes, sms, kAttnMaxCtas, &nc, k.stream);
    if (st != SPEC_OK) return st;
  } else {
    const int st = k.dtype == SPEC_F32 ? launch_any<float>(a, nc, k.stream)
                                       : launch_any<__nv_bfloat16>(a, nc, k.stream);
    if (st != SPEC_OK) return st;
  }
  return launch_attn_join(a, nc, k.dtype, k.stream);
}

}  // namespace sv
