// Appending tokens to the 8-bit paged KV cache.
//
// A block of tokens and head (bs x D numbers) is held as e4m3 codes c and one
// scale s, value = c * s. A call writes n tokens of a row at positions
// L .. L + n - 1 (L = seq_lens[b], unchanged); for each block that they touch
//   s_new = 2^ceil(log2(amax / 448))   amax over the block's new tokens,
//   s     = max(s_new, s_old)          when the block keeps tokens before L,
//   c     = e4m3(x / s),  c_kept = e4m3(c_old * s_old / s) when s grew.
// The scale is a power of two: e4m3 is itself a floating-point format, so a
// finer scale would buy accuracy in its subnormal tail only, and x / s is
// exact. Each number is thus rounded ONCE (half a step, 2^-4 relative), and
// kept codes move to a coarser scale without another rounding unless they
// fall below 2^-6 of the new range.
//
// Bound by memory: reads 2 or 4 bytes and writes 1 byte a number. One warp
// takes one (row, block, plane, head); neighbouring warps take neighbouring
// heads, whose tokens are adjacent in k and v. The block's new tokens stay in
// registers between the maximum and the rounding (up to 2048 bf16 numbers of
// a warp; longer blocks read the rest again, from L2). Their loads are issued
// before the block table answers, the maximum is taken on the packed bit patterns
// (magnitudes order as integers), and x / s is a product with the exact 1 / s.
// Measured: 12 prompts of up to 4099 tokens (8 heads x 128, bf16), 227 MB read and
// written, 39 us = 5.9 TB/s (fp32, 378 MB: 72 us); with divisions per number and per address, and the loads
// behind the block table, 97 us. 256 rows of 5 tokens: 6.0 us, latency.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8.cuh"

namespace sv {

constexpr int kApThreads = 256;

struct AppendArgs {
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* pool;    // already at the layer
  float* scales;    // already at the layer
  const int32_t* bt;
  const int32_t* sl;
  const int32_t* nn;
  int NB, H, D, bs, B, T, MB, J;
  int64_t block_bytes, block_scales;  // strides of one block id
  int32_t* err;
};

// Eight numbers of k or v: their bits, the largest magnitude's bits (bf16: two
// halves at once), their values.
template <bool kF32>
struct Eight {
  uint4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* p) {
    w[0] = *reinterpret_cast<const uint4*>(p);
    if (kF32) w[kF32 ? 1 : 0] = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
    const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = kF32 ? max(m, v[i] & 0x7fffffffu) : __vmaxu2(m, v[i] & 0x7fff7fffu);
    if (kF32) {
      const uint4 x = w[kF32 ? 1 : 0];
      m = max(max(m, x.x & 0x7fffffffu), x.y & 0x7fffffffu);
      m = max(max(m, x.z & 0x7fffffffu), x.w & 0x7fffffffu);
    }
    return m;
  }
  // In fp32. `guard`: NaN becomes 0, infinities the largest finite number (a NaN code
  // would spread to rows that do not see its token).
  __device__ __forceinline__ void values(float* f, bool guard) const {
    const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    if (kF32) {
      const uint4 x = w[kF32 ? 1 : 0];
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __uint_as_float(v[i]);
        f[4 + i] = __uint_as_float(u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    }
    if (guard) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        f[i] = f[i] != f[i] ? 0.0f : fminf(fmaxf(f[i], -FLT_MAX), FLT_MAX);
    }
  }
};

template <bool kF32>
__global__ void __launch_bounds__(kApThreads) kv_q8_append_kernel(const AppendArgs a) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * (kApThreads / 32) + (threadIdx.x >> 5);
  const uint32_t unit = task % (2 * a.H), w = task / (2 * a.H);  // unit: plane and head
  const int plane = unit >= uint32_t(a.H), h = int(unit) - plane * a.H;
  const int b = int(w / a.J), jw = int(w % a.J);
  pdl_wait();
  if (b >= a.B) return;
  const int L = a.sl[b], n = a.nn ? a.nn[b] : a.T;
  if (L < 0 || n < 0 || n > a.T || int64_t(L) + n > int64_t(a.MB) * a.bs) {
    if (a.err && jw == 0 && plane == 0 && h == 0 && lane == 0) atomicOr(a.err, SPEC_DERR_BAD_LENGTH);
    return;
  }
  const int j = L / a.bs + jw;
  const int start = j * a.bs;  // position of the block's first token
  if (n == 0 || start >= L + n) return;
  constexpr int kEb = kF32 ? 4 : 2;
  const int first = max(L - start, 0);             // offset of the first new token
  const int cnt = min(a.bs, L + n - start) - first;
  const int id = a.bt[int64_t(b) * a.MB + j];
  const int64_t tok = int64_t(a.H) * a.D * kEb;    // bytes from token to token
  const uint8_t* x = (plane ? a.v : a.k) +
                     (int64_t(b) * a.T + (start + first - L)) * tok + int64_t(h) * a.D * kEb;
  const int gpt = a.D >> 3;                        // groups of 8 numbers a token
  const int groups = cnt * gpt;
  constexpr int kHold = kF32 ? 4 : 8;              // groups that a lane keeps
  auto at = [&](int g) {
    const int t = g / gpt;
    return x + t * tok + (g - t * gpt) * 8 * kEb;
  };
  Eight<kF32> raw[kHold];
  if (32 % gpt == 0) {  // a lane's groups are 32 / gpt tokens apart
    const uint8_t* p = at(lane);
    const int64_t step = 32 / gpt * tok;
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (lane + 32 * i < groups) raw[i].load(p + i * step);
  } else {
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (lane + 32 * i < groups) raw[i].load(at(lane + 32 * i));
  }
  if (id < 0 || id >= a.NB) {
    if (a.err && lane == 0) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
    return;
  }
  uint8_t* codes = a.pool + id * a.block_bytes + int64_t(unit) * a.bs * a.D;
  float* sp = a.scales + id * a.block_scales + unit;
  const float was = first > 0 ? *sp : 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (lane + 32 * i < groups) top = raw[i].top(top);
  for (int g = lane + 32 * kHold; g < groups; g += 32) {
    Eight<kF32> r;
    r.load(at(g));
    top = r.top(top);
  }
  if (!kF32) top = max(top << 16, top & 0xffff0000u);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool guard = top >= 0x7f800000u;  // an infinity or a NaN among the numbers
  if (guard) {
    float m = 0.0f;
#pragma unroll 1
    for (int g = lane; g < groups; g += 32) {
      Eight<kF32> r;
      float f[8];
      r.load(at(g));
      r.values(f, true);
#pragma unroll
      for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(f[q]));
    }
    top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
  }
  float scale = q8_pow2(q8_scale_exp(__uint_as_float(top)));
  if (first > 0) scale = fmaxf(scale, was);
  // an older and larger scale may be any number that the caller has put there
  const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
  const float inv = 1.0f / scale;
  if (first > 0 && scale != was) {
    const float r = was / scale;
    const int words = first * a.D / 16;
    for (int g = lane; g < words; g += 32) {
      uint4 c = *reinterpret_cast<const uint4*>(codes + g * 16);
      uint32_t* cw = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[4];
        e4m3x4_to_f32(cw[q], f);
        cw[q] = f32x4_to_e4m3(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
      }
      *reinterpret_cast<uint4*>(codes + g * 16) = c;
    }
  }
  uint8_t* to = codes + int64_t(first) * a.D;
  auto put = [&](int g, const Eight<kF32>& r) {
    float f[8];
    r.values(f, false);
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] *= inv;
    uint2 c;
    c.x = f32x4_to_e4m3(f[0], f[1], f[2], f[3]);
    c.y = f32x4_to_e4m3(f[4], f[5], f[6], f[7]);
    *reinterpret_cast<uint2*>(to + g * 8) = c;
  };
  if (exact && !guard) {
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (lane + 32 * i < groups) put(lane + 32 * i, raw[i]);
    for (int g = lane + 32 * kHold; g < groups; g += 32) {
      Eight<kF32> r;
      r.load(at(g));
      put(g, r);
    }
  } else {
#pragma unroll 1
    for (int g = lane; g < groups; g += 32) {
      Eight<kF32> r;
      float f[8];
      r.load(at(g));
      r.values(f, true);
      uint2 c;
      c.x = f32x4_to_e4m3(f[0] / scale, f[1] / scale, f[2] / scale, f[3] / scale);
      c.y = f32x4_to_e4m3(f[4] / scale, f[5] / scale, f[6] / scale, f[7] / scale);
      *reinterpret_cast<uint2*>(to + g * 8) = c;
    }
  }
  if (lane == 0) {
    *sp = scale;
    if (guard && a.err) atomicOr(a.err, SPEC_DERR_VALUE);
  }
}

int launch_kv_q8_append(const Q8AppendLaunch& k) {
  AppendArgs a;
  a.k = static_cast<const uint8_t*>(k.k);
  a.v = static_cast<const uint8_t*>(k.v);
  const int64_t layer_bytes = int64_t(2) * k.H * k.bs * k.D;
  a.pool = static_cast<uint8_t*>(k.pool) + k.layer * layer_bytes;
  a.scales = k.scales + int64_t(k.layer) * 2 * k.H;
  a.bt = k.block_table;
  a.sl = k.seq_lens;
  a.nn = k.num_new;
  a.NB = k.num_blocks;
  a.H = k.H;
  a.D = k.D;
  a.bs = k.bs;
  a.B = k.B;
  a.T = k.T;
  a.MB = k.max_blocks;
  a.J = (k.T + 2 * k.bs - 2) / k.bs;  // blocks that T tokens can touch
  a.block_bytes = k.num_layers * layer_bytes;
  a.block_scales = int64_t(k.num_layers) * 2 * k.H;
  a.err = k.err;
  const int64_t tasks = int64_t(k.B) * a.J * 2 * k.H;
  const int64_t grid = (tasks + kApThreads / 32 - 1) / (kApThreads / 32);
  if (tasks > INT32_MAX) return SPEC_ENOTSUP;
  cudaStream_t st = static_cast<cudaStream_t>(k.stream);
  return k.dtype == SPEC_F32
             ? launch_pdl(kv_q8_append_kernel<true>, dim3(unsigned(grid)), dim3(kApThreads), 0, st, a)
             : launch_pdl(kv_q8_append_kernel<false>, dim3(unsigned(grid)), dim3(kApThreads), 0, st, a);
}

}  // namespace sv
