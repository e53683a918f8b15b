// Norms of queries and keys, rotary positions, and the same with keys and values
// written to the 8-bit paged cache.
//
//   norm    y = x * w / sqrt(mean(x^2) + eps) over a head's D numbers, where w is given
//   turn    pair i of the first 2 * half numbers by the angle p * inv_freq[i]:
//           (a, b) -> f (a cos - b sin, b cos + a sin); a pair is (i, i + half), or
//           (2 i, 2 i + 1) interleaved; the numbers after them stay
//   cache   as kv_q8_append (kv_q8_append.cu), from the fp32 numbers: a key is rounded once
//
// Angles. A frequency is held as a 64-bit fraction of a turn, so that p * inv_freq modulo
// a turn is one integer product, exact to 2^-54 turns per position; an fp32 angle of
// position 100 000 would be off by 0.004 rad, which keys and queries far from each other
// do not share. sin and cos of the eighth turn that is left are Taylor polynomials (the
// first terms left out are below 2e-9 and 2e-10).
//
// Split. A CTA takes the new tokens of one cache block (without a cache: 16 tokens) of a
// row: it makes their table of cos and sin in shared memory once for all heads, then its
// warps take tasks. A lane holds two vectors of a head, those that belong to each other
// in the turn, so that only the norm's sum crosses lanes: 8 lanes a head of 128 bf16
// numbers, 4 heads a warp. A task is two such loads of one token's heads, or with a cache
// a plane and head of the block: its numbers stay in registers from the maximum to the
// rounding (as many as 64 a lane hold; those of longer blocks are made twice). Few tokens:
// the tasks of a block are split over several CTAs, each with the table.
//
// Bound by memory: every number is read and written once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8.cuh"

namespace sv {

constexpr int kNrThreads = 256, kNrWarps = kNrThreads / 32;
constexpr int kNrTile = 16;              // tokens of a CTA without a cache
constexpr int kNrTable = 64 * 1024;      // bytes of cos and sin at most
constexpr int kNrHold = 64;              // numbers that a lane keeps

struct NormRopeArgs {
  const uint8_t *q, *k, *v;              // first token; v: with a cache
  uint8_t *qo, *ko;                      // ko: without a cache
  int64_t q_step, k_step, v_step, qo_step, ko_step;  // bytes from token to token
  const void *qw, *kw;                   // [D] of the tensors' type; null: no norm
  const float* freq;                     // [half]
  const int32_t *sl, *nn, *pos;          // pos [B, T]; null: sl + t. nn null: T
  int Hq, H, D, half, B, T, interleaved;
  float eps, factor;
  uint8_t* pool;                         // at the layer; the rest is for a cache
  float* scales;
  const int32_t* bt;
  int NB, bs, MB, J;                     // J: blocks (tiles) that T tokens can touch
  int64_t block_bytes, block_scales;
  int32_t* err;
};

// A frequency as a fraction of a turn, in units of 2^-64. |w| up to 2^64: beyond it the
// quotient has no fraction left, and infinities and NaN give 0.
__device__ __forceinline__ uint64_t turn_fraction(float w) {
  double t = double(w) * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return t < 1.0 ? static_cast<uint64_t>(t * 18446744073709551616.0) : 0ull;
}

// cos and sin of p * (fraction of a turn), times f.
__device__ __forceinline__ float2 turned(uint64_t fraction, int p, float f) {
  const uint64_t a = fraction * static_cast<uint64_t>(int64_t(p));
  // to the nearest quarter turn, and what is left of it, at most an eighth of a turn
  const uint64_t b = a + (uint64_t(1) << 61);
  const uint32_t quarter = uint32_t(b >> 62);
  const int64_t left = static_cast<int64_t>(a - (uint64_t(quarter) << 62));
  // (quarter 4 wraps to 0, and so does its difference)
  constexpr float kUnit = float(6.283185307179586 / 17179869184.0);  // 2 pi 2^-34
  const float x = float(int32_t(left >> 30)) * kUnit;
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!, ...
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * s, x, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!, ...
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  if (quarter & 1u) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2u) {
    c = -c;
    s = -s;
  }
  return make_float2(c * f, s * f);
}

// N numbers at an address that is a multiple of their size.
template <bool kF32, int N>
__device__ __forceinline__ void load_numbers(const void* p, float* f) {
  if constexpr (kF32 && N == 4) {
    const float4 v = *static_cast<const float4*>(p);
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else if constexpr (kF32) {
    f[0] = *static_cast<const float*>(p);
  } else if constexpr (N == 1) {
    f[0] = __uint_as_float(uint32_t(*static_cast<const uint16_t*>(p)) << 16);
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const uint4 v = *static_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = *static_cast<const uint2*>(p);
      w[0] = v.x;
      w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <bool kF32, int N>
__device__ __forceinline__ void store_numbers(void* p, const float* f) {
  if constexpr (kF32 && N == 4) {
    *static_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else if constexpr (kF32) {
    *static_cast<float*>(p) = f[0];
  } else if constexpr (N == 1) {
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16(f[0]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if constexpr (N == 8) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* f) {
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) =
        make_uint2(f32x4_to_e4m3(f[0], f[1], f[2], f[3]), f32x4_to_e4m3(f[4], f[5], f[6], f[7]));
  else if constexpr (N == 4)
    *reinterpret_cast<uint32_t*>(p) = f32x4_to_e4m3(f[0], f[1], f[2], f[3]);
  else
    *p = uint8_t(f32x4_to_e4m3(f[0], 0.0f, 0.0f, 0.0f));
}

// N: numbers of a vector; N = 1 is for sizes, strides and addresses that longer ones do not
// fit, and for blocks whose table would be too large: a lane takes up to 4 pairs of a head
// and makes its angles itself.
template <bool kF32, int N, bool kCache>
__global__ void __launch_bounds__(kNrThreads, 2) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int E = kF32 ? 4 : 2, U = N == 1 ? 4 : 1;
  constexpr int kPasses = kNrHold / (2 * N * U);
  extern __shared__ __align__(16) uint8_t sm[];  // fractions [half], then the table
  uint64_t* fractions = reinterpret_cast<uint64_t*>(sm);
  float2* table = reinterpret_cast<float2*>(sm + (a.half * 8 + 15) / 16 * 16);
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int b = int(blockIdx.x / unsigned(a.J)), jw = int(blockIdx.x % unsigned(a.J));
  const int n = a.nn ? a.nn[b] : a.T, L = a.sl ? a.sl[b] : 0;
  if (L < 0 || n < 0 || n > a.T || (kCache && int64_t(L) + n > int64_t(a.MB) * a.bs)) {
    if (a.err && jw == 0 && blockIdx.y == 0 && tid == 0) atomicOr(a.err, SPEC_DERR_BAD_LENGTH);
    return;
  }
  int j = 0, first = 0, t0, cnt;  // the block, the offset of its first new token, the tokens
  if (kCache) {
    j = L / a.bs + jw;
    const int start = j * a.bs;
    first = max(L - start, 0);
    t0 = start + first - L;
    cnt = min(a.bs - first, n - t0);
  } else {
    t0 = jw * kNrTile;
    cnt = min(kNrTile, n - t0);
  }
  if (cnt <= 0) return;

  const int pairs = a.D / (2 * N), turning = a.half / N;  // vector pairs of a head
  const int lanes = pairs <= 1 ? 1 : N == 1 ? 32 : 1 << (32 - __clz(pairs - 1));  // of a head
  const int heads = 32 / lanes;                           // of a warp
  const int sub = lane / lanes, u = lane % lanes;
  const int32_t* pos = a.pos ? a.pos + int64_t(b) * a.T + t0 : nullptr;
  auto position = [&](int t) { return pos ? pos[t] : L + t0 + t; };
  for (int i = tid; i < a.half; i += kNrThreads) fractions[i] = turn_fraction(a.freq[i]);
  __syncthreads();
  if constexpr (N > 1) {
    for (int i = tid; i < cnt * a.half; i += kNrThreads) {
      const int t = i / a.half, p = i - t * a.half, x = p / N, y = p % N;
      // by halves of y, then x: the lanes of a head read 16 bytes side by side
      table[((t * (N / 2) + y / 2) * turning + x) * 2 + (y & 1)] =
          turned(fractions[p], position(t), a.factor);
    }
    __syncthreads();
  }

  // numbers of unit x of a head: vectors at ea and eb
  auto place = [&](int x, int& ea, int& eb) {
    const bool apart = !a.interleaved && x < turning;
    ea = apart ? x * N : 2 * x * N;
    eb = apart ? ea + a.half : ea + N;
  };
  auto fetch = [&](const uint8_t* head, bool on, float (*x)[2][N]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int w = u + 32 * i;
      int ea, eb;
      place(w, ea, eb);
      if (on && w < pairs) {
        load_numbers<kF32, N>(head + ea * E, x[i][0]);
        load_numbers<kF32, N>(head + eb * E, x[i][1]);
      } else {
#pragma unroll
        for (int y = 0; y < N; ++y) x[i][0][y] = x[i][1][y] = 0.0f;
      }
    }
  };
  // norm and turn of a head that `lanes` lanes hold
  auto finish = [&](float (*x)[2][N], const void* weight, int t) {
    if (weight) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int y = 0; y < N; ++y) s = fmaf(x[i][0][y], x[i][0][y], fmaf(x[i][1][y], x[i][1][y], s));
      for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float r = 1.0f / sqrtf(s / float(a.D) + a.eps);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int w = u + 32 * i;
        if (w >= pairs) continue;
        int ea, eb;
        place(w, ea, eb);
        float g[2][N];
        load_numbers<kF32, N>(static_cast<const uint8_t*>(weight) + ea * E, g[0]);
        load_numbers<kF32, N>(static_cast<const uint8_t*>(weight) + eb * E, g[1]);
#pragma unroll
        for (int y = 0; y < N; ++y) {
          x[i][0][y] *= r * g[0][y];
          x[i][1][y] *= r * g[1][y];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int w = u + 32 * i;
      if (w >= turning) continue;
      float2 cs[N];
      if constexpr (N == 1) {
        cs[0] = turned(fractions[w], position(t), a.factor);
      } else {
#pragma unroll
        for (int y = 0; y < N / 2; ++y) {
          const float4 v =
              *reinterpret_cast<const float4*>(&table[((t * (N / 2) + y) * turning + w) * 2]);
          cs[2 * y] = make_float2(v.x, v.y);
          cs[2 * y + 1] = make_float2(v.z, v.w);
        }
      }
      auto turn = [](float& p, float& q, float2 c) {
        const float x0 = p, y0 = q;
        p = x0 * c.x - y0 * c.y;
        q = y0 * c.x + x0 * c.y;
      };
      if (N == 1 || !a.interleaved) {
#pragma unroll
        for (int y = 0; y < N; ++y) turn(x[i][0][y], x[i][1][y], cs[y]);
      } else if constexpr (N > 1) {
#pragma unroll
        for (int y = 0; y < N / 2; ++y) {
          turn(x[i][0][2 * y], x[i][0][2 * y + 1], cs[y]);
          turn(x[i][1][2 * y], x[i][1][2 * y + 1], cs[N / 2 + y]);
        }
      }
    }
  };
  auto put = [&](uint8_t* head, bool on, float (*x)[2][N]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int w = u + 32 * i;
      int ea, eb;
      place(w, ea, eb);
      if (on && w < pairs) {
        store_numbers<kF32, N>(head + ea * E, x[i][0]);
        store_numbers<kF32, N>(head + eb * E, x[i][1]);
      }
    }
  };

  const int64_t token0 = int64_t(b) * a.T + t0;
  const int planes = kCache ? 2 * a.H : 0;
  const int q_groups = (a.Hq + 2 * heads - 1) / (2 * heads);
  const int k_groups = kCache ? 0 : (a.H + 2 * heads - 1) / (2 * heads);
  const int groups = q_groups + k_groups;
  const int64_t tasks = planes + int64_t(cnt) * groups;
  for (int64_t task = blockIdx.y * kNrWarps + (tid >> 5); task < tasks;
       task += int64_t(gridDim.y) * kNrWarps) {
    if (task >= planes) {
      // ---------------------------------------------------- two loads of a token's heads
      const int x = int(task - planes), t = x / groups;
      int g = x - t * groups;
      const bool is_k = g >= q_groups;
      if (is_k) g -= q_groups;
      const int h0 = 2 * g * heads + sub, many = is_k ? a.H : a.Hq;
      const uint8_t* from = is_k ? a.k + (token0 + t) * a.k_step : a.q + (token0 + t) * a.q_step;
      uint8_t* to = is_k ? a.ko + (token0 + t) * a.ko_step : a.qo + (token0 + t) * a.qo_step;
      const void* weight = is_k ? a.kw : a.qw;
      float x0[U][2][N], x1[U][2][N];
      const int64_t o0 = int64_t(h0) * a.D * E, o1 = o0 + int64_t(heads) * a.D * E;
      fetch(from + o0, h0 < many, x0);
      fetch(from + o1, h0 + heads < many, x1);
      finish(x0, weight, t);
      put(to + o0, h0 < many, x0);
      if (2 * g * heads + heads >= many) continue;
      finish(x1, weight, t);
      put(to + o1, h0 + heads < many, x1);
    } else if constexpr (kCache) {
      // ---------------------------------------------------- a plane and head of the block
      const int plane = task >= a.H, h = int(task) - plane * a.H;
      const uint8_t* from = (plane ? a.v : a.k) + int64_t(h) * a.D * E;
      const int64_t step = plane ? a.v_step : a.k_step;
      const void* weight = plane ? nullptr : a.kw;
      const int id = a.bt[int64_t(b) * a.MB + j];
      auto head_of = [&](int t) { return from + (token0 + t) * step; };
      auto make = [&](float (*x)[2][N], int t) {
        if (plane == 0) finish(x, weight, min(t, cnt - 1));
      };
      uint32_t top = 0;
      auto larger = [&](const float (*x)[2][N]) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int y = 0; y < N; ++y)
            top = max(top, max(__float_as_uint(x[i][0][y]) & 0x7fffffffu,
                               __float_as_uint(x[i][1][y]) & 0x7fffffffu));
      };
      // NaN becomes 0, infinities the largest finite number (a NaN code would spread to
      // rows that do not see its token)
      auto guard = [&](float (*x)[2][N]) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int y = 0; y < 2 * N; ++y) {
            float& f = x[i][y / N][y % N];
            f = f != f ? 0.0f : fminf(fmaxf(f, -FLT_MAX), FLT_MAX);
          }
      };
      float x[kPasses][U][2][N];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int t = p * heads + sub;
        fetch(head_of(t), t < cnt, x[p]);
      }
      if (id < 0 || id >= a.NB) {
        if (a.err && lane == 0) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
        continue;
      }
      uint8_t* codes = a.pool + id * a.block_bytes + int64_t(task) * a.bs * a.D;
      float* sp = a.scales + id * a.block_scales + task;
      const float was = first > 0 ? *sp : 0.0f;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        if (p * heads >= cnt) continue;
        make(x[p], p * heads + sub);
        larger(x[p]);
      }
#pragma unroll 1
      for (int t = kPasses * heads; t < cnt; t += heads) {
        float y[U][2][N];
        fetch(head_of(t + sub), t + sub < cnt, y);
        make(y, t + sub);
        larger(y);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const bool bad = top >= 0x7f800000u;
      if (bad) {
        top = 0;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          guard(x[p]);
          larger(x[p]);
        }
#pragma unroll 1
        for (int t = kPasses * heads; t < cnt; t += heads) {
          float y[U][2][N];
          fetch(head_of(t + sub), t + sub < cnt, y);
          make(y, t + sub);
          guard(y);
          larger(y);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (a.err && lane == 0) atomicOr(a.err, SPEC_DERR_VALUE);
      }
      float scale = q8_pow2(q8_scale_exp(__uint_as_float(top)));
      if (first > 0) scale = fmaxf(scale, was);
      // an older and larger scale may be any number that the caller has put there
      const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
      const float inv = 1.0f / scale;
      if (first > 0 && scale != was) {
        const float r = was / scale;
        for (int i = lane; i < first * a.D / 16; i += 32) {
          uint4 c = *reinterpret_cast<const uint4*>(codes + i * 16);
          uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float f[4];
            e4m3x4_to_f32(w[y], f);
            w[y] = f32x4_to_e4m3(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
          }
          *reinterpret_cast<uint4*>(codes + i * 16) = c;
        }
      }
      auto encode = [&](float (*v)[2][N], int t) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int w = u + 32 * i;
          int ea, eb;
          place(w, ea, eb);
          if (t >= cnt || w >= pairs) continue;
#pragma unroll
          for (int y = 0; y < 2 * N; ++y) {
            float& f = v[i][y / N][y % N];
            f = exact ? f * inv : f / scale;
          }
          uint8_t* to = codes + int64_t(first + t) * a.D;
          store_codes<N>(to + ea, v[i][0]);
          store_codes<N>(to + eb, v[i][1]);
        }
      };
#pragma unroll
      for (int p = 0; p < kPasses; ++p) encode(x[p], p * heads + sub);
#pragma unroll 1
      for (int t = kPasses * heads; t < cnt; t += heads) {
        float y[U][2][N];
        fetch(head_of(t + sub), t + sub < cnt, y);
        make(y, t + sub);
        if (bad) guard(y);
        encode(y, t + sub);
      }
      if (lane == 0) *sp = scale;
    }
  }
}

namespace {

template <bool kF32, int N, bool kCache>
int launch_shape(const NormRopeArgs& a, int tokens, int sms, cudaStream_t st) {
  auto kern = norm_rope_kernel<kF32, N, kCache>;
  const size_t fractions = (size_t(a.half) * 8 + 15) / 16 * 16;
  const size_t smem = fractions + (N > 1 ? size_t(tokens) * a.half * 8 : 0);
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kern, kNrTable + 2048, done) != SPEC_OK) return SPEC_ECUDA;
  // few tokens: the tasks of a tile over several CTAs, up to a task for each warp
  const int64_t tiles = int64_t(a.B) * a.J;
  const int pairs = a.D / (2 * N);
  int lanes = N == 1 ? 32 : 1;
  while (lanes < pairs && lanes < 32) lanes *= 2;
  const int heads = 2 * (32 / lanes);
  const int64_t groups = (a.Hq + heads - 1) / heads + (kCache ? 0 : (a.H + heads - 1) / heads);
  const int64_t tasks = (kCache ? 2 * a.H : 0) + groups * (tokens < a.T ? tokens : a.T);
  int64_t parts = 2 * int64_t(sms) / tiles, most = (tasks + kNrWarps - 1) / kNrWarps;
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  if (tiles > INT32_MAX) return SPEC_ENOTSUP;
  if (parts > 65535) parts = 65535;
  return launch_pdl(kern, dim3(unsigned(tiles), unsigned(parts)), dim3(kNrThreads), smem, st, a);
}

template <bool kF32, bool kCache>
int launch_type(const NormRopeArgs& a, int tokens, int sms, uintptr_t bits, cudaStream_t st) {
  // `bits`: every address and stride or-ed together
  const bool table = int64_t(tokens) * a.half * 8 <= kNrTable;
  auto fits = [&](int n) {
    return table && a.half % n == 0 && a.D % (2 * n) == 0 && bits % (n * (kF32 ? 4 : 2)) == 0;
  };
  if constexpr (!kF32)
    if (fits(8)) return launch_shape<kF32, 8, kCache>(a, tokens, sms, st);
  if (fits(4)) return launch_shape<kF32, 4, kCache>(a, tokens, sms, st);
  return launch_shape<kF32, 1, kCache>(a, tokens, sms, st);
}

}  // namespace

int launch_norm_rope(const NormRopeLaunch& r) {
  NormRopeArgs a = {};
  const int E = r.dtype == SPEC_F32 ? 4 : 2;
  a.q = static_cast<const uint8_t*>(r.q);
  a.k = static_cast<const uint8_t*>(r.k);
  a.v = static_cast<const uint8_t*>(r.v);
  a.qo = static_cast<uint8_t*>(r.q_out);
  a.ko = static_cast<uint8_t*>(r.k_out);
  a.q_step = r.q_stride * E;
  a.k_step = r.k_stride * E;
  a.v_step = r.v_stride * E;
  a.qo_step = r.q_out_stride * E;
  a.ko_step = r.k_out_stride * E;
  a.qw = r.q_weight;
  a.kw = r.k_weight;
  a.freq = r.inv_freq;
  a.sl = r.seq_lens;
  a.nn = r.num_new;
  a.pos = r.positions;
  a.Hq = r.Hq;
  a.H = r.H;
  a.D = r.D;
  a.half = r.half;
  a.B = r.B;
  a.T = r.T;
  a.interleaved = r.interleaved;
  a.eps = r.eps;
  a.factor = r.factor;
  a.err = r.err;
  uintptr_t bits = 0;
  for (const void* p : {r.q, r.k, r.v, (const void*)r.q_out, (const void*)r.k_out, r.q_weight,
                        r.k_weight})
    bits |= reinterpret_cast<uintptr_t>(p);
  bits |= uintptr_t(a.q_step | a.k_step | a.v_step | a.qo_step | a.ko_step);
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ECUDA;
  if (dev < 64) sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ECUDA;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  cudaStream_t st = static_cast<cudaStream_t>(r.stream);
  if (!r.pool) {
    a.J = (r.T + kNrTile - 1) / kNrTile;
    const int tokens = r.T < kNrTile ? r.T : kNrTile;
    return r.dtype == SPEC_F32 ? launch_type<true, false>(a, tokens, sms, bits, st)
                               : launch_type<false, false>(a, tokens, sms, bits, st);
  }
  const int64_t layer_bytes = int64_t(2) * r.H * r.bs * r.D;
  a.pool = static_cast<uint8_t*>(r.pool) + r.layer * layer_bytes;
  a.scales = r.scales + int64_t(r.layer) * 2 * r.H;
  a.bt = r.block_table;
  a.NB = r.num_blocks;
  a.bs = r.bs;
  a.MB = r.max_blocks;
  a.J = (r.T + 2 * r.bs - 2) / r.bs;
  a.block_bytes = r.num_layers * layer_bytes;
  a.block_scales = int64_t(r.num_layers) * 2 * r.H;
  const int tokens = r.T < r.bs ? r.T : r.bs;
  return r.dtype == SPEC_F32 ? launch_type<true, true>(a, tokens, sms, bits, st)
                             : launch_type<false, true>(a, tokens, sms, bits, st);
}

}  // namespace sv
