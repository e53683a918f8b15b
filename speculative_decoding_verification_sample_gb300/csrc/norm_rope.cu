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
// a turn is one integer product, exact to 2^-53 turns per position (times |inv_freq| above 1: the
// quotient by 2 pi is fp64's); an fp32 angle of position 100 000 would be off by 0.004 rad, which
// keys and queries far from each other do not share. sin and cos of the eighth turn that is left are Taylor polynomials (the
// first terms left out are below 2e-9 and 2e-10).
//
// Split. A CTA takes the new tokens of one cache block (without a cache: 16 or 8 tokens) of
// a row: it makes their table of cos and sin in shared memory once for all heads, then its
// warps take tasks. A lane holds two vectors of a head, those that belong to each other in
// the turn, so that only the norm's sum crosses lanes: 8 lanes a head of 128 bf16 numbers,
// 4 heads a warp, a unit. A task is up to 4 units (8 with 8-byte vectors) of queries, or with
// a cache a plane and head of the block, whose numbers are taken twice from shared memory:
// for the maximum, then for the rounding. Each warp copies its next task while it works on
// one, a lane its own numbers. Few tokens: the tasks of a block are split over several CTAs,
// each with the table.
//
// Bound by memory for long prompts (every number is read and written once) and, next to
// that, by the instructions: about 20 a number (loads into registers with two CTAs an SM,
// all tasks unrolled, took 306 us where this takes 150: 12 prompts, 0.85 GB, 5.5 TB/s; pairs
// of numbers in one instruction took as many with the moves that they need, 157). Prompts without
// the cache wait: 4 rows of 4099 tokens take 74 us (floor 50) with the memory at 47 % and the
// issue slots at 42 %, as 2052 CTAs of 8 tokens each begin with lengths, fractions and the table.
// Verification steps of 256 rows take the device 13 us without and 17 with the cache (floor 4),
// one token 3 and 4 us; a call from Python takes at least 11 to 15 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace sv {

constexpr int kNrThreads = 256, kNrWarps = kNrThreads / 32;
constexpr int kNrTile = 16;              // tokens of a CTA without a cache, at most
constexpr int kNrTable = 64 * 1024;      // bytes of cos and sin at most

struct NormRopeArgs {
  const uint8_t *q, *k, *v;              // first token; v: with a cache
  uint8_t *qo, *ko;                      // ko: without a cache
  int64_t q_step, k_step, v_step, qo_step, ko_step;  // bytes from token to token
  const void *qw, *kw;                   // [D] of the tensors' type; null: no norm
  const float* freq;                     // [half]
  const int32_t *sl, *nn, *pos;          // pos [B, T]; null: sl + t. nn null: T
  int Hq, H, D, half, B, T;
  float eps, factor;
  uint8_t* pool;                         // at the layer; the rest is for a cache
  float* scales;
  const int32_t* bt;
  int NB, bs, MB, J;                     // J: blocks (tiles) that T tokens can touch
  int64_t block_bytes, block_scales;
  int tile;                              // tokens of a CTA without a cache
  int per;                               // units of a task
  int32_t* err;
};

// A frequency as a fraction of a turn, in units of 2^-64. From 2^52 turns on the quotient has no
// fraction left, and gives 0, as infinities and NaN do.
__device__ __forceinline__ uint64_t turn_fraction(float w) {
  double t = double(w) * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return t < 1.0 ? static_cast<uint64_t>(t * 18446744073709551616.0) : 0ull;
}

// cos and sin of p * (fraction of a turn), times f.
__device__ __forceinline__ float2 turned(uint64_t fraction, int64_t p, float f) {
  const uint64_t a = fraction * static_cast<uint64_t>(p);
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

// N numbers at an address that is a multiple of their size, as they are, in W registers.
template <bool kF32, int N>
constexpr int kNrWords = N == 1 ? 1 : N * (kF32 ? 4 : 2) / 4;

template <bool kF32, int N>
__device__ __forceinline__ void load_raw(const void* p, uint32_t* w) {
  if constexpr (kNrWords<kF32, N> == 4) {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (kNrWords<kF32, N> == 2) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else if constexpr (kF32) {
    w[0] = *static_cast<const uint32_t*>(p);
  } else {
    w[0] = *static_cast<const uint16_t*>(p);
  }
}

template <bool kF32, int N>
__device__ __forceinline__ void widen(const uint32_t* w, float* f) {
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
  } else if constexpr (N == 1) {
    f[0] = __uint_as_float(w[0] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// N numbers from global to shared memory; cp_async_wait before they are read.
template <bool kF32, int N>
__device__ __forceinline__ void copy_raw(uint8_t* to, const uint8_t* from) {
  constexpr int kBytes = 4 * kNrWords<kF32, N>;
  if constexpr (!kF32 && N == 1)  // (there is no such copy of 2 bytes)
    *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint16_t*>(from);
  else if constexpr (kBytes == 16)
    cp_async16(to, from, true);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from),
                 "n"(kBytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>  // all groups but the newest N
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// A warp's ring: two tasks' numbers as they are, units of `heads` heads, two vectors a lane.
constexpr int kNrHalf = 4096;
template <bool kF32, int N>
constexpr int kNrUnits = kNrHalf / ((N == 1 ? 4 : 1) * 2 * 32 * 4 * kNrWords<kF32, N>);
constexpr int kNrCtas = 3;  // of an SM

// N: numbers of a vector; N = 1 is for sizes, strides and addresses that longer ones do not
// fit, and for blocks whose table would be too large: a lane takes up to 4 pairs of a head
// and makes its angles itself.
template <bool kF32, int N, bool kCache, bool kInterleaved>
__global__ void __launch_bounds__(kNrThreads, kNrCtas) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int E = kF32 ? 4 : 2, U = N == 1 ? 4 : 1, W = kNrWords<kF32, N>;
  constexpr int kUnits = kNrUnits<kF32, N>;
  extern __shared__ __align__(16) uint8_t sm[];  // rings, fractions [half], weights [2][D], the table
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
    t0 = jw * a.tile;
    cnt = min(a.tile, n - t0);
  }
  if (cnt <= 0) return;

  const int pairs = a.D / (2 * N), turning = a.half / N;  // vector pairs of a head
  const int lanes = pairs <= 1 ? 1 : N == 1 ? 32 : 1 << (32 - __clz(pairs - 1));  // of a head
  const int heads = 32 / lanes;                           // of a warp
  const int sub = lane / lanes, u = lane % lanes;
  // numbers of unit x of a head: vectors at ea and eb
  auto place = [&](int x, int& ea, int& eb) {
    const bool apart = !kInterleaved && x < turning;
    ea = apart ? x * N : 2 * x * N;
    eb = apart ? ea + a.half : ea + N;
  };
  int off[U][2];  // a lane's vectors in a head, bytes
#pragma unroll
  for (int i = 0; i < U; ++i) {
    int ea, eb;
    place(u + 32 * i, ea, eb);
    off[i][0] = ea * E;
    off[i][1] = eb * E;
  }
  // A lane reads only what it has copied itself; where there is nothing (lanes beyond a head,
  // heads and tokens beyond the last) it copies nothing, and what it makes of that is not used.
  constexpr int kVector = 32 * 4 * W, kUnit = U * 2 * kVector;
  uint8_t* const mine = sm + (tid >> 5) * 2 * kNrHalf + lane * 4 * W;
  int half_at = 0;  // of the task at work
  auto fetch = [&](const uint8_t* head, bool on, uint8_t* to) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (on && u + 32 * i < pairs) {
        copy_raw<kF32, N>(to + 2 * i * kVector, head + off[i][0]);
        copy_raw<kF32, N>(to + (2 * i + 1) * kVector, head + off[i][1]);
      }
  };

  // A task: a plane and head of the block, or `per` units of queries (without a cache: and
  // keys), token by token. A plane's tokens beyond what a warp holds follow in further loads.
  const int64_t token0 = int64_t(b) * a.T + t0;
  const int planes = kCache ? 2 * a.H : 0;
  const int q_groups = (a.Hq + heads - 1) / heads;
  const int groups = q_groups + (kCache ? 0 : (a.H + heads - 1) / heads);
  const int units = cnt * groups;
  const int tasks = planes + (units + a.per - 1) / a.per;
  const int head_step = heads * a.D * E;
  auto fetch_plane = [&](int task, int t, uint8_t* to) {
    const int plane = task >= a.H, h = task - plane * a.H;
    const int64_t step = plane ? a.v_step : a.k_step, unit_step = heads * step;
    const uint8_t* from = (plane ? a.v : a.k) + (token0 + t + sub) * step + int64_t(h) * a.D * E;
#pragma unroll 1
    for (const uint8_t* end = to + kNrHalf; to < end && t < cnt; to += kUnit) {
      fetch(from, t + sub < cnt, to);
      from += unit_step;
      t += heads;
    }
  };
  // the units from `first_unit`: f(head, whether there is one, token, keys, place in the ring)
  auto walk = [&](int first_unit, const uint8_t* q, int64_t q_step, const uint8_t* k,
                  int64_t k_step, uint8_t* at, auto&& f) {
    int t = first_unit / groups, g = first_unit - t * groups;
    const uint8_t* const end = at + a.per * kUnit;
#pragma unroll 1
    while (at < end && t < cnt) {
      // units of one tensor and token
      const bool is_k = !kCache && g >= q_groups;
      const int64_t first_head = int64_t(is_k ? g - q_groups : g) * heads + sub;
      const uint8_t* head = (is_k ? k : q) + (token0 + t) * (is_k ? k_step : q_step) +
                            first_head * (a.D * E);
      int left = (is_k ? a.H : a.Hq) - int(first_head);  // heads from there
      const int g_end = is_k ? groups : q_groups;
#pragma unroll 1
      do {
        f(head, left > 0, t, is_k, at);
        head += head_step;
        left -= heads;
        at += kUnit;
      } while (++g < g_end && at < end);
      if (g == groups) g = 0, ++t;
    }
  };
  auto fetch_units = [&](int first_unit, uint8_t* to) {
    walk(first_unit, a.q, a.q_step, a.k, a.k_step, to,
         [&](const uint8_t* head, bool on, int, bool, uint8_t* at) { fetch(head, on, at); });
  };
  auto fetch_task = [&](int task, uint8_t* to) {
    if (task < planes) fetch_plane(task, 0, to);
    else if (task < tasks) fetch_units((task - planes) * a.per, to);
    cp_async_commit();
  };
  int task = blockIdx.y * kNrWarps + (tid >> 5);
  fetch_task(task, mine);

  // ------------------------------------------------------------------ the tile's table
  uint64_t* fractions = reinterpret_cast<uint64_t*>(sm + kNrWarps * 2 * kNrHalf);
  float4* weights = reinterpret_cast<float4*>(fractions + (a.half + 1) / 2 * 2);
  float4* table = weights + a.D / 2;
  const int32_t* pos = a.pos ? a.pos + int64_t(b) * a.T + t0 : nullptr;
  // (in 64 bits: the tokens after a length near the largest int are past it)
  auto position = [&](int t) -> int64_t { return pos ? pos[t] : int64_t(L) + t0 + t; };
  for (int i = tid; i < a.half; i += kNrThreads) fractions[i] = turn_fraction(a.freq[i]);
  if constexpr (N > 1) {
    // by quarters of what a lane needs of them: the lanes of a head read side by side
    for (int i = tid; i < 2 * pairs; i += kNrThreads) {
      const int w = i % pairs;
      const uint8_t* from = static_cast<const uint8_t*>(i < pairs ? a.qw : a.kw);
      if (!from) continue;
      int ea, eb;
      place(w, ea, eb);
      uint32_t r[2][W];
      float f[2][N];
      load_raw<kF32, N>(from + ea * E, r[0]);
      load_raw<kF32, N>(from + eb * E, r[1]);
      widen<kF32, N>(r[0], f[0]);
      widen<kF32, N>(r[1], f[1]);
      float4* to = weights + (i < pairs ? 0 : a.D / 4) + w;
#pragma unroll
      for (int y = 0; y < 2 * N; y += 4)
        to[y / 4 * pairs] =
            make_float4(f[y / N][y % N], f[y / N][y % N + 1], f[y / N][y % N + 2], f[y / N][y % N + 3]);
    }
  }
  __syncthreads();
  if constexpr (N > 1) {
    float* to = reinterpret_cast<float*>(table);
    for (int i = tid; i < cnt * a.half; i += kNrThreads) {
      const int t = i / a.half, p = i - t * a.half, x = p / N, y = p % N;
      const float2 v = turned(fractions[p], position(t), a.factor);
      // N cosines, then N sines, by four
      const int at = (t * (N / 2) + y / 4) * turning + x;
      to[4 * at + y % 4] = v.x;
      to[4 * (at + N / 4 * turning) + y % 4] = v.y;
    }
    __syncthreads();
  }

  // norm and turn of a head that `lanes` lanes hold
  const float share = 1.0f / float(a.D);
  auto finish = [&](float (*x)[2][N], int is_k, int t) {
    const void* weight = is_k ? a.kw : a.qw;
    if (weight) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float one = 0.0f, two = 0.0f;
#pragma unroll
        for (int y = 0; y < N; ++y) {
          one = fmaf(x[i][0][y], x[i][0][y], one);
          two = fmaf(x[i][1][y], x[i][1][y], two);
        }
        if (u + 32 * i < pairs) s += one + two;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float r = rsqrtf(fmaf(s, share, a.eps));
      if constexpr (N > 1) {
        if (u < pairs) {
          const float4* from = weights + (is_k ? a.D / 4 : 0) + u;
#pragma unroll
          for (int y = 0; y < 2 * N; y += 4) {
            const float4 v = from[y / 4 * pairs];
            const float g[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) x[0][(y + z) / N][(y + z) % N] *= r * g[z];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int w = u + 32 * i;
          if (w >= pairs) continue;
          uint32_t g[2][W];
          float f[2];
          load_raw<kF32, N>(static_cast<const uint8_t*>(weight) + off[i][0], g[0]);
          load_raw<kF32, N>(static_cast<const uint8_t*>(weight) + off[i][1], g[1]);
          widen<kF32, N>(g[0], f);
          widen<kF32, N>(g[1], f + 1);
          x[i][0][0] *= r * f[0];
          x[i][1][0] *= r * f[1];
        }
      }
    }
    auto turn = [](float& p, float& q, float c, float s) {
      const float x0 = p, y0 = q;
      p = x0 * c - y0 * s;
      q = y0 * c + x0 * s;
    };
    if constexpr (N == 1) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int w = u + 32 * i;
        if (w >= turning) continue;
        const float2 v = turned(fractions[w], position(t), a.factor);
        turn(x[i][0][0], x[i][1][0], v.x, v.y);
      }
    } else if (u < turning) {
      const float4* from = table + t * (N / 2) * turning + u;
#pragma unroll
      for (int y = 0; y < N; y += 4) {
        const float4 vc = from[y / 4 * turning], vs = from[(N + y) / 4 * turning];
        const float c[4] = {vc.x, vc.y, vc.z, vc.w}, s[4] = {vs.x, vs.y, vs.z, vs.w};
        if constexpr (!kInterleaved) {
#pragma unroll
          for (int z = 0; z < 4; ++z) turn(x[0][0][y + z], x[0][1][y + z], c[z], s[z]);
        } else {
          // pairs 4 (y / 4) ... of the unit: of its first vector, then of the second
          float* p = &x[0][2 * y / N][2 * y % N];
          turn(p[0], p[1], c[0], s[0]);
          turn(p[2], p[3], c[1], s[1]);
          p = &x[0][(2 * y + 4) / N][(2 * y + 4) % N];
          turn(p[0], p[1], c[2], s[2]);
          turn(p[2], p[3], c[3], s[3]);
        }
      }
    }
  };
  auto number = [&](const uint8_t* from, float (*x)[2][N]) {
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) {
      uint32_t w[W];
      load_words<W>(from + i * kVector, w);
      widen<kF32, N>(w, x[i / 2][i % 2]);
    }
  };

  const int stride = gridDim.y * kNrWarps;
#pragma unroll 1
  for (; task < tasks; task += stride, half_at ^= kNrHalf) {
    uint8_t* const held = mine + half_at;
    fetch_task(task + stride, mine + (half_at ^ kNrHalf));
    cp_async_wait<1>();
    if (task >= planes) {
      // ---------------------------------------------------- units of queries and keys
      walk((task - planes) * a.per, a.qo, a.qo_step, a.ko, a.ko_step, held,
           [&](const uint8_t* at, bool on, int t, bool is_k, uint8_t* from) {
             float x[U][2][N];
             number(from, x);
             finish(x, is_k, t);
             uint8_t* head = const_cast<uint8_t*>(at);
#pragma unroll
             for (int i = 0; i < U; ++i)
               if (on && u + 32 * i < pairs) {
                 store_numbers<kF32, N>(head + off[i][0], x[i][0]);
                 store_numbers<kF32, N>(head + off[i][1], x[i][1]);
               }
           });
    } else if constexpr (kCache) {
      // ---------------------------------------------------- a plane and head of the block
      const int plane = task >= a.H;
      const int id = a.bt[int64_t(b) * a.MB + j];
      if (id < 0 || id >= a.NB) {
        if (a.err && lane == 0) atomicOr(a.err, SPEC_DERR_BAD_BLOCK);
        continue;
      }
      uint8_t* codes = a.pool + id * a.block_bytes + int64_t(task) * a.bs * a.D;
      float* sp = a.scales + id * a.block_scales + task;
      const float was = first > 0 ? *sp : 0.0f;
      // f(numbers, token) for all tokens of the block, made from what is held or loaded again
      const int span = kUnits * heads;
      bool again = false;
      auto sweep = [&](auto&& f) {
#pragma unroll 1
        for (int c = 0; c < cnt; c += span) {
          if (again || c > 0) {
            fetch_plane(task, c, held);
            cp_async_commit();
            cp_async_wait<0>();
          }
#pragma unroll 1
          for (int i = 0; i < kUnits && c + i * heads < cnt; ++i) {
            const int t = c + i * heads + sub;
            float x[U][2][N];
            number(held + i * kUnit, x);
            if (plane == 0) finish(x, 1, min(t, cnt - 1));
            f(x, t);
          }
        }
        again = cnt > span;
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
      uint32_t top = 0;
      bool bad = false;
#pragma unroll 1
      for (;;) {
        sweep([&](float (*x)[2][N], int t) {
          if (bad) guard(x);
          if (t >= cnt) return;
#pragma unroll
          for (int i = 0; i < U; ++i)
#pragma unroll
            for (int y = 0; y < N && u + 32 * i < pairs; ++y)
              top = max(top, max(__float_as_uint(x[i][0][y]) & 0x7fffffffu,
                                 __float_as_uint(x[i][1][y]) & 0x7fffffffu));
        });
        top = __reduce_max_sync(0xffffffffu, top);
        if (bad || top < 0x7f800000u) break;
        bad = true;
        top = 0;
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
      sweep([&](float (*x)[2][N], int t) {
        if (bad) guard(x);
        if (t >= cnt) return;
        uint8_t* to = codes + int64_t(first + t) * a.D;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          if (u + 32 * i >= pairs) continue;
          float* f = x[i][0];
          if (exact) {
#pragma unroll
            for (int y = 0; y < 2 * N; ++y) f[y] *= inv;
          } else {
#pragma unroll
            for (int y = 0; y < 2 * N; ++y) f[y] /= scale;
          }
          store_codes<N>(to + off[i][0] / E, x[i][0]);
          store_codes<N>(to + off[i][1] / E, x[i][1]);
        }
      });
      if (lane == 0) *sp = scale;
    }
  }
}

namespace {

template <bool kF32, int N, bool kCache, bool kInterleaved>
int launch_shape(const NormRopeArgs& a, int tokens, int sms, cudaStream_t st) {
  auto kern = norm_rope_kernel<kF32, N, kCache, kInterleaved>;
  const size_t fractions = (size_t(a.half) * 8 + 15) / 16 * 16;
  const size_t smem = kNrWarps * 2 * kNrHalf + fractions + (N > 1 ? size_t(a.D) * 8 + size_t(tokens) * a.half * 8 : 0);
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kern, kNrWarps * 2 * kNrHalf + kNrTable + 4096, done) != SPEC_OK) return SPEC_ECUDA;
  // few tokens: the tasks of a tile over several CTAs, up to a task for each warp, and less in
  // a task than a warp can hold
  const int64_t tiles = int64_t(a.B) * a.J;
  if (tiles > INT32_MAX) return SPEC_ENOTSUP;
  const int pairs = a.D / (2 * N);
  int lanes = N == 1 ? 32 : 1;
  while (lanes < pairs && lanes < 32) lanes *= 2;
  const int heads = 32 / lanes;
  const int64_t groups = (a.Hq + heads - 1) / heads + (kCache ? 0 : (a.H + heads - 1) / heads);
  const int64_t units = groups * (tokens < a.T ? tokens : a.T);
  if (units > INT32_MAX / 2) return SPEC_ENOTSUP;
  // The longer the tasks, the fewer of them wait: the longest that leave no warp much less
  // to do than another.
  const int64_t each = units * tiles / (int64_t(sms) * kNrCtas * kNrWarps);  // of a warp
  const int most_units = each < 1 ? 1 : each < kNrUnits<kF32, N> ? int(each) : kNrUnits<kF32, N>;
  NormRopeArgs with = a;
  int64_t least = INT64_MAX;
  for (int per = most_units; per > 0; --per) {
    const int64_t rounds = ((units + per - 1) / per + kNrWarps - 1) / kNrWarps * per;
    if (rounds < least) least = rounds, with.per = per;
  }
  const int64_t tasks = (kCache ? 2 * a.H : 0) + (units + with.per - 1) / with.per;
  int64_t parts = kNrCtas * int64_t(sms) / tiles, most = (tasks + kNrWarps - 1) / kNrWarps;
  parts = parts < 1 ? 1 : parts > most ? most : parts;
  if (parts > 65535) parts = 65535;
  return launch_pdl(kern, dim3(unsigned(tiles), unsigned(parts)), dim3(kNrThreads), smem, st, with);
}

template <bool kF32, bool kCache, bool kInterleaved>
int launch_type(const NormRopeArgs& a, int tokens, int sms, uintptr_t bits, cudaStream_t st) {
  // `bits`: every address and stride or-ed together
  const bool table = int64_t(tokens) * a.half * 8 <= kNrTable;
  auto fits = [&](int n) {
    return table && a.half % n == 0 && a.D % (2 * n) == 0 && bits % (n * (kF32 ? 4 : 2)) == 0;
  };
  if constexpr (!kF32)
    if (fits(8)) return launch_shape<kF32, 8, kCache, kInterleaved>(a, tokens, sms, st);
  if (fits(4)) return launch_shape<kF32, 4, kCache, kInterleaved>(a, tokens, sms, st);
  return launch_shape<kF32, 1, kCache, kInterleaved>(a, tokens, sms, st);
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
  auto launch = [&](auto cache, int tokens) {
    constexpr bool kCache = decltype(cache)::value;
    const bool f32 = r.dtype == SPEC_F32;
    if (r.interleaved)
      return f32 ? launch_type<true, kCache, true>(a, tokens, sms, bits, st)
                 : launch_type<false, kCache, true>(a, tokens, sms, bits, st);
    return f32 ? launch_type<true, kCache, false>(a, tokens, sms, bits, st)
               : launch_type<false, kCache, false>(a, tokens, sms, bits, st);
  };
  if (!r.pool) {
    // half of it where the last round of CTAs would be a large part of them all
    a.tile = int64_t(r.B) * ((r.T + kNrTile - 1) / kNrTile) > int64_t(4) * sms * kNrCtas
                 ? kNrTile
                 : kNrTile / 2;
    a.J = (r.T + a.tile - 1) / a.tile;
    return launch(std::false_type{}, r.T < a.tile ? r.T : a.tile);
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
  return launch(std::true_type{}, r.T < r.bs ? r.T : r.bs);
}

}  // namespace sv
