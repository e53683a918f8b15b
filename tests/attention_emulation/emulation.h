// The tensor-core attention kernel's source compiled for the host: one CTA, a fiber per
// thread, in a random order of the warps. What the kernel waits for and synchronises with
// is modelled as documented: mbarriers (phases, arrivals, bytes), named barriers, warp-wide
// instructions, asynchronous copies, products and commits with random durations, TMEM's
// allocation and columns. The numbers are not: scores are random, a copy moves nothing.
//
// Ends the program with a message where the kernel would do what is not defined: an
// arrival too many, lanes of a warp at different warp-wide instructions, threads of a
// barrier at different ones, memory or TMEM outside its bounds, an exit with copies or
// products in flight, threads that wait for ever.
#pragma once
#include <sys/mman.h>
#include <ucontext.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <random>
#include <string>
#include <type_traits>
#include <utility>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __noinline__ __attribute__((noinline))
#define __launch_bounds__(...)
#define __grid_constant__

struct dim3 {
  unsigned x = 1, y = 1, z = 1;
};
struct alignas(8) float2 { float x, y; };
struct alignas(16) float4 { float x, y, z, w; };
struct alignas(8) int2 { int x, y; };
struct alignas(16) int4 { int x, y, z, w; };
struct alignas(8) uint2 { uint32_t x, y; };
struct alignas(16) uint4 { uint32_t x, y, z, w; };
struct alignas(16) ulonglong2 { unsigned long long x, y; };
inline float2 make_float2(float a, float b) { return {a, b}; }
inline int2 make_int2(int a, int b) { return {a, b}; }
inline int4 make_int4(int a, int b, int c, int d) { return {a, b, c, d}; }
inline uint2 make_uint2(uint32_t a, uint32_t b) { return {a, b}; }
inline uint4 make_uint4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return {a, b, c, d}; }
struct CUtensorMap {};
using std::max;
using std::min;

template <class To, class From>
To bits(From x) {
  To u{};
  memcpy(&u, &x, std::min(sizeof u, sizeof x));
  return u;
}
inline uint32_t __float_as_uint(float f) { return bits<uint32_t>(f); }
inline float __uint_as_float(uint32_t u) { return bits<float>(u); }
struct __nv_bfloat16 {
  uint16_t b;
  explicit __nv_bfloat16(float f) : b(__float_as_uint(f) >> 16) {}
};
inline __nv_bfloat16 __float2bfloat16(float f) { return __nv_bfloat16(f); }

// ------------------------------------------------------------------ threads
struct Fiber {
  ucontext_t context;
  int id;
  bool done = false;
  std::function<bool()> ready;  // what it waits for
  const char* where = "";
  int line = 0;
};
inline std::vector<Fiber> fibers;
inline Fiber* cur;
inline ucontext_t scheduler;
inline std::mt19937 rng;
inline uint64_t now_ns;
inline dim3 blockIdx, gridDim, blockDim;
struct Tid {
  struct {
    operator int() const { return cur->id; }
  } x;
};
inline Tid threadIdx;

[[noreturn]] inline void fail(const std::string& what) {
  printf("FAIL: %s (thread %d, %.1f us)\n", what.c_str(), cur ? cur->id : -1, 1e-3 * now_ns);
  fflush(stdout);
  _Exit(1);
}
inline void wait_for(std::function<bool()> f, const char* where, int line) {
  if (f()) return;
  cur->ready = f;
  cur->where = where;
  cur->line = line;
  swapcontext(&cur->context, &scheduler);
  cur->ready = nullptr;
}

struct Event {  // an asynchronous completion
  uint64_t t;
  std::function<void()> f;
};
inline std::vector<Event> events;
inline bool stalling;  // one of them comes so late that waits run out
inline int late_in;    // how many come before it
inline uint64_t after(uint64_t most) {
  return now_ns + 1 + rng() % most + (stalling && late_in-- == 0 ? 350000 + rng() % 600000 : 0);
}

// ------------------------------------------------------------------ warps
struct Collective {
  int n = 0, round = 0, line = 0;
  const char* kind = nullptr;
  uint64_t in[32], out[32];
};
inline Collective collectives[64];
// Every lane of the warp has to come to the same one.
inline const uint64_t* collective(const char* kind, int line, uint64_t v) {
  Collective& c = collectives[cur->id / 32];
  if (c.n == 0) {
    c.kind = kind;
    c.line = line;
  } else if (c.line != line || strcmp(c.kind, kind)) {
    fail(std::string("a warp's lanes at ") + kind + " in line " + std::to_string(line) + " and " +
         c.kind + " in line " + std::to_string(c.line));
  }
  c.in[cur->id % 32] = v;
  const int round = c.round;
  if (++c.n == 32) {
    memcpy(c.out, c.in, sizeof c.in);
    c.n = 0;
    ++c.round;
  } else {
    wait_for([&c, round] { return c.round != round; }, kind, line);
  }
  return c.out;
}
template <class T>
T shfl(T x, int from, int line) {
  const uint64_t* all = collective("shfl", line, bits<uint64_t>(x));
  return from >= 0 ? bits<T>(all[from]) : x;
}
inline uint32_t ballot(bool p, int line) {
  const uint64_t* all = collective("vote", line, p);
  uint32_t r = 0;
  for (int i = 0; i < 32; ++i) r |= uint32_t(all[i] != 0) << i;
  return r;
}
#define __shfl_xor_sync(mask, x, o) shfl(x, cur->id % 32 ^ (o), __LINE__)
#define __shfl_up_sync(mask, x, o) shfl(x, cur->id % 32 - int(o), __LINE__)
#define __ballot_sync(mask, p) ballot(p, __LINE__)
#define __all_sync(mask, p) (ballot(p, __LINE__) == ~0u)
#define __any_sync(mask, p) (ballot(p, __LINE__) != 0u)
#define __syncwarp() collective("syncwarp", __LINE__, 0)
inline float redux_max(float x, int line) {
  const uint64_t* all = collective("redux", line, bits<uint64_t>(x));
  float m = -INFINITY;
  for (int i = 0; i < 32; ++i) m = fmaxf(m, bits<float>(all[i]));
  return m;
}
inline int __popc(uint32_t x) { return __builtin_popcount(x); }
inline int __clz(int x) { return x ? __builtin_clz(x) : 32; }

// ------------------------------------------------------------------ barriers of the CTA
struct Barrier {
  int n = 0, round = 0, count = 0;
  bool any = false, result = false;
  std::string kind;
};
inline Barrier barriers[16];
inline bool barrier(int id, int count, const char* kind, bool x, int line) {
  collective("barrier", line, 0);  // a warp comes as one
  Barrier& b = barriers[id];
  if (b.n == 0) {
    b.count = count;
    b.kind = kind;
    b.any = false;
  } else if (b.count != count || b.kind != kind) {
    fail("barrier " + std::to_string(id) + " used in two ways at once");
  }
  b.any |= x;
  const int round = b.round;
  if (++b.n == count) {
    b.result = b.any;
    b.n = 0;
    ++b.round;
  } else {
    wait_for([&b, round] { return b.round != round; }, kind, line);
  }
  return b.result;
}
#define __syncthreads() barrier(0, blockDim.x, "sync", false, __LINE__)

// ------------------------------------------------------------------ arithmetic
inline float2 __fmul2_rn(float2 a, float2 b) { return {a.x * b.x, a.y * b.y}; }
inline float2 __fadd2_rn(float2 a, float2 b) { return {a.x + b.x, a.y + b.y}; }
inline float2 __ffma2_rn(float2 a, float2 b, float2 c) {
  return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)};
}
inline float __fdividef(float a, float b) { return a / b; }
inline uint32_t __vmaxu2(uint32_t a, uint32_t b) {
  return max(a & 0xffffu, b & 0xffffu) | max(a >> 16, b >> 16) << 16;
}
inline uint32_t __byte_perm(uint32_t a, uint32_t, uint32_t) { return a; }
inline int atomicOr(int32_t* p, int v) { return std::exchange(*p, *p | v); }

// ------------------------------------------------------------------ shared memory
inline uint8_t* shared;
inline size_t shared_bytes;

namespace sv {
constexpr uint32_t kWaitLimit = 1u << 22, kSuspendNs = 20000;
inline uint64_t kWaitNs;
inline uint64_t global_ns() { return now_ns; }
inline uint32_t smem_u32(const void* p) {
  return uint32_t(static_cast<const uint8_t*>(p) - shared);
}

struct MBarrier {
  uint32_t count;
  int64_t pending, bytes;
  uint64_t phase;
  void settle() {
    if (pending == 0 && bytes == 0) {
      ++phase;
      pending = count;
    }
  }
};
inline std::map<uint64_t*, MBarrier> mbarriers;
inline MBarrier& mbarrier(uint64_t* b) {
  auto it = mbarriers.find(b);
  if (it == mbarriers.end()) fail("an mbarrier that is not initialised");
  return it->second;
}
inline void mbar_init(uint64_t* b, uint32_t n) { mbarriers[b] = {n, n, 0, 0}; }
inline void fence_mbar_init() {}
inline void arrive(uint64_t* b, int64_t bytes) {
  MBarrier& m = mbarrier(b);
  if (m.pending == 0) fail("an arrival too many");
  m.bytes += bytes;
  --m.pending;
  m.settle();
}
inline void mbar_arrive(uint64_t* b) { arrive(b, 0); }
inline void mbar_arrive_expect_tx(uint64_t* b, uint32_t bytes) { arrive(b, bytes); }
inline bool mbar_done(uint64_t* b, uint32_t parity) { return (mbarrier(b).phase & 1) != parity; }
inline bool mbar_try_wait(uint64_t* b, uint32_t parity, uint32_t ns) {
  const uint64_t until = now_ns + rng() % ns;
  wait_for([=] { return mbar_done(b, parity) || now_ns >= until; }, "try_wait", 0);
  return mbar_done(b, parity);
}
inline bool mbar_wait(uint64_t* b, uint32_t parity) {
  const uint64_t until = now_ns + 2000000;
  while (!mbar_try_wait(b, parity, kSuspendNs))
    if (now_ns > until) fail("what is in flight does not end");
  return true;
}
inline void pdl_wait() {}
inline void pdl_trigger() {}
inline float ex2_approx(float x) { return exp2f(x); }

// ------------------------------------------------------------------ TMEM and products
inline bool tmem_live;
inline uint32_t tmem_base, tmem_cols;
inline int products, copies;  // in flight
inline uint64_t last_product;
struct Columns {
  uint32_t from, to;
  uint64_t until;
};
inline std::vector<Columns> written;
inline std::function<float()> score;
inline void tmem_access(uint32_t addr, uint32_t n) {
  const uint32_t col = (addr & 0xffffu) - tmem_base, lane = addr >> 16;
  if (!tmem_live || col + n > tmem_cols) fail("TMEM outside of the allocation");
  if (lane % 32 || lane / 32 != uint32_t(cur->id / 32 % 4)) fail("TMEM lanes of another warp");
  for (const Columns& c : written)
    if (!stalling && c.until > now_ns && col < c.to && col + n > c.from)
      fail("TMEM columns that a product in flight writes");
}
inline void tmem_alloc(uint32_t* to, uint32_t cols) {
  collective("alloc", 0, 0);
  tmem_live = true;
  tmem_cols = cols;
  *to = tmem_base;
}
inline void tmem_relinquish() {}
inline void tmem_dealloc(uint32_t addr, uint32_t cols) {
  collective("dealloc", 0, 0);
  if (cur->id % 32) return;
  if (!tmem_live || addr != tmem_base || cols != tmem_cols) fail("TMEM freed that is not held");
  if (products) fail("TMEM freed with products in flight");
  tmem_live = false;
}
inline void tmem_load(uint32_t addr, float* f, int line) {
  collective("tmem_ld", line, 0);
  tmem_access(addr, 8);
  for (int i = 0; i < 8; ++i) f[i] = score();
}
inline void tmem_store(uint32_t addr, const float*, int line) {
  collective("tmem_st", line, 0);
  tmem_access(addr, 8);
}
#define tmem_ld8(addr, f) tmem_load(addr, f, __LINE__)
#define tmem_st8(addr, f) tmem_store(addr, f, __LINE__)
inline void tmem_wait_ld() { collective("wait_ld", 0, 0); }
inline void tmem_wait_st() { collective("wait_st", 0, 0); }
inline void tc_fence_before() {}
inline void tc_fence_after() {}
inline void fence_async_smem() {}
inline uint64_t tc_desc(uint32_t addr, uint32_t, uint32_t, uint32_t) { return addr >> 4; }
constexpr uint32_t tc_idesc(int, int, int, int, int, int n) { return n; }
inline void tc_mma_f8(uint32_t d, uint64_t, uint64_t, uint32_t n, bool) {
  const uint32_t col = (d & 0xffffu) - tmem_base;
  if (!tmem_live || col + n > tmem_cols) fail("a product outside of the TMEM allocation");
  ++products;
  last_product = max(last_product, after(300));
  if (written.size() > 64) written.erase(written.begin(), written.begin() + 32);
  written.push_back({col, col + n, last_product});
  events.push_back({last_product, [] { --products; }});
}
inline void tc_commit(uint64_t* b) {
  last_product = max(last_product + 1, now_ns + 1);
  events.push_back({last_product, [b] { arrive(b, 0); }});
}

// ------------------------------------------------------------------ copies
inline uint32_t box_bytes;
inline void tma_tile_3d(void* dst, const void*, int, int, int, uint64_t* b) {
  uint8_t* p = static_cast<uint8_t*>(dst);
  if (p < shared || p + box_bytes > shared + shared_bytes) fail("a copy outside of shared memory");
  ++copies;
  events.push_back({after(3000), [b] {
                      MBarrier& m = mbarrier(b);
                      --copies;
                      if ((m.bytes -= box_bytes) < 0) fail("more bytes than a phase expects");
                      m.settle();
                    }});
}
inline void tma_prefetch_map(const void*) {}
inline void cp_async4(void* dst, const void* src) { memcpy(dst, src, 4); }
inline void cp_async16(void* dst, const void* src, bool ok) {
  if (ok) memcpy(dst, src, 16);
  else memset(dst, 0, 16);
}
inline int async_loads[1024];  // of a thread, in flight
inline void cp_async_wait_all() {
  wait_for([me = cur->id] { return async_loads[me] == 0; }, "cp.async.wait_all", 0);
}
inline void cp_async_arrive(uint64_t* b) {
  ++async_loads[cur->id];
  events.push_back({after(2000), [b, me = cur->id] {
                      --async_loads[me];
                      arrive(b, 0);
                    }});
}
inline float q8_pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
inline uint32_t f16x2_to_e4m3(uint32_t v) { return v >> 8 & 0xffff; }
inline uint32_t e4m3x2_to_f16(uint32_t c) { return c << 8; }
}  // namespace sv
