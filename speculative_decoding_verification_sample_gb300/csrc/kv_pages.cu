// Blocks of a paged KV cache: reserving, forking and freeing.
//
// A row's logical position j lies in block block_table[b][j / bs] at offset
// j % bs; unused entries are -1; free ids lie on a stack. A block may be held
// by several rows: extra_refs[x] counts its holders beyond the first, so a
// block that was never shared reads 0 and the commit calls, which pop and push
// blocks of one holder, need no change. With L = seq_lens:
//   reserve  entries [ceil(L/bs), ceil((L+n)/bs)) that are -1 take
//            free_stack[top-1-r], r the entry's rank in row-major order;
//   fork     entries [0, L/bs) are shared (extra_refs + 1 each); a partly
//            filled tail block is copied (its L % bs tokens and its scales)
//            into a block of the child's own, popped in the order of the pairs;
//   free     every entry of a listed row loses one holder; a block without any
//            goes onto the stack, in the order in which it is first listed.
//
// Each call moves a few kilobytes of tables, so it is bound by the latency of
// dependent global accesses and by launches, not by bandwidth. The entries of all
// rows form one flat list (a prefix sum over the rows' spans, a binary search back),
// so long and short rows balance; a thread holds 8 consecutive entries in registers
// through all phases, and lists of up to 8192 are planned by one CTA, longer ones by
// ONE cluster of 8 CTAs whose phases are separated by the hardware cluster barrier
// instead of launches (a cluster costs about 3 us more to launch). Each CTA owns a
// contiguous part of the list and the parts' counts go through distributed shared
// memory, which makes the order of pops and pushes a function of the inputs alone.
// All-or-nothing: nothing is written before every check has passed; what the
// checks themselves write (claims in seq_lens, counts in extra_refs) is undone.
//
// Measured, device time of a call: reserve 5.2 us for one block a row of 256 rows (8.8 us
// for 9 thousand blocks), fork 9.3 us for 4 rows and 27 us for 128 rows of 512-4096
// tokens (32 layers x 8 heads x 128), free 6.6 us for 5 rows and 21 us for 200 rows.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"

namespace sv {

namespace cg = cooperative_groups;

constexpr int kPgThreads = 1024;
constexpr int kPgCluster = 8;
constexpr int kPgHeld = 8;        // entries that a thread holds
constexpr int kPgMaxRows = 8192;  // rows (or pairs) of one call: the prefix sums lie in shared memory
constexpr int kPgRowsPerThread = kPgMaxRows / kPgThreads;
constexpr int kForkThreads = 256;
constexpr int kForkWords = 8;     // 16-byte words that a thread of a copy has in flight
constexpr int kForkMinPlanes = 8; // planes of a tail block that one CTA copies, at least

struct PgShared {
  int prefix[kPgMaxRows + 1];  // flat index of each row's first entry
  int warp[kPgThreads / 32];
  int cnt[4], err[4];          // this CTA's share of each exchange, read by the cluster
};

// The CTAs that plan together: C = 1 or kPgCluster.
template <int C>
struct PgTeam {
  __device__ __forceinline__ static int rank() {
    return C == 1 ? 0 : int(cg::this_cluster().block_rank());
  }
  __device__ __forceinline__ static void sync() {
    if (C == 1) __syncthreads();
    else cg::this_cluster().sync();
  }
  // First and last step of a kernel: the exchanges' sums start at 0, and a CTA's shared
  // memory stays until nobody reads it any more.
  __device__ __forceinline__ static void enter(PgShared& sh) {
    if (threadIdx.x < 4) sh.cnt[threadIdx.x] = sh.err[threadIdx.x] = 0;
    __syncthreads();
  }
  __device__ __forceinline__ static void leave() {
    if (C != 1) cg::this_cluster().sync();
  }
};

// Block-wide exclusive scan (kPgThreads threads); `total` is the block's sum.
__device__ int pg_scan(int v, int* warp, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // the previous call's readers
  if (lane == 31) warp[w] = inc;
  __syncthreads();
  int x = warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  const int before = __shfl_sync(0xffffffffu, x, w > 0 ? w - 1 : 0);
  return (w > 0 ? before : 0) + inc - v;
}

// Over the team: sum of the counts, union of the errors, sum over lower ranks. Each
// exchange of a kernel has a place of its own, so one barrier is enough.
struct PgAll {
  int cnt, err, before;
};
template <int C>
__device__ PgAll pg_exchange(PgShared& sh, int place, int cnt, int err) {
  const int c = __reduce_add_sync(0xffffffffu, cnt);
  const int e = __reduce_or_sync(0xffffffffu, err);
  if ((threadIdx.x & 31) == 0) {
    if (c) atomicAdd(&sh.cnt[place], c);
    if (e) atomicOr(&sh.err[place], e);
  }
  PgTeam<C>::sync();
  if (C == 1) return PgAll{sh.cnt[place], sh.err[place], 0};
  cg::cluster_group cl = cg::this_cluster();
  PgAll r{0, 0, 0};
  const int me = cl.block_rank();
  int cs[C];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const PgShared* o = cl.map_shared_rank(&sh, k);
    cs[k] = o->cnt[place];
    r.err |= o->err[place];
  }
#pragma unroll
  for (int k = 0; k < C; ++k) {
    r.cnt += cs[k];
    if (k < me) r.before += cs[k];
  }
  return r;
}

// A CTA's part [e0, e1) of a flat list, in rounds; a thread has `held` consecutive
// entries of a round, kPgHeld at most.
template <int C>
struct PgPart {
  int e0, e1, held, rounds;
  __device__ PgPart(int total) {
    const int r = PgTeam<C>::rank();
    e0 = int(int64_t(total) * r / C);
    e1 = int(int64_t(total) * (r + 1) / C);
    // the same for every CTA of the team: all of them run all rounds
    const int most = (total + C - 1) / C;
    held = min(kPgHeld, max(1, (most + kPgThreads - 1) / kPgThreads));
    rounds = (most + kPgThreads * held - 1) / (kPgThreads * held);
  }
  __device__ __forceinline__ int at(int round, int k) const {
    const int e = e0 + (round * kPgThreads + int(threadIdx.x)) * held + k;
    return k < held && e < e1 ? e : -1;
  }
};

// prefix[] of n spans given by span(i); each thread takes consecutive rows.
template <class F>
__device__ int pg_prefix(PgShared& sh, int n, F span) {
  const int per = (n + kPgThreads - 1) / kPgThreads;
  const int i0 = threadIdx.x * per;
  int v[kPgRowsPerThread], sum = 0;
#pragma unroll
  for (int k = 0; k < kPgRowsPerThread; ++k) {
    v[k] = k < per && i0 + k < n ? span(i0 + k) : 0;
    sum += v[k];
  }
  int total;
  int at = pg_scan(sum, sh.warp, total);
#pragma unroll
  for (int k = 0; k < kPgRowsPerThread; ++k) {
    if (k < per && i0 + k < n) sh.prefix[i0 + k] = at;
    at += v[k];
  }
  if (threadIdx.x == 0) sh.prefix[n] = total;
  __syncthreads();
  return total;
}

// The row that holds flat entry e: the last i with prefix[i] <= e.
__device__ int pg_row(const PgShared& sh, int n, int e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (sh.prefix[m] <= e) lo = m;
    else hi = m - 1;
  }
  return lo;
}

__device__ __forceinline__ int pg_cdiv(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------ reserve
struct ReserveArgs {
  int32_t* bt;
  const int32_t* sl;
  const int32_t* nn;  // null: n for every row
  int n, NB, bs, B, MB;
  const int32_t* fs;
  int32_t* ftop;
  int32_t* status;
};

template <int C>
__device__ __forceinline__ void reserve_body(const ReserveArgs& a, PgShared& sh) {
  const int tid = threadIdx.x, rank = PgTeam<C>::rank();
  PgTeam<C>::enter(sh);
  pdl_trigger();
  pdl_wait();
  const int top = *a.ftop;
  int err = 0;
  const int total = pg_prefix(sh, a.B, [&](int b) {
    const int L = a.sl[b], n = a.nn ? a.nn[b] : a.n;
    if (L < 0 || n < 0 || int64_t(L) + n > int64_t(a.MB) * a.bs) {
      err |= SPEC_DERR_BAD_LENGTH;
      return 0;
    }
    return pg_cdiv(L + n, a.bs) - pg_cdiv(L, a.bs);
  });
  const PgPart<C> part(total);
  int32_t* slot[kPgHeld];
  int x[kPgHeld];
  auto load = [&](int round) {  // entries of this thread, 0 where there is none
    int b = part.at(round, 0) >= 0 ? pg_row(sh, a.B, part.at(round, 0)) : 0;
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) {
      const int e = part.at(round, k);
      slot[k] = nullptr;
      x[k] = 0;
      if (e >= 0) {
        while (sh.prefix[b + 1] <= e) ++b;
        slot[k] = a.bt + int64_t(b) * a.MB + pg_cdiv(a.sl[b], a.bs) + (e - sh.prefix[b]);
        x[k] = *slot[k];
      }
    }
  };
  int cnt = 0;
  for (int r = 0; r < part.rounds; ++r) {
    load(r);
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) {
      cnt += x[k] == -1;
      if (x[k] < -1 || x[k] >= a.NB) err |= SPEC_DERR_BAD_BLOCK;
    }
  }
  PgAll all = pg_exchange<C>(sh, 0, cnt, err);
  const int need = all.cnt, base = all.before;
  err = all.err;
  if (err == 0 && (top < 0 || top > a.NB || need > top)) err = SPEC_DERR_NO_SPACE;
  if (err == 0) {
    int pe = 0;
    for (int i = rank * kPgThreads + tid; i < need; i += C * kPgThreads) {
      const int y = a.fs[top - 1 - i];
      if (y < 0 || y >= a.NB) pe = SPEC_DERR_BAD_BLOCK;
    }
    err = pg_exchange<C>(sh, 1, 0, pe).err;
  }
  PgTeam<C>::leave();
  if (err != 0) {
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  int carry = base;
  for (int r = 0; r < part.rounds; ++r) {
    if (part.rounds > 1) load(r);
    int mine = 0, sum;
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) mine += x[k] == -1;
    int at = carry + pg_scan(mine, sh.warp, sum);
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k)
      if (x[k] == -1) *slot[k] = a.fs[top - 1 - at++];
    carry += sum;
  }
  if (rank == 0 && tid == 0) {
    *a.ftop = top - need;
    *a.status = 0;
  }
}

__global__ void __launch_bounds__(kPgThreads) kv_reserve_kernel(const ReserveArgs a) {
  __shared__ PgShared sh;
  reserve_body<1>(a, sh);
}
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_reserve_cluster_kernel(const ReserveArgs a) {
  __shared__ PgShared sh;
  reserve_body<kPgCluster>(a, sh);
}

// One CTA where it can hold `entries` (an upper bound), else a cluster.
template <class Kern, class Args>
int launch_plan(Kern one, Kern cluster, int64_t entries, const Args& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return entries <= kPgThreads * kPgHeld
             ? launch_pdl(one, dim3(1), dim3(kPgThreads), 0, st, a)
             : launch_pdl(cluster, dim3(kPgCluster), dim3(kPgThreads), 0, st, a);
}

int launch_kv_reserve(const KvReserveLaunch& k) {
  ReserveArgs a{k.block_table, k.seq_lens, k.num_new, k.n, k.num_blocks, k.block_size, k.B,
                k.max_blocks, k.free_stack, k.free_top, k.status};
  const int64_t row = k.num_new ? k.max_blocks : k.n / k.block_size + 1;
  return launch_plan(kv_reserve_kernel, kv_reserve_cluster_kernel, k.B * row, a, k.stream);
}

// ------------------------------------------------------------------ fork
struct ForkArgs {
  int32_t* bt;
  int32_t* sl;
  int32_t* refs;
  const int32_t* src;
  const int32_t* dst;
  uint8_t* pool;
  float* scales;  // null: the pool has none
  int NB, bs, B, MB, n, planes, tb;
  int chunk;      // planes that a CTA of the copy takes
  int32_t* fs;
  int32_t* ftop;
  int32_t* status;
};

template <int C>
__device__ __forceinline__ void fork_plan_body(const ForkArgs& a, PgShared& sh) {
  const int tid = threadIdx.x, rank = PgTeam<C>::rank();
  PgTeam<C>::enter(sh);
  pdl_wait();
  // From here on the copies may start: they read the parents' tables and blocks,
  // which this kernel does not change, and wait for it before they write.
  pdl_trigger();
  const int top = *a.ftop;
  int err = 0, mine = 0;  // mine: pairs of this thread with a partly filled tail block
  const int total = pg_prefix(sh, a.n, [&](int i) {
    const int s = a.src[i], d = a.dst[i];
    if (s < 0 || s >= a.B || d < 0 || d >= a.B) {
      err |= SPEC_DERR_BAD_SLOT;
      return 0;
    }
    const int L = a.sl[s];
    if (L < 0 || L > int64_t(a.MB) * a.bs || a.sl[d] != 0) {
      err |= SPEC_DERR_BAD_LENGTH;
      return 0;
    }
    mine += L % a.bs != 0;
    return pg_cdiv(L, a.bs);
  });
  const PgPart<C> part(total);
  int32_t* to[kPgHeld];  // the child's entry, null for the tail block
  int x[kPgHeld];
  int bad = 0;
  auto load = [&](int round) {
    int i = part.at(round, 0) >= 0 ? pg_row(sh, a.n, part.at(round, 0)) : 0;
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) {
      const int e = part.at(round, k);
      to[k] = nullptr;
      if (e >= 0) {
        while (sh.prefix[i + 1] <= e) ++i;
        const int j = e - sh.prefix[i], s = a.src[i];
        x[k] = a.bt[int64_t(s) * a.MB + j];
        to[k] = a.bt + int64_t(a.dst[i]) * a.MB + j;
        if (x[k] < 0 || x[k] >= a.NB || *to[k] != -1) bad = SPEC_DERR_BAD_BLOCK;
        if ((j + 1) * int64_t(a.bs) > __ldcg(&a.sl[s])) to[k] = nullptr;
      }
    }
  };
  for (int r = 0; r < part.rounds; ++r) load(r);
  err = pg_exchange<C>(sh, 0, 0, err | bad).err;
  // tails are ranked in the order of the pairs (the prefix gave a thread the same ones)
  const int per = (a.n + kPgThreads - 1) / kPgThreads, i0 = tid * per;
  int tails;
  const int at = pg_scan(mine, sh.warp, tails);
  if (err == 0 && (top < 0 || top > a.NB || tails > top)) err = SPEC_DERR_NO_SPACE;
  // Children must be distinct and no child may be a parent: rank 0 claims each
  // child by an exchange on its length, which is 0 until then; a claim that
  // finds another one, or a parent that turns out to be claimed, is an error.
  if (err == 0) {
    int pe = 0;
    if (rank == 0) {
      for (int k = tid; k < tails; k += kPgThreads) {
        const int y = a.fs[top - 1 - k];
        if (y < 0 || y >= a.NB) pe |= SPEC_DERR_BAD_BLOCK;
      }
      for (int i = i0; i < i0 + per && i < a.n; ++i)
        if (atomicExch(&a.sl[a.dst[i]], -1) != 0) pe |= SPEC_DERR_BAD_SLOT;
      __syncthreads();
      for (int i = i0; i < i0 + per && i < a.n; ++i)
        if (__ldcg(&a.sl[a.src[i]]) < 0) pe |= SPEC_DERR_BAD_SLOT;
    }
    err = pg_exchange<C>(sh, 1, 0, pe).err;
    if (err != 0 && rank == 0)
      for (int i = i0; i < i0 + per && i < a.n; ++i) a.sl[a.dst[i]] = 0;
  }
  PgTeam<C>::leave();
  if (err != 0) {
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  for (int r = 0; r < part.rounds; ++r) {
    if (part.rounds > 1) load(r);
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k)
      if (to[k]) {
        *to[k] = x[k];
        atomicAdd(&a.refs[x[k]], 1);
      }
  }
  if (rank == 0) {
    int r = at;
    for (int i = i0; i < i0 + per && i < a.n; ++i) {
      const int L = __ldcg(&a.sl[a.src[i]]);
      if (L % a.bs != 0) a.bt[int64_t(a.dst[i]) * a.MB + L / a.bs] = a.fs[top - 1 - r++];
    }
    if (tid == 0) {
      *a.ftop = top - tails;
      *a.status = 0;
    }
  }
}

__global__ void __launch_bounds__(kPgThreads) kv_fork_plan_kernel(const ForkArgs a) {
  __shared__ PgShared sh;
  fork_plan_body<1>(a, sh);
}
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_fork_plan_cluster_kernel(const ForkArgs a) {
  __shared__ PgShared sh;
  fork_plan_body<kPgCluster>(a, sh);
}

// The tail blocks' tokens and scales: CTA (chunk, pair) copies `chunk`
// planes: 8 when there are few pairs, more when that would be many waves of CTAs with
// the latency of their table reads each. 128 pairs of 512 planes of 16 x 128 bytes, 126 MB
// read and written: 8 planes a CTA with a division a word 24 us, as here 20.7 us alone
// (6.1 TB/s).
// Bound by memory: it reads and writes L % bs tokens of every plane. Its
// first loads do not wait for the plan, which changes neither the parents' rows nor
// any block; they test what the plan has not yet vouched for.
__global__ void __launch_bounds__(kForkThreads) kv_fork_copy_kernel(const ForkArgs a) {
  pdl_trigger();
  const int i = blockIdx.y, s = __ldcg(&a.src[i]), d = __ldcg(&a.dst[i]);
  const int L = s >= 0 && s < a.B ? __ldcg(&a.sl[s]) : 0;
  const int off = L > 0 && L <= int64_t(a.MB) * a.bs ? L % a.bs : 0;
  const int j = off ? L / a.bs : 0;
  const int64_t x = off ? __ldcg(&a.bt[int64_t(s) * a.MB + j]) : -1;
  const bool some = x >= 0 && x < a.NB;
  const int p0 = blockIdx.x * a.chunk;
  const int np = min(a.chunk, a.planes - p0);
  const int64_t plane = int64_t(a.bs) * a.tb;
  const int vec = off * (a.tb / 16);  // 16-byte words of a plane's tokens
  const uint8_t* from = a.pool + ((some ? x : 0) * a.planes + p0) * plane;
  uint8_t* to = a.pool;
  bool waited = false;
  int64_t y = 0;
  // until the plan is done and says that it has changed the tables
  auto plan_ok = [&]() {
    if (!waited) {
      waited = true;
      pdl_wait();
      if (__ldcg(a.status) != 0) return false;
      if (blockIdx.x == 0 && threadIdx.x == 0) a.sl[d] = L;
      if (some) y = __ldcg(&a.bt[int64_t(d) * a.MB + j]);
      to = a.pool + (y * a.planes + p0) * plane;
    }
    return true;
  };
  // a warp takes two planes at a time, four times 32 words of each
  const int lane = threadIdx.x & 31;
  constexpr int kWarps = kForkThreads / 32, kEach = kForkWords / 2;
  for (int p = threadIdx.x >> 5; some && p < np; p += 2 * kWarps) {
    const bool two = p + kWarps < np;
    for (int g0 = lane; g0 - lane < vec; g0 += 32 * kEach) {
      uint4 v[2][kEach];
      const int64_t o = p * plane + int64_t(g0) * 16;
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (g0 + 32 * k < vec) {
          v[0][k] = __ldcg(reinterpret_cast<const uint4*>(from + o + 512 * k));
          if (two) v[1][k] = __ldcg(reinterpret_cast<const uint4*>(from + o + kWarps * plane + 512 * k));
        }
      if (!plan_ok()) return;
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (g0 + 32 * k < vec) {
          *reinterpret_cast<uint4*>(to + o + 512 * k) = v[0][k];
          if (two) *reinterpret_cast<uint4*>(to + o + kWarps * plane + 512 * k) = v[1][k];
        }
    }
  }
  if (!plan_ok() || !some) return;
  if (a.scales)
    for (int p = threadIdx.x; p < np; p += kForkThreads)
      a.scales[y * a.planes + p0 + p] = a.scales[x * a.planes + p0 + p];
}

int launch_kv_fork(const KvForkLaunch& k) {
  ForkArgs a{k.block_table, k.seq_lens, k.extra_refs, k.src_rows, k.dst_rows,
             static_cast<uint8_t*>(k.kv_pool), k.kv_scales, k.num_blocks, k.block_size, k.B,
             k.max_blocks, k.n, k.planes, k.token_bytes, 0, k.free_stack, k.free_top, k.status};
  // about two waves of 8 CTAs an SM, 152 of them
  const int64_t share = int64_t(k.n) * k.planes / 2432;
  a.chunk = int(share < kForkMinPlanes ? kForkMinPlanes : share < k.planes ? share : k.planes);
  const int st = launch_plan(kv_fork_plan_kernel, kv_fork_plan_cluster_kernel,
                             int64_t(k.n) * k.max_blocks, a, k.stream);
  if (st != SPEC_OK) return st;
  const int chunks = (k.planes + a.chunk - 1) / a.chunk;
  return launch_pdl(kv_fork_copy_kernel, dim3(chunks, k.n), dim3(kForkThreads), 0,
                    static_cast<cudaStream_t>(k.stream), a);
}

// ------------------------------------------------------------------ free
struct FreeArgs {
  int32_t* bt;
  int32_t* sl;
  int32_t* refs;
  const int32_t* rows;
  int NB, B, MB, n;
  int32_t* fs;
  int32_t* ftop;
  int32_t* status;
};

// Phases over the flat list of the listed rows' entries (E = n * MB of them, at
// most 2^30):
//   1 one holder less for every entry: a block without any reads -1, one that
//     is listed more often than it is held reads less (an error);
//   2 a block at -1 takes the lowest flat index e that lists it, as INT_MIN + e,
//     far below any count;
//   3 the entry whose index its block holds pushes it, ranked by a scan;
//   4 that entry sets the count to 0; all entries are cleared.
template <int C>
__device__ __forceinline__ void free_body(const FreeArgs& a, PgShared& sh) {
  const int tid = threadIdx.x, rank = PgTeam<C>::rank(), step = C * kPgThreads;
  constexpr int kTaken = -(1 << 30);  // counts lie above, taken blocks below or at it
  PgTeam<C>::enter(sh);
  pdl_trigger();
  pdl_wait();
  const int top = *a.ftop;
  const int E = a.n * a.MB;
  const PgPart<C> part(E);
  int err = 0;
  // calls f(row, k) for this thread's rows that are in range, the k-th of them
  auto each_row = [&](auto f) {
    for (int i = rank * kPgThreads + tid, k = 0; i < a.n; i += step, ++k) {
      const int r = a.rows[i];
      if (r >= 0 && r < a.B) f(r, k);
      else err |= SPEC_DERR_BAD_SLOT;
    }
  };
  each_row([&](int r, int) {
    if (a.sl[r] < 0) err |= SPEC_DERR_BAD_LENGTH;
  });
  int32_t* slot[kPgHeld];
  int x[kPgHeld];  // block ids, -1: none
  auto load = [&](int round) {
    const int e0 = max(0, part.at(round, 0));
    int i = e0 / a.MB, j = e0 - i * a.MB - 1;
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) {
      slot[k] = nullptr;
      x[k] = -1;
      if (part.at(round, k) >= 0) {
        if (++j == a.MB) {
          j = 0;
          ++i;
        }
        const int r = a.rows[i];
        if (r >= 0 && r < a.B) {
          slot[k] = a.bt + int64_t(r) * a.MB + j;
          x[k] = *slot[k];
        }
      }
    }
  };
  // calls f(entry's flat index, k) for every entry that holds a block
  auto each = [&](auto f) {
    for (int r = 0; r < part.rounds; ++r) {
      if (part.rounds > 1) load(r);
#pragma unroll
      for (int k = 0; k < kPgHeld; ++k)
        if (x[k] >= 0) f(part.at(r, k), k);
    }
  };
  int bad = 0;
  for (int r = 0; r < part.rounds; ++r) {
    load(r);
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k)
      if (x[k] < -1 || x[k] >= a.NB) bad |= SPEC_DERR_BAD_BLOCK;
  }
  if (top < 0 || top > a.NB) bad |= SPEC_DERR_BAD_BLOCK;
  PgTeam<C>::sync();  // every length has been read
  // rows must be distinct: each is claimed by complementing its length
  uint32_t claimed = 0;
  each_row([&](int r, int k) {
    const int L = __ldcg(&a.sl[r]);
    if (L < 0 || atomicCAS(&a.sl[r], L, ~L) != L) bad |= SPEC_DERR_BAD_SLOT;
    else claimed |= 1u << k;
  });
  auto unclaim = [&]() {  // only reached with every CTA past its claims
    each_row([&](int r, int k) {
      if (claimed >> k & 1u) a.sl[r] = ~__ldcg(&a.sl[r]);
    });
  };
  // rows out of range and lengths come before the rest
  err = pg_exchange<C>(sh, 0, 0, err << 16 | bad).err;
  if (err != 0) {
    PgTeam<C>::leave();
    unclaim();
    if (rank == 0 && tid == 0) *a.status = err >> 16 ? err >> 16 : err;
    return;
  }
  each([&](int, int k) { atomicSub(&a.refs[x[k]], 1); });
  PgTeam<C>::sync();
  each([&](int e, int k) {
    const int r = __ldcg(&a.refs[x[k]]);
    if (r < -1 && r > kTaken) err |= SPEC_DERR_BAD_BLOCK;
    else if (r <= -1) atomicMin(&a.refs[x[k]], INT_MIN + e);
  });
  PgTeam<C>::sync();
  int cnt = 0;
  uint32_t push = 0;  // this thread's entries that push, of the last round
  auto find_pushes = [&](int r) {
    push = 0;
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k)
      if (x[k] >= 0 && __ldcg(&a.refs[x[k]]) == INT_MIN + part.at(r, k)) push |= 1u << k;
  };
  for (int r = 0; r < part.rounds; ++r) {
    if (part.rounds > 1) load(r);
    find_pushes(r);
    cnt += __popc(push);
  }
  PgAll all = pg_exchange<C>(sh, 1, cnt, err);
  err = all.err;
  if (all.cnt > a.NB - top) err |= SPEC_DERR_BAD_BLOCK;  // some id would be held twice
  if (err != 0) {
    each([&](int, int k) {
      if (__ldcg(&a.refs[x[k]]) <= kTaken) a.refs[x[k]] = -1;
    });
    PgTeam<C>::sync();
    each([&](int, int k) { atomicAdd(&a.refs[x[k]], 1); });
    unclaim();
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  int carry = top + all.before;
  for (int r = 0; r < part.rounds; ++r) {
    if (part.rounds > 1) {
      load(r);
      find_pushes(r);
    }
    int sum;
    int at = carry + pg_scan(__popc(push), sh.warp, sum);
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k)
      if (push >> k & 1u) a.fs[at++] = x[k];
    carry += sum;
  }
  PgTeam<C>::sync();  // every entry has been compared before a count changes
  for (int r = 0; r < part.rounds; ++r) {
    if (part.rounds > 1) {
      load(r);
      find_pushes(r);  // a block is its pusher's until that entry comes
    }
#pragma unroll
    for (int k = 0; k < kPgHeld; ++k) {
      if (push >> k & 1u) a.refs[x[k]] = 0;
      if (slot[k]) *slot[k] = -1;
    }
  }
  each_row([&](int r, int) { a.sl[r] = 0; });
  if (rank == 0 && tid == 0) {
    *a.ftop = top + all.cnt;
    *a.status = 0;
  }
}

__global__ void __launch_bounds__(kPgThreads) kv_free_kernel(const FreeArgs a) {
  __shared__ PgShared sh;
  free_body<1>(a, sh);
}
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_free_cluster_kernel(const FreeArgs a) {
  __shared__ PgShared sh;
  free_body<kPgCluster>(a, sh);
}

int launch_kv_free(const KvFreeLaunch& k) {
  FreeArgs a{k.block_table, k.seq_lens, k.extra_refs, k.rows, k.num_blocks, k.B, k.max_blocks,
             k.n, k.free_stack, k.free_top, k.status};
  return launch_plan(kv_free_kernel, kv_free_cluster_kernel, int64_t(k.n) * k.max_blocks, a,
                     k.stream);
}

}  // namespace sv
