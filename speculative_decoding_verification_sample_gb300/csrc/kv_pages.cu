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
// dependent global accesses, not by bandwidth: the planning runs as ONE cluster
// of 8 CTAs x 1024 threads whose phases are separated by the hardware cluster
// barrier (well under a microsecond) instead of launches. The entries of all
// rows form one flat list (a prefix sum over the rows' spans, a binary search
// back), so long and short rows balance; each CTA owns a contiguous part of
// it and the parts' counts go through distributed shared memory, which makes
// the order of pops and pushes a function of the inputs alone.
// All-or-nothing: nothing is written before every check has passed; what the
// checks themselves write (claims in seq_lens, counts in extra_refs) is undone.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "launch_util.cuh"
#include "ptx.cuh"

namespace sv {

namespace cg = cooperative_groups;

constexpr int kPgThreads = 1024;
constexpr int kPgCluster = 8;
constexpr int kPgMaxRows = 8192;  // rows (or pairs) of one call: the prefix sums lie in shared memory
constexpr int kPgRowsPerThread = kPgMaxRows / kPgThreads;
constexpr int kForkThreads = 256;
constexpr int kForkPlanes = 8;  // planes of a tail block that one CTA copies

struct PgShared {
  int prefix[kPgMaxRows + 1];  // flat index of each row's first entry
  int warp[kPgThreads / 32];
  int cnt, err;                // this CTA's share, read by the cluster
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

// Block-wide sum of counts and union of bits into sh.cnt, sh.err.
__device__ void pg_publish(PgShared& sh, int cnt, int err) {
  __syncthreads();
  if (threadIdx.x == 0) sh.cnt = sh.err = 0;
  __syncthreads();
  const int c = __reduce_add_sync(0xffffffffu, cnt);
  const int e = __reduce_or_sync(0xffffffffu, err);
  if ((threadIdx.x & 31) == 0) {
    if (c) atomicAdd(&sh.cnt, c);
    if (e) atomicOr(&sh.err, e);
  }
  __syncthreads();
}

// Cluster-wide: sum of the counts, union of the errors, sum over lower ranks.
struct PgAll {
  int cnt, err, before;
};
__device__ PgAll pg_exchange(cg::cluster_group& cl, PgShared& sh, int cnt, int err) {
  pg_publish(sh, cnt, err);
  cl.sync();
  PgAll r{0, 0, 0};
  const int me = cl.block_rank();
#pragma unroll
  for (int k = 0; k < kPgCluster; ++k) {
    const PgShared* o = cl.map_shared_rank(&sh, k);
    const int c = o->cnt;
    r.cnt += c;
    r.err |= o->err;
    if (k < me) r.before += c;
  }
  cl.sync();  // the values may be replaced, or the CTA may leave
  return r;
}

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

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_reserve_kernel(const ReserveArgs a) {
  __shared__ PgShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, rank = cl.block_rank();
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
  const int e0 = int(int64_t(total) * rank / kPgCluster);
  const int e1 = int(int64_t(total) * (rank + 1) / kPgCluster);
  auto slot = [&](int e) -> int32_t* {
    const int b = pg_row(sh, a.B, e);
    return a.bt + int64_t(b) * a.MB + pg_cdiv(a.sl[b], a.bs) + (e - sh.prefix[b]);
  };
  int cnt = 0;
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *slot(e);
    cnt += x == -1;
    if (x < -1 || x >= a.NB) err |= SPEC_DERR_BAD_BLOCK;
  }
  PgAll all = pg_exchange(cl, sh, cnt, err);
  const int need = all.cnt, base = all.before;
  err = all.err;
  if (err == 0 && (top < 0 || top > a.NB || need > top)) err = SPEC_DERR_NO_SPACE;
  if (err == 0) {
    int pe = 0;
    for (int i = rank * kPgThreads + tid; i < need; i += kPgCluster * kPgThreads) {
      const int x = a.fs[top - 1 - i];
      if (x < 0 || x >= a.NB) pe = SPEC_DERR_BAD_BLOCK;
    }
    err = pg_exchange(cl, sh, 0, pe).err;
  }
  if (err != 0) {
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  int carry = base;
  for (int f = e0; f < e1; f += kPgThreads) {  // uniform over the CTA: the scan synchronises
    const int e = f + tid;
    int32_t* p = e < e1 ? slot(e) : nullptr;
    const bool want = p && *p == -1;
    int sum;
    const int r = carry + pg_scan(want, sh.warp, sum);
    if (want) *p = a.fs[top - 1 - r];
    carry += sum;
  }
  if (rank == 0 && tid == 0) {
    *a.ftop = top - need;
    *a.status = 0;
  }
}

int launch_kv_reserve(const KvReserveLaunch& k) {
  ReserveArgs a{k.block_table, k.seq_lens, k.num_new, k.n, k.num_blocks, k.block_size, k.B,
                k.max_blocks, k.free_stack, k.free_top, k.status};
  return launch_pdl(kv_reserve_kernel, dim3(kPgCluster), dim3(kPgThreads), 0,
                    static_cast<cudaStream_t>(k.stream), a);
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
  int32_t* fs;
  int32_t* ftop;
  int32_t* status;
};

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_fork_plan_kernel(const ForkArgs a) {
  __shared__ PgShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, rank = cl.block_rank();
  pdl_trigger();
  pdl_wait();
  const int top = *a.ftop;
  int err = 0;
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
    return pg_cdiv(L, a.bs);
  });
  const int e0 = int(int64_t(total) * rank / kPgCluster);
  const int e1 = int(int64_t(total) * (rank + 1) / kPgCluster);
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int i = pg_row(sh, a.n, e), j = e - sh.prefix[i];
    const int x = a.bt[int64_t(a.src[i]) * a.MB + j];
    if (x < 0 || x >= a.NB || a.bt[int64_t(a.dst[i]) * a.MB + j] != -1) err |= SPEC_DERR_BAD_BLOCK;
  }
  // tails: pairs with a partly filled block, ranked in the order of the pairs
  const int per = (a.n + kPgThreads - 1) / kPgThreads, i0 = tid * per;
  int mine = 0;
  PgAll all = pg_exchange(cl, sh, 0, err);
  err = all.err;
  if (err == 0)
    for (int i = i0; i < i0 + per && i < a.n; ++i) mine += a.sl[a.src[i]] % a.bs != 0;
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
        const int x = a.fs[top - 1 - k];
        if (x < 0 || x >= a.NB) pe |= SPEC_DERR_BAD_BLOCK;
      }
      for (int i = i0; i < i0 + per && i < a.n; ++i)
        if (atomicExch(&a.sl[a.dst[i]], -1) != 0) pe |= SPEC_DERR_BAD_SLOT;
      __syncthreads();
      for (int i = i0; i < i0 + per && i < a.n; ++i)
        if (__ldcg(&a.sl[a.src[i]]) < 0) pe |= SPEC_DERR_BAD_SLOT;
    }
    err = pg_exchange(cl, sh, 0, pe).err;
    if (err != 0 && rank == 0)
      for (int i = i0; i < i0 + per && i < a.n; ++i) a.sl[a.dst[i]] = 0;
  }
  if (err != 0) {
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int i = pg_row(sh, a.n, e), j = e - sh.prefix[i], s = a.src[i];
    if ((j + 1) * int64_t(a.bs) > __ldcg(&a.sl[s])) continue;  // the tail block
    const int x = a.bt[int64_t(s) * a.MB + j];
    a.bt[int64_t(a.dst[i]) * a.MB + j] = x;
    atomicAdd(&a.refs[x], 1);
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

// The tail blocks' tokens and scales: CTA (chunk, pair) copies kForkPlanes
// planes. Bound by memory: it reads and writes L % bs tokens of every plane.
__global__ void __launch_bounds__(kForkThreads) kv_fork_copy_kernel(const ForkArgs a) {
  pdl_trigger();
  pdl_wait();  // the plan
  if (*a.status != 0) return;
  const int i = blockIdx.y, s = a.src[i], d = a.dst[i];
  const int L = a.sl[s], off = L % a.bs;  // a parent's length does not change
  if (blockIdx.x == 0 && threadIdx.x == 0) a.sl[d] = L;
  if (off == 0) return;
  const int j = L / a.bs;
  const int64_t x = a.bt[int64_t(s) * a.MB + j], y = a.bt[int64_t(d) * a.MB + j];
  const int p0 = blockIdx.x * kForkPlanes;
  const int np = min(kForkPlanes, a.planes - p0);
  const int64_t plane = int64_t(a.bs) * a.tb;
  const uint8_t* from = a.pool + (x * a.planes + p0) * plane;
  uint8_t* to = a.pool + (y * a.planes + p0) * plane;
  const int vec = off * (a.tb / 16);  // 16-byte words of a plane's tokens
  const int total = np * vec;
  constexpr int kUnroll = 4;
  for (int g0 = threadIdx.x; g0 < total; g0 += kForkThreads * kUnroll) {
    uint4 v[kUnroll];
    int64_t o[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int g = g0 + k * kForkThreads;
      o[k] = -1;
      if (g < total) {
        const int p = g / vec;
        o[k] = p * plane + int64_t(g - p * vec) * 16;
        v[k] = ldg_nc_v4(from + o[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (o[k] >= 0) *reinterpret_cast<uint4*>(to + o[k]) = v[k];
  }
  if (a.scales && threadIdx.x < np)
    a.scales[y * a.planes + p0 + threadIdx.x] = a.scales[x * a.planes + p0 + threadIdx.x];
}

int launch_kv_fork(const KvForkLaunch& k) {
  ForkArgs a{k.block_table, k.seq_lens, k.extra_refs, k.src_rows, k.dst_rows,
             static_cast<uint8_t*>(k.kv_pool), k.kv_scales, k.num_blocks, k.block_size, k.B,
             k.max_blocks, k.n, k.planes, k.token_bytes, k.free_stack, k.free_top, k.status};
  cudaStream_t st = static_cast<cudaStream_t>(k.stream);
  if (launch_pdl(kv_fork_plan_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, st, a) != SPEC_OK)
    return SPEC_ECUDA;
  const int chunks = (k.planes + kForkPlanes - 1) / kForkPlanes;
  return launch_pdl(kv_fork_copy_kernel, dim3(chunks, k.n), dim3(kForkThreads), 0, st, a);
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

// Phases over the flat list of the listed rows' entries (E = n * MB of them):
//   1 one holder less for every entry: a block without any reads -1, one that
//     is listed more often than it is held reads less (an error);
//   2 a block at -1 takes the lowest flat index that lists it, as index - E - 1
//     (below -1, so never mistaken for a count);
//   3 the entry whose index its block holds pushes it, ranked by a scan;
//   4 that entry sets the count to 0; all entries are cleared.
__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
    kv_free_kernel(const FreeArgs a) {
  __shared__ PgShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, rank = cl.block_rank();
  pdl_trigger();
  pdl_wait();
  const int top = *a.ftop;
  const int E = a.n * a.MB;
  const int e0 = int(int64_t(E) * rank / kPgCluster), e1 = int(int64_t(E) * (rank + 1) / kPgCluster);
  const int step = kPgCluster * kPgThreads;
  int err = 0;
  for (int i = rank * kPgThreads + tid; i < a.n; i += step) {
    const int r = a.rows[i];
    if (r < 0 || r >= a.B) err |= SPEC_DERR_BAD_SLOT;
    else if (a.sl[r] < 0) err |= SPEC_DERR_BAD_LENGTH;
  }
  err = pg_exchange(cl, sh, 0, err).err;
  if (err != 0) {
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  // rows must be distinct: each is claimed by complementing its length
  auto entry = [&](int e) -> int32_t* { return a.bt + int64_t(a.rows[e / a.MB]) * a.MB + e % a.MB; };
  for (int i = rank * kPgThreads + tid; i < a.n; i += step) {
    int32_t* p = &a.sl[a.rows[i]];
    const int L = *reinterpret_cast<volatile int32_t*>(p);
    if (L < 0 || atomicCAS(p, L, ~L) != L) err |= SPEC_DERR_BAD_SLOT;
  }
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *entry(e);
    if (x < -1 || x >= a.NB) err |= SPEC_DERR_BAD_BLOCK;
  }
  if (top < 0 || top > a.NB) err |= SPEC_DERR_BAD_BLOCK;
  auto unclaim = [&]() {  // only reached with every CTA past its claims
    for (int i = rank * kPgThreads + tid; i < a.n; i += step) {
      int32_t* p = &a.sl[a.rows[i]];
      const int L = __ldcg(p);
      if (L < 0) atomicCAS(p, L, ~L);  // a row listed twice is undone once
    }
  };
  err = pg_exchange(cl, sh, 0, err).err;
  if (err != 0) {
    unclaim();
    if (rank == 0 && tid == 0) *a.status = err;
    return;
  }
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *entry(e);
    if (x >= 0) atomicSub(&a.refs[x], 1);
  }
  cl.sync();
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *entry(e);
    if (x >= 0 && __ldcg(&a.refs[x]) < -1) err |= SPEC_DERR_BAD_BLOCK;
  }
  auto give_back = [&]() {
    for (int e = e0 + tid; e < e1; e += kPgThreads) {
      const int x = *entry(e);
      if (x >= 0) atomicAdd(&a.refs[x], 1);
    }
    unclaim();
    if (rank == 0 && tid == 0) *a.status = err;
  };
  err = pg_exchange(cl, sh, 0, err).err;
  if (err != 0) {
    give_back();
    return;
  }
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *entry(e);
    if (x >= 0 && __ldcg(&a.refs[x]) <= -1) atomicMin(&a.refs[x], e - E - 1);
  }
  cl.sync();
  int cnt = 0;
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    const int x = *entry(e);
    cnt += x >= 0 && __ldcg(&a.refs[x]) == e - E - 1;
  }
  PgAll all = pg_exchange(cl, sh, cnt, 0);
  if (all.cnt > a.NB - top) {  // some id would be held twice
    for (int e = e0 + tid; e < e1; e += kPgThreads) {
      const int x = *entry(e);
      if (x >= 0 && __ldcg(&a.refs[x]) < -1) a.refs[x] = -1;
    }
    cl.sync();
    err = SPEC_DERR_BAD_BLOCK;
    give_back();
    return;
  }
  int carry = top + all.before;
  for (int f = e0; f < e1; f += kPgThreads) {
    const int e = f + tid;
    const int x = e < e1 ? *entry(e) : -1;
    const bool push = x >= 0 && __ldcg(&a.refs[x]) == e - E - 1;
    int sum;
    const int r = carry + pg_scan(push, sh.warp, sum);
    if (push) a.fs[r] = x;
    carry += sum;
  }
  cl.sync();  // every entry has been compared before a count changes
  for (int e = e0 + tid; e < e1; e += kPgThreads) {
    int32_t* p = entry(e);
    const int x = *p;
    if (x >= 0 && __ldcg(&a.refs[x]) == e - E - 1) a.refs[x] = 0;
    *p = -1;
  }
  for (int i = rank * kPgThreads + tid; i < a.n; i += step) a.sl[a.rows[i]] = 0;
  if (rank == 0 && tid == 0) {
    *a.ftop = top + all.cnt;
    *a.status = 0;
  }
}

int launch_kv_free(const KvFreeLaunch& k) {
  FreeArgs a{k.block_table, k.seq_lens, k.extra_refs, k.rows, k.num_blocks, k.B, k.max_blocks,
             k.n, k.free_stack, k.free_top, k.status};
  return launch_pdl(kv_free_kernel, dim3(kPgCluster), dim3(kPgThreads), 0,
                    static_cast<cudaStream_t>(k.stream), a);
}

}  // namespace sv
