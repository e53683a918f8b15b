// The plan of the prefix attention (kv_prefix.cuh), and the kernel that joins its parts.
//
// The plan. A cluster of 8 CTAs: each makes out in its own shared memory the rows' places in
// the list of members (the first, if one is listed twice), the groups' first rows and
// shortest lengths, and compares its share of the tables with those of the first rows;
// the first CTA takes the first differences from all and sums up the units. Where tables are too
// short to share anything by the estimate it only looks at the lists. Bound by latency, and for
// many long tables by reading them (as far as the rows reach, once): in a graph 3.7 us for lists
// alone, 8 us for 130 rows, 13 us for 256 rows that share 1000 blocks.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "kv_prefix.cuh"
#include "launch_util.cuh"

namespace sv {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8, kPlanThreads = 1024;
constexpr int kPlanChunk = 256;  // table entries that a warp compares at a time

struct PlanArgs {
  const int32_t *bt, *sl, *nn, *starts, *members;
  int NG, NE, T, G, H, NB, bs, B, MB, always, could;
  int per;  // queries of a warp of the join
  uint8_t* plan;
  int32_t* err;
};

// A test knob, read at every launch: share whatever rows have in common.
static bool share_always() {
  const char* s = std::getenv("SPECVERIFY_SHARE");
  return s && s[0] == '1';
}

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    kv_prefix_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t sm[];
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int64_t sums[3][kWarps];
  __shared__ int longest;  // of the members
  int32_t *common = sm, *first = common + a.NG, *shortest = first + a.NG, *live = shortest + a.NG,
          *starts = live + a.NG, *row_entry = starts + a.NG + 1;
  const cg::cluster_group cluster = cg::this_cluster();
  const bool lead = cluster.block_rank() == 0;
  const PrefixLayout lay = prefix_layout(a.B, a.NG, a.NE);
  PrefixHeader* head = reinterpret_cast<PrefixHeader*>(a.plan);
  PrefixGroup* groups = reinterpret_cast<PrefixGroup*>(a.plan + lay.groups);
  PrefixRow* rows = reinterpret_cast<PrefixRow*>(a.plan + sizeof(PrefixHeader));
  int64_t* prefix = reinterpret_cast<int64_t*>(a.plan + lay.prefix);
  int32_t* members = reinterpret_cast<int32_t*>(a.plan + lay.members);
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  for (int b = tid; b < a.B; b += kPlanThreads) row_entry[b] = INT32_MAX;
  for (int g = tid; g < a.NG; g += kPlanThreads) {
    first[g] = shortest[g] = common[g] = INT32_MAX;
    live[g] = 0;
  }
  if (tid == 0) longest = 0;
  pdl_wait();
  if (lead && tid == 0) head->magic = 0;

  // the list's bounds
  bool bad = false;
  for (int g = tid; g <= a.NG; g += kPlanThreads) {
    const int s = a.starts[g];
    starts[g] = s;
    bad = bad || s < 0 || s > a.NE || (g > 0 && s < a.starts[g - 1]);
  }
  bad = __syncthreads_or(bad);
  if (bad && lead && tid == 0 && a.err) atomicOr(a.err, SPEC_DERR_BAD_SLOT);
  const int e0 = bad ? 0 : starts[0], e1 = bad ? 0 : starts[a.NG];

  for (int i = e0 + tid; i < e1; i += kPlanThreads) {
    const int r = a.members[i];
    if (r >= 0 && r < a.B) atomicMin(&row_entry[r], i);
    else if (lead && a.err) atomicOr(a.err, SPEC_DERR_BAD_SLOT);
  }
  __syncthreads();
  auto group_of = [&](int i) {  // the last group that starts at or before entry i
    int lo = 0, hi = a.NG - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (starts[m] <= i) lo = m;
      else hi = m - 1;
    }
    return lo;
  };
  auto lengths = [&](int r, int& L, int& n) {  // whether they are valid
    L = a.sl[r];
    n = a.nn ? a.nn[r] : a.T;
    return L >= 0 && n >= 0 && n <= a.T && int64_t(L) + n <= int64_t(a.MB) * a.bs;
  };
  int top = 0;
  for (int i = e0 + tid; i < e1; i += kPlanThreads) {
    const int r = a.members[i];
    int member = -1;  // none: without queries
    if (r >= 0 && r < a.B) {
      int L, n;
      if (row_entry[r] != i) {
        if (lead && a.err) atomicOr(a.err, SPEC_DERR_BAD_SLOT);
      } else if (lengths(r, L, n) && n > 0) {
        member = r;
        const int g = group_of(i);
        atomicMin(&first[g], i);
        atomicMin(&shortest[g], L);
        atomicAdd(&live[g], 1);
        top = max(top, L);
      }
    }
    if (lead) members[i] = member;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0 && top > 0) atomicMax(&longest, top);
  // (the first CTA's shared memory is written by the others below)
  if (a.could) cluster.sync();
  else if (!lead) return;

  // Tables against the first row's, a warp 256 entries at a time, as far as rows reach: over the
  // whole width, tables for 131072 tokens took 47 us instead of 13 (256 rows behind 16000).
  const int chunks = a.could ? (longest / a.bs + kPlanChunk - 1) / kPlanChunk : 0;
  const int64_t tasks = int64_t(e1 - e0) * chunks;
  for (int64_t t = int64_t(cluster.block_rank()) * (kPlanThreads / 32) + (tid >> 5); t < tasks;
       t += kPlanCtas * kPlanThreads / 32) {
    const int i = e0 + int(t / chunks), j0 = int(t % chunks) * kPlanChunk;
    const int g = group_of(i);
    if (live[g] < 2) continue;
    const int j1 = min(shortest[g] / a.bs, j0 + kPlanChunk);
    if (j0 >= j1 || *reinterpret_cast<volatile int32_t*>(&common[g]) <= j0) continue;
    const int r = a.members[i];
    int L, n;
    if (r < 0 || r >= a.B || row_entry[r] != i || !lengths(r, L, n) || n == 0) continue;
    const int32_t* mine = a.bt + int64_t(r) * a.MB;
    const int32_t* other = a.bt + int64_t(a.members[first[g]]) * a.MB;
    int x[kPlanChunk / 32], y[kPlanChunk / 32];
#pragma unroll
    for (int k = 0; k < kPlanChunk / 32; ++k) {
      const int j = j0 + 32 * k + lane;
      x[k] = j < j1 ? mine[j] : 0;
      y[k] = j < j1 ? other[j] : 0;
    }
    int at = INT32_MAX;
#pragma unroll
    for (int k = kPlanChunk / 32 - 1; k >= 0; --k) {
      const int j = j0 + 32 * k + lane;
      if (j < j1 && (x[k] != y[k] || x[k] < 0 || x[k] >= a.NB)) at = j;
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (at != INT32_MAX && lane == 0) atomicMin(&common[g], at);
  }
  if (!lead) {
    __syncthreads();
    int32_t* to = cluster.map_shared_rank(common, 0);
    for (int g = tid; g < a.NG; g += kPlanThreads)
      if (common[g] != INT32_MAX) atomicMin(&to[g], common[g]);
  }
  if (a.could) cluster.sync();
  if (!lead) return;

  // What the groups share, in tiles, and what that saves. common[] holds it from here on.
  const int R = a.T * a.G;
  int64_t saved = 0, units_of = 0;
  int item = 0;
  for (int g = tid; g < a.NG; g += kPlanThreads) {
    const int tiles = bad || !a.could || live[g] < 2 ? 0
                                         : int(int64_t(min(common[g], shortest[g] / a.bs)) * a.bs /
                                               kPfTile);
    const int64_t gain =
        tiles == 0 ? 0 : pf_alone(live[g], tiles, R) - pf_shared(live[g], starts[g + 1] - starts[g], tiles, R);
    common[g] = a.always || gain > 0 ? tiles : 0;
    if (gain > 0) {
      const int64_t nq = int64_t(starts[g + 1] - starts[g]) * R;
      saved += gain;
      units_of += pf_units(nq, tiles);
      item = max(item, int(pf_item_units(nq > 128 ? kPfTwoUnits : kPfOneUnits, tiles)));
    }
  }
  bool share = a.always;
  if (a.could && !a.always) {
    auto sum_of = [](int64_t x) {  // of a warp
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      return x;
    };
    saved = sum_of(saved);
    units_of = sum_of(units_of);
    item = __reduce_max_sync(0xffffffffu, item);
    if (lane == 0) {
      sums[0][tid >> 5] = saved;
      sums[1][tid >> 5] = units_of;
      sums[2][tid >> 5] = item;
    }
    __syncthreads();
    static_assert(kWarps == 32, "a lane for each");
    saved = sum_of(sums[0][lane]) * a.H;
    units_of = sum_of(sums[1][lane]) * a.H;
    item = __reduce_max_sync(0xffffffffu, int(sums[2][lane]));
    share = saved > kPfLeast + pf_pieces(item, units_of, a.per);
  }
  __syncthreads();  // common[], and sums have been read
  auto shared_tiles = [&](int g) { return share ? common[g] : 0; };

  for (int b = tid; b < a.B; b += kPlanThreads) {
    PrefixRow r = {};
    const bool ok = lengths(b, r.L, r.n);
    r.group = r.at = -1;
    const int i = row_entry[b];
    if (ok && r.n > 0 && i != INT32_MAX) {
      const int g = group_of(i);
      r.skip = shared_tiles(g);
      if (r.skip > 0) {
        r.group = g;
        r.at = i - starts[g];
      }
    }
    rows[b] = r;
  }

  // units, and their sums from group to group: each thread some consecutive ones
  const int mine = (a.NG + kPlanThreads - 1) / kPlanThreads;
  auto entry = [&](int e) -> int64_t {
    const int tiles = shared_tiles(e);
    const int s0 = bad ? 0 : starts[e], many = bad ? 0 : starts[e + 1] - s0;
    groups[e] = PrefixGroup{tiles, tiles > 0 ? a.members[first[e]] : 0, s0, many};
    return a.H * pf_units(int64_t(many) * R, tiles);
  };
  int64_t sum = 0;
  for (int x = 0; x < mine; ++x) {
    const int e = tid * mine + x;
    if (e >= a.NG) break;
    prefix[e] = sum;  // of this thread's so far
    sum += entry(e);
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sums[0][tid >> 5] = inc;
  __syncthreads();
  for (int w = 0; w < (tid >> 5); ++w) inc += sums[0][w];
  for (int x = 0; x < mine; ++x) {
    const int e = tid * mine + x;
    if (e >= a.NG) break;
    prefix[e] += inc - sum;
  }
  if (tid == kPlanThreads - 1) {
    prefix[a.NG] = inc;
    head->units = inc;
    head->B = a.B;
    head->T = a.T;
    head->G = a.G;
    head->H = a.H;
    head->bs = a.bs;
    head->MB = a.MB;
    head->NG = a.NG;
    head->NE = a.NE;
    head->magic = kPrefixMagic;
  }
}

int launch_kv_prefix_plan(const KvPrefixPlanLaunch& k) {
  PlanArgs a;
  a.bt = k.block_table;
  a.sl = k.seq_lens;
  a.nn = k.num_new;
  a.starts = k.group_starts;
  a.members = k.group_rows;
  a.NG = k.num_groups;
  a.NE = k.num_members;
  a.T = k.T;
  a.G = k.G;
  a.H = k.H;
  a.NB = k.num_blocks;
  a.bs = k.block_size;
  a.B = k.B;
  a.MB = k.max_blocks;
  a.always = share_always();
  a.could = a.always || pf_could(a.B, a.MB, a.bs, a.T * a.G, a.H);
  a.per = pf_join_queries(int64_t(a.B) * a.H, a.T * a.G, kPfSms);
  a.plan = static_cast<uint8_t*>(k.plan);
  a.err = k.err;
  const size_t smem = (5 * size_t(a.NG) + 1 + a.B) * 4;
  static std::atomic<uint64_t> done{0};
  if (allow_smem(kv_prefix_plan_kernel, 200 * 1024, done) != SPEC_OK) return SPEC_ECUDA;
  return launch_pdl(kv_prefix_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), smem,
                    static_cast<cudaStream_t>(k.stream), a);
}

size_t kv_prefix_plan_size(int B, int num_groups, int num_members) {
  return prefix_layout(B, num_groups, num_members).bytes;
}

// ------------------------------------------------------------------ joining
// A warp takes up to 8 queries of a row and kv head. What their pieces are is found four lanes a
// query side by side: the row's own part, the first piece of the prefix (in the place of the
// query) and the second (in that of a CTA); further pieces, of items that cross several CTAs,
// come by two. Then the queries follow one by one, the lanes over the head's numbers. (Found for
// one query at a time, this was most of 750 instructions a query.) Bound by those that are left
// and by memory: 23 us for 40960 queries of 128 numbers.
constexpr int kPfJoinThreads = 256, kPfJoinWarps = kPfJoinThreads / 32;

template <int D>
__global__ void __launch_bounds__(kPfJoinThreads) kv_prefix_join_kernel(const PfArgs a, int ctas, int per) {
  constexpr int N = D / 32;  // numbers of a lane
  constexpr uint32_t kAll = 0xffffffffu;
  pdl_trigger();
  pdl_wait();
  const PfPlan p = pf_plan(a, ctas);
  const int R = a.T * a.G, chunks = (R + per - 1) / per;
  const int warp = blockIdx.x * kPfJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int bh = warp / chunks, b = bh / a.H, h = bh - b * a.H, r0 = (warp - bh * chunks) * per;
  if (b >= a.B) return;
  // rows that share nothing, and those whose lengths are not the plan's, are done
  if (!p.ok) return;
  const PrefixRow row = p.rows[b];
  if (row.group < 0 || row.L != a.sl[b] || row.n != (a.nn ? a.nn[b] : a.T)) return;
  auto quotient = [](int64_t n, int d) -> int64_t {
    return n >> 32 == 0 ? int64_t(uint32_t(n) / uint32_t(d)) : n / d;
  };
  const int r = r0 + (lane >> 2), t = r / a.G;
  const int64_t query = (int64_t(b) * a.T + t) * a.H * a.G + h * a.G + r - t * a.G;
  // even lanes: the item of the prefix, odd lanes: the row's own keys, one piece
  const bool own = lane & 1, has = (lane >> 2) < per && r < R && t < row.n;
  const int x0 = row.at * R + r;
  int64_t u = 0, end = 0;
  int w = kPfOneUnits, c0 = 0, c1 = 0;
  if (has && !own) {
    const PrefixGroup g = p.groups[row.group];
    const int qb = x0 / 256;
    const int64_t base = p.prefix[row.group],
                  per_h = quotient(p.prefix[row.group + 1] - base, a.H);
    if (int64_t(g.count) * R - qb * 256 > 128) w = kPfTwoUnits;
    u = base + h * per_h + qb * pf_item_units(kPfTwoUnits, g.tiles);
    end = u + pf_item_units(w, g.tiles);
    c0 = pf_owner(p, u + kPfItemUnits);
    c1 = pf_owner(p, end - 1);
  }
  // piece x of the lane's item: its statistics and numbers, if any
  auto piece = [&](int x, float2& st, const float*& part) {
    st = make_float2(-INFINITY, 0.0f);
    part = nullptr;
    const int c = c0 + x;
    if (!has || c > c1) return;
    if (x == 0) {
      st = (own ? a.stats[1] : a.stats[0])[query];
      part = (own ? a.parts[1] : a.parts[0]) + query * D;
      return;
    }
    const int64_t u0 = pf_share(p, c) - u, u1 = min(pf_share(p, c + 1), end) - u;
    if (pf_cut(u0, w) < pf_cut(u1, w)) {  // else no tile begins there
      const int64_t at = int64_t(c) * 256 + x0 % 256;
      st = a.mid_stats[at];
      part = a.mid + at * D;
    }
  };
  auto most = [](float x) {  // of four lanes
    x = fmaxf(x, __shfl_xor_sync(kAll, x, 1));
    return fmaxf(x, __shfl_xor_sync(kAll, x, 2));
  };
  auto sum = [](float x) {
    x += __shfl_xor_sync(kAll, x, 1);
    return x + __shfl_xor_sync(kAll, x, 2);
  };
  float2 st;
  const float* part;
  piece(lane >> 1 & 1, st, part);
  const float m = most(st.x), base = m == -INFINITY ? 0.0f : m;
  const float weight = ex2_approx(st.x - base), l = sum(st.y * weight);
  int more = max(c1 - c0, __shfl_xor_sync(kAll, c1 - c0, 1));

  for (int k = 0; k < per && r0 + k < R; ++k) {
    float o[N] = {};
    // the four pieces that the lanes of query k have
    auto add = [&](const float* part, float weight) {
      float v[4][N], f[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint64_t from = __shfl_sync(kAll, reinterpret_cast<uint64_t>(part), 4 * k + y);
        f[y] = __shfl_sync(kAll, weight, 4 * k + y);
#pragma unroll
        for (int i = 0; i < N; ++i) v[y][i] = 0.0f;
        if (from == 0) continue;
        const float* at = reinterpret_cast<const float*>(from) + N * lane;
        if constexpr (N == 4) {
          const float4 x = *reinterpret_cast<const float4*>(at);
          v[y][0] = x.x;
          v[y][1] = x.y;
          v[y][N - 2] = x.z;
          v[y][N - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(at);
          v[y][0] = x.x;
          v[y][1] = x.y;
        }
      }
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] += v[y][i] * f[y];
    };
    add(part, weight);
    float lk = __shfl_sync(kAll, l, 4 * k), mk = __shfl_sync(kAll, m, 4 * k);
    const int last = __shfl_sync(kAll, more, 4 * k);
#pragma unroll 1
    for (int x = 2; x <= last; x += 2) {
      float2 st2;
      const float* part2;
      piece(x + (lane >> 1 & 1), st2, part2);
      const float mn = fmaxf(mk, __shfl_sync(kAll, most(st2.x), 4 * k));
      const float base2 = mn == -INFINITY ? 0.0f : mn, was = ex2_approx(mk - base2);
      const float weight2 = ex2_approx(st2.x - base2);
      lk = lk * was + __shfl_sync(kAll, sum(st2.y * weight2), 4 * k);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] *= was;
      mk = mn;
      add(part2, weight2);
    }
    const float inv = lk == 0.0f ? 0.0f : 1.0f / lk;
    uint32_t x[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
      x[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    const int64_t at = __shfl_sync(kAll, query, 4 * k);
    uint32_t* to =
        reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + at * D) + N / 2 * lane;
    if constexpr (N == 4) *reinterpret_cast<uint2*>(to) = make_uint2(x[0], x[N / 2 - 1]);
    else *to = x[0];
  }
}

namespace {

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Places {  // byte offsets in the workspace
  size_t parts[2], stats[2], mid, mid_stats, each, bytes;
};
Places places(int B, int T, int H, int G, int D) {
  const int64_t queries = int64_t(B) * T * H * G;
  Places p;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t x = at;
    at += up256(n);
    return x;
  };
  for (int i = 0; i < 2; ++i) {
    p.parts[i] = take(size_t(queries) * D * sizeof(float));
    p.stats[i] = take(size_t(queries) * sizeof(float2));
  }
  p.mid = take(size_t(kPfMaxCtas) * 256 * D * sizeof(float));
  p.mid_stats = take(size_t(kPfMaxCtas) * 256 * sizeof(float2));
  p.each = take(kv_q8_attention_workspace(T, G, D));
  p.bytes = at;
  return p;
}

}  // namespace

bool kv_prefix_takes(int dtype, int D, int bs, int64_t planes) {
  return kv_q8_attention_on_tc(dtype, D, bs, planes) && bs % 16 == 0;
}

size_t kv_prefix_workspace(int B, int T, int H, int G, int D) {
  return places(B, T, H, G, D).bytes;
}

int launch_kv_prefix_attention(const Q8AttnLaunch& k, const void* plan, size_t plan_bytes) {
  if (!share_always() && !pf_could(k.B, k.max_blocks, k.bs, k.T * k.G, k.H))
    return launch_kv_q8_attention(k);
  PfArgs a = {};
  const int64_t layer_bytes = int64_t(2) * k.H * k.bs * k.D;
  a.q = k.q;
  a.pool = static_cast<const uint8_t*>(k.pool) + k.layer * layer_bytes;
  a.scales = k.scales + int64_t(k.layer) * 2 * k.H;
  a.bt = k.block_table;
  a.sl = k.seq_lens;
  a.nn = k.num_new;
  a.out = k.out;
  a.plan = static_cast<const uint8_t*>(plan);
  a.plan_bytes = plan_bytes;
  a.scale_log2 = float(double(k.softmax_scale) * 1.4426950408889634);
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
  const Places p = places(k.B, k.T, k.H, k.G, k.D);
  uint8_t* ws = static_cast<uint8_t*>(k.workspace);
  for (int i = 0; i < 2; ++i) {
    a.parts[i] = reinterpret_cast<float*>(ws + p.parts[i]);
    a.stats[i] = reinterpret_cast<float2*>(ws + p.stats[i]);
  }
  a.mid = reinterpret_cast<float*>(ws + p.mid);
  a.mid_stats = reinterpret_cast<float2*>(ws + p.mid_stats);
  a.err = k.err;
  // the failure-detection knobs of kv_q8_attention
  a.wait_ns = kWaitNs;
  a.stall_row = -1;
  if (const char* row = std::getenv("SPECVERIFY_STALL_ROW")) {
    const long b = std::strtol(row, nullptr, 10);
    if (b >= 0 && b < a.B) a.stall_row = int(b);
    if (const char* ns = std::getenv("SPECVERIFY_IDLE_NS")) {
      const long long v = std::strtoll(ns, nullptr, 10);
      if (v > 0 && uint64_t(v) < kWaitNs) a.wait_ns = uint64_t(v);
    }
  }
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ECUDA;
  if (dev < 64) sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ECUDA;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  const int ctas = sms < kPfMaxCtas ? sms : kPfMaxCtas;
  a.plane0 = k.layer * 2 * k.H;
  a.planes_per_block = k.num_layers * 2 * k.H;
  const int st = launch_pf_attention(a, k.pool, int64_t(k.num_blocks) * a.planes_per_block, ctas,
                                     k.stream);
  if (st != SPEC_OK) return st;
  Q8AttnLaunch rows = k;
  rows.workspace = ws + p.each;
  rows.plan = plan;
  rows.plan_bytes = plan_bytes;
  rows.own = a.parts[1];
  rows.own_stats = a.stats[1];
  const int sr = launch_kv_q8_attention(rows);
  if (sr != SPEC_OK) return sr;
  cudaStream_t stream = static_cast<cudaStream_t>(k.stream);
  const int R = a.T * a.G, per = pf_join_queries(int64_t(a.B) * a.H, R, sms);
  const int chunks = (R + per - 1) / per;
  const int64_t warps = int64_t(a.B) * a.H * chunks;
  const dim3 grid(unsigned((warps + kPfJoinWarps - 1) / kPfJoinWarps));
  return a.D == 128
             ? launch_pdl(kv_prefix_join_kernel<128>, grid, dim3(kPfJoinThreads), 0, stream, a, ctas, per)
             : launch_pdl(kv_prefix_join_kernel<64>, grid, dim3(kPfJoinThreads), 0, stream, a, ctas, per);
}

}  // namespace sv
