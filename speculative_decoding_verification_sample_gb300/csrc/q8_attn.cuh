// Attention of a row's newest tokens over its 8-bit paged cache: the parts that
// the kernels share (arguments, visible keys, the split of the work).
//
// Row b holds L = seq_lens[b] committed tokens and n new ones (positions
// L .. L + n - 1, already in the cache). Query t of head hq sees key j when
//   chain: j <= L + t, and with a window w also j > L + t - w or j < sinks;
//   tree:  j < L, or bit j - L of tree_mask[b][t] is set;
// and computes, over the keys it sees, with z_j = softmax_scale * q . k_j,
//   out = sum_j exp(z_j - m) v_j / sum_j exp(z_j - m),  m = max_j z_j.
//
// Split. A key tile is 128 positions. An item is (row, kv head, row block): the
// query rows r = t * G + g of one kv head (G = q heads per kv head) in blocks
// of `rows_per_block`, so that a tile is read once for all of them. The units
// (item, tile) of the batch form one list, b outermost and the tile innermost,
// and CTA c of NC takes units [W c / NC, W (c + 1) / NC): equal work whatever
// the lengths, few rows or many. An item that lies in one CTA is written at
// once; one that crosses CTAs leaves in each a part (maximum, sum, unnormalised
// output), joined by a second kernel in CTA order, so the result does not
// depend on timing.
//
// With a plan (kv_prefix.cuh) rows may leave their first tiles, which they share
// with others, to another kernel: such a row begins at its tile `skip`, and what
// would be its output is left as a part.
#pragma once
#include <cstdint>

#include "../../include/specverify.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace sv {

constexpr int kAttnTile = 128;

// A plan of shared prefixes (kv_prefix.cuh): what it was made for, from byte 256 its rows, then
// the groups, their units from group to group, and the list of members.
struct alignas(16) PrefixHeader {
  int32_t magic, B, T, G, H, bs, MB, NG, NE;
  int64_t units;
  int32_t pad[52];
};
static_assert(sizeof(PrefixHeader) == 256, "the rows follow it");
constexpr int32_t kPrefixMagic = 0x70667832;
struct alignas(16) PrefixRow {
  int32_t L, n;       // as the plan found them
  int32_t skip;       // tiles that the row shares: those of its group, else 0
  int32_t group, at;  // group (skip 0: -1) and the row's place among its members
  int32_t pad[3];
};
struct PrefixGroup {  // tiles 0: nothing is shared
  int32_t tiles, row, entry, count;  // shared tiles, a row of the group, its members
};
struct PrefixLayout {  // byte offsets
  size_t groups, prefix, members, bytes;
};
__host__ __device__ inline PrefixLayout prefix_layout(int B, int NG, int NE) {
  PrefixLayout l;
  l.groups = sizeof(PrefixHeader) + size_t(B) * sizeof(PrefixRow);
  l.prefix = l.groups + size_t(NG) * sizeof(PrefixGroup);
  l.members = l.prefix + (size_t(NG) + 1) * 8;
  l.bytes = (l.members + size_t(NE) * 4 + 255) / 256 * 256;
  return l;
}
// Whether a plan of `bytes` was made for such calls (at least a header). The header is read in
// three loads that wait for nothing, and nothing waits for a part of the answer. (One comparison
// after the other, with a plan that shares nothing the kernel took 107 instead of 96 us for 130
// rows of 8 kv heads; without a plan it takes 90.)
__device__ __forceinline__ bool prefix_fits(const uint8_t* plan, size_t bytes, int B, int T, int G,
                                            int H, int bs, int MB) {
  const int4* h = reinterpret_cast<const int4*>(plan);
  const int4 x = h[0], y = h[1];      // magic, B, T, G; H, bs, MB, NG
  const int NE = h[2].x;
  const int other = (x.x ^ kPrefixMagic) | (x.y ^ B) | (x.z ^ T) | (x.w ^ G) | (y.x ^ H) | (y.y ^ bs) |
                    (y.z ^ MB);
  const bool sizes = (uint32_t(y.w) <= 1u << 20) & (uint32_t(NE) <= 1u << 20);
  return (other == 0) & sizes & (prefix_layout(B, y.w, NE).bytes <= bytes);
}
__device__ __forceinline__ const PrefixRow* prefix_row(const uint8_t* plan, int b) {
  return reinterpret_cast<const PrefixRow*>(plan + sizeof(PrefixHeader)) + b;
}

struct AttnArgs {
  static constexpr bool kPlan = false;
  const void* q;         // [B, T, H * G, D]
  const uint8_t* pool;   // at the layer
  const float* scales;   // at the layer
  const int32_t* bt;
  const int32_t* sl;
  const int32_t* nn;         // null: T
  const uint32_t* tree;      // null: chain
  void* out;
  float scale_log2;          // softmax_scale * log2(e)
  int window, sinks;
  int NB, H, G, D, bs, B, T, MB;
  int64_t block_bytes, block_scales;
  int R, RB, rows_per_block;  // rows of one kv head, their blocks
  float* parts;               // [2 NC][rows_per_block][D] unnormalised outputs
  float2* stats;              // [2 NC][rows_per_block] (maximum in log2 units, sum)
  int4* joins;                // [NC] (item row, kv head, row block, first CTA); x < 0: none
  int32_t* err;
  uint64_t wait_ns;           // limit of a wait of the tensor-core kernel
  int stall_row;              // -1, or the row whose V tiles are withheld (a test)
  int plane0;                 // tensor-map plane index of (block 0, this layer, keys, head 0)
  int planes_per_block;       // planes from block to block
};
// With a plan. Kernels are made for either: tests of a pointer in the kernels for calls without
// one took them from 207 to 220 us (256 rows of 512 to 4096 tokens).
struct PlanAttnArgs : AttnArgs {
  static constexpr bool kPlan = true;
  const uint8_t* plan;        // at least a header and B rows
  size_t plan_bytes;
  float* own;                 // [B T H G][D]: the parts of rows with shared tiles
  float2* own_stats;          // [B T H G]
};

struct RowSpan {
  int L, n, end;           // committed and new tokens; end = L + n
  int lo, sink_end;        // some query may see positions [0, sink_end) and [lo, end) only
  int sink_tiles, win_tile;  // tiles [0, sink_tiles) and [win_tile, ...)
  int tiles;
  bool bad;
};

__device__ __forceinline__ bool plan_fits(const PlanAttnArgs& a) {
  return prefix_fits(a.plan, a.plan_bytes, a.B, a.T, a.G, a.H, a.bs, a.MB);
}

template <class Args>
__device__ __forceinline__ RowSpan row_span(const Args& a, int b) {
  RowSpan s;
  s.L = a.sl[b];
  s.n = a.nn ? a.nn[b] : a.T;
  s.bad = s.L < 0 || s.n < 0 || s.n > a.T || int64_t(s.L) + s.n > int64_t(a.MB) * a.bs;
  s.lo = s.sink_end = 0;
  int skip = 0;
  if constexpr (Args::kPlan) {
    // lengths that changed since the plan was made: the row's keys are not the plan's
    const int4 r = *reinterpret_cast<const int4*>(prefix_row(a.plan, b));
    s.bad = s.bad | (r.x != s.L) | (r.y != s.n) | !plan_fits(a);
    skip = r.z;
  }
  if (s.bad || s.n == 0) {
    s.end = s.tiles = s.sink_tiles = s.win_tile = 0;
    return s;
  }
  s.end = s.L + s.n;
  const int all = (s.end + kAttnTile - 1) / kAttnTile;
  s.sink_tiles = 0;
  s.win_tile = Args::kPlan ? max(0, min(skip, s.L / kAttnTile)) : 0;
  if (a.window > 0 && s.L >= a.window) {
    s.lo = s.L - a.window + 1;
    s.sink_end = min(a.sinks, s.end);
    s.win_tile = s.lo / kAttnTile;
    s.sink_tiles = (s.sink_end + kAttnTile - 1) / kAttnTile;
    if (s.sink_tiles >= s.win_tile) s.sink_tiles = s.win_tile = 0;
  }
  s.tiles = s.sink_tiles + all - s.win_tile;
  return s;
}

__device__ __forceinline__ int tile_start(const RowSpan& s, int k) {
  return (k < s.sink_tiles ? k : k - s.sink_tiles + s.win_tile) * kAttnTile;
}

// Whether a row's outputs are left as parts (calls with a plan have no window).
template <class Args>
__device__ __forceinline__ bool leaves_part(const RowSpan& s) {
  return Args::kPlan && s.win_tile > 0;
}

// May a query of the row see a position of [p, p + n)? Blocks for which this is
// false are not read (a caller with a window may have freed them).
__device__ __forceinline__ bool needed(const RowSpan& s, int p, int n) {
  return p < s.end && (p + n > s.lo || p < s.sink_end);
}

// Does query t see key j (t < n, j < end)?
__device__ __forceinline__ bool sees(const AttnArgs& a, const RowSpan& s, uint32_t tmask, int t,
                                     int j) {
  if (t >= s.n || j >= s.end) return false;
  if (a.tree) return j < s.L || ((tmask >> (j - s.L)) & 1u);
  return j <= s.L + t && (a.window == 0 || j > s.L + t - a.window || j < a.sinks);
}

// Does every query of the row see every key of the tile that starts at p?
__device__ __forceinline__ bool tile_open(const AttnArgs& a, const RowSpan& s, int p) {
  const int last = p + kAttnTile - 1;
  if (s.n < a.T || last > s.L - (a.tree ? 1 : 0)) return false;
  return a.window == 0 || p > s.L + s.n - 1 - a.window || last < a.sinks;
}

// ------------------------------------------------------------------ split
struct AttnPlan {
  int64_t W;         // units of the batch
  int64_t u0, u1;    // this CTA's
  int nc;            // CTAs that take part: no more than units, so none of them is empty
};

// One stretch of consecutive tiles of one item.
struct Segment {
  int b, h, rb, t0, t1;  // tiles [t0, t1) of RowSpan::tiles
  RowSpan s;
  int64_t u;             // unit index of tile t0
};

// Every thread of the CTA; in shared memory `prefix` takes blockDim.x + 1 tile counts,
// `warp_sum` one of each warp.
template <class Args>
__device__ __forceinline__ AttnPlan attn_plan(const Args& a, int64_t* prefix, int64_t* warp_sum,
                                              int nc, int c) {
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  int64_t sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b < a.B) sum += row_span(a, b).tiles;
  }
  // inclusive scan: warps by shuffles, then their totals by every thread
  const int lane = threadIdx.x & 31;
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_sum[threadIdx.x >> 5] = inc;
  __syncthreads();
  for (int w = 0; w < int(threadIdx.x >> 5); ++w) inc += warp_sum[w];
  prefix[threadIdx.x + 1] = inc;
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
  AttnPlan p;
  p.W = prefix[blockDim.x] * a.H * a.RB;
  p.nc = int(min(int64_t(nc), p.W));
  // W c / nc, in 32 bits where that does
  auto share = [&](int i) -> int64_t {
    const int64_t n = p.W * i;
    return n >> 32 == 0 ? int64_t(uint32_t(n) / uint32_t(p.nc)) : n / p.nc;
  };
  p.u0 = c < p.nc ? share(c) : 0;
  p.u1 = c < p.nc ? share(c + 1) : 0;
  return p;
}

// The segment that starts at unit u of [u, u1).
template <class Args>
__device__ __forceinline__ Segment find_segment(const Args& a, const int64_t* prefix, int64_t u,
                                                int64_t u1) {
  const int64_t U = int64_t(a.H) * a.RB;
  // 64-bit division is a long routine: only where 32 bits do not do
  auto quotient = [](int64_t n, int64_t d) -> int64_t {
    return (n | d) >> 32 == 0 ? int64_t(uint32_t(n) / uint32_t(d)) : n / d;
  };
  const int64_t x = quotient(u, U);
  const int per = (a.B + blockDim.x - 1) / blockDim.x;
  int lo = 0, hi = (a.B + per - 1) / per - 1;  // the last chunk with prefix <= x
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (prefix[m] <= x) lo = m;
    else hi = m - 1;
  }
  Segment g;
  int64_t at = prefix[lo];
  int b = lo * per;
  RowSpan s = row_span(a, b);
  while (at + s.tiles <= x) {
    at += s.tiles;
    s = row_span(a, ++b);
  }
  const int64_t rem = u - at * U;
  const int hr = int(quotient(rem, s.tiles));
  g.b = b;
  g.s = s;
  g.t0 = int(rem - int64_t(hr) * s.tiles);
  g.h = hr / a.RB;
  g.rb = hr - g.h * a.RB;
  g.u = u;
  g.t1 = int(min(int64_t(s.tiles), g.t0 + (u1 - u)));
  return g;
}

// The segment after g, which ended its item (the caller checks that units are left).
template <class Args>
__device__ __forceinline__ void next_segment(const Args& a, Segment& g, int64_t u1) {
  g.u += g.t1 - g.t0;
  g.t0 = 0;
  if (++g.rb == a.RB) {
    g.rb = 0;
    if (++g.h == a.H) {
      g.h = 0;
      do g.s = row_span(a, ++g.b);
      while (g.s.tiles == 0);
    }
  }
  g.t1 = int(min(int64_t(g.s.tiles), u1 - g.u));
}

// Rows without keys: zeros, or NaN where the row's lengths are invalid. By thread
// `me` of `threads` of a CTA.
template <class T, class Args>
__device__ __forceinline__ void write_empty_rows(const Args& a, int c, int nc, int me,
                                                 int threads) {
  for (int b = c; b < a.B; b += nc) {
    const RowSpan s = row_span(a, b);
    if (s.tiles > 0) continue;
    const int64_t n = int64_t(a.T) * a.H * a.G * a.D;
    T* o = static_cast<T*>(a.out) + b * n;
    const T v = T(s.bad ? __uint_as_float(0x7fc00000u) : 0.0f);
    for (int64_t i = me; i < n; i += threads) o[i] = v;
    if (s.bad && a.err && me == 0) {
      int bit = SPEC_DERR_BAD_LENGTH;
      if constexpr (Args::kPlan) bit = plan_fits(a) ? bit : SPEC_DERR_BAD_SLOT;
      atomicOr(a.err, bit);
    }
  }
}

// The item that ends in CTA c and began in an earlier one, for the joining
// kernel (one thread). The CTA of unit u is the largest c with W c / NC <= u.
__device__ __forceinline__ void write_join(const AttnArgs& a, const AttnPlan& p, const Segment* first,
                                           int c) {
  int4 j = make_int4(-1, 0, 0, 0);
  if (first && first->t0 > 0 && first->t1 == first->s.tiles) {
    const int64_t begin = first->u - first->t0;
    int64_t c0 = begin * p.nc / p.W;
    while (p.W * (c0 + 1) / p.nc <= begin) ++c0;
    while (p.W * c0 / p.nc > begin) --c0;
    j = make_int4(first->b, first->h, first->rb, int(c0));
    // the first part lies in slot 1 of its CTA unless the item begins with the CTA
    if (p.W * c0 / p.nc != begin) j.w |= 1 << 30;
  }
  a.joins[c] = j;
}

// The tensor-core kernel (kv_q8_attention_tc.cu): whether it takes a call, its
// rows per block, and its launch, which sets `nc` to the number of CTAs.
bool attn_tc_takes(int dtype, int D, int bs, int64_t planes);
int attn_tc_rows(int R);
int launch_attn_tc(const AttnArgs& a, const void* pool_base, int64_t planes, int sms, int max_ctas,
                   int* nc, void* stream);
int launch_attn_tc(const PlanAttnArgs& a, const void* pool_base, int64_t planes, int sms,
                   int max_ctas, int* nc, void* stream);

}  // namespace sv
