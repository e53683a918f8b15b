// Attention of rows whose block tables begin with the same blocks: the plan, the
// split of the work, and the parts that the kernels share.
//
// What is computed is kv_q8_attention's (q8_attn.cuh), without a window. For a group
// of rows the key tiles (128 positions) that every row of it has in common and sees
// whole, the prefix, are read once for all of their queries, by a kernel in which those
// are the products' M rows; what follows is each row's own and left to kv_q8_attention's
// kernel, in which a few queries are the products' N columns. Softmax sums over disjoint
// keys join exactly: a part is (m, l, o) with m >= about the largest z_j, l = sum
// 2^(z_j - m), o = sum 2^(z_j - m) v_j in log2 units, and parts add up as
// 2^(m_i - M) (l_i, o_i). A row that shares nothing is kv_q8_attention's from end to end.
// (An earlier form took the rows' own keys with queries as M rows too, four rows in one M
// tile: 246 us for 8 times 16 candidates of drafts, where each row by itself takes 179.)
//
// Sharing pays where the prefix is long and the rows are many: the plan compares, for each
// group, what its tiles cost row by row with what they cost shared, and shares nothing at all
// where that saves less than the two kernels more cost once they have work.
//
// Split of the shared part. A group's queries (all rows of it, row by row) are taken in
// blocks of 256, two M tiles of the tensor core, the last one maybe one tile. An item is
// (group, kv head, block). The units of all items form one list, groups outermost, then kv
// heads, blocks, tiles; CTA c of NC takes units [W c / NC, W (c + 1) / NC), of each item the
// tiles that begin there. A piece that begins its item leaves its part in the place of its
// queries, another one in the place of its CTA, which has at most one such. Everything
// follows from the plan, so the result does not depend on timing.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "ptx.cuh"
#include "q8_attn.cuh"

namespace sv {

constexpr int kPfTile = 128;      // keys of a tile, queries of an M tile
constexpr int kPfMaxCtas = 256;   // bound of the work split, for the workspace

// What an item costs, in units of 0.36 us: its beginning and end (queries, parts), a key tile
// with two M tiles, one with one (measured: 64 items of 94 tiles more take 86 and 57 us longer).
constexpr int kPfItemUnits = 24, kPfTwoUnits = 6, kPfOneUnits = 4;
__host__ __device__ inline int64_t pf_item_units(int w, int64_t tiles) {
  return kPfItemUnits + w * tiles;
}
// Units of one kv head of a group with nq queries and `tiles` key tiles (none: no items).
__host__ __device__ inline int64_t pf_units(int64_t nq, int64_t tiles) {
  const int64_t full = nq / 256;
  const int rest = int(nq % 256);
  if (tiles == 0) return 0;
  return full * pf_item_units(kPfTwoUnits, tiles) +
         (rest > 128 ? pf_item_units(kPfTwoUnits, tiles)
          : rest > 0 ? pf_item_units(kPfOneUnits, tiles)
                     : 0);
}
// The estimate by which the plan shares, in 10 ns of an SM for each kv head. What a row costs
// either way (its item of kv_q8_attention's kernel, 1 to 6 us with its change) is not in it.
//
// Fitted to 7502 measured pairs of times, the same call with a plan that shares nothing and with
// all shared: 2 to 256 rows in 1 to 8 groups, 2 to 256 tiles in common, 1 to 16 kv heads of 64 and
// 128 numbers, 1 to 128 queries a row and kv head. The way taken is more than 5 % slower than the
// other in 2.5 % of them; with heads of 128 at most 1.14 times, with heads of 64, for which the
// plan shares late (it is not told of them), 1.30. (A price of 0.60 us a tile, changes of items
// included, and none for the join's further pieces: 4.8 %, 2.9 times.) Some of them, with 8 kv
// heads of 128, row by row and shared, us:
//
//   queries  rows     4 tiles        8       16       24       32       64      128      256
//      4     1 x 16    21, 34   22, 35   25, 38   28, 39   32, 40   45, 45   79, 57  130, 68
//     20     1 x 16    25, 41   26, 45   32, 46   33, 52   40, 52   56, 57   84, 76  146, 110
//     20     8 x 16    64, 90   76, 93  101, 107 133, 132 163, 148 289, 210
//     64     8 x 8     63, 108  81, 109 113, 128 144, 142 175, 152 298, 212 544, 324
//    128     8 x 16   175, 283 236, 311 357, 377 479, 432 598, 485
//
// kPfTile keys of one row, with the columns that its queries take in kv_q8_attention's kernel.
__host__ __device__ inline int pf_tile_price(int columns) {
  return columns <= 8    ? 52
         : columns <= 16 ? 55
         : columns <= 24 ? 57
         : columns <= 32 ? 67
         : columns <= 48 ? 79
                         : 115;
}
// What `tiles` tiles of `rows` rows with R queries each cost row by row: blocks of up to 64.
__host__ __device__ inline int64_t pf_alone(int64_t rows, int64_t tiles, int R) {
  const int blocks = (R + 63) / 64;
  return rows * tiles * blocks * pf_tile_price((R + blocks - 1) / blocks);
}
// The same shared: the units, 0.32 us each by the fit, the parts and their join 0.13 us a query.
__host__ __device__ inline int64_t pf_shared(int64_t rows, int64_t many, int64_t tiles, int R) {
  return 32 * pf_units(many * R, tiles) + rows * R * 13;
}
// What the kernels cost once they find work, whatever it is: 27 us of all SMs (kPfSms of them).
constexpr int kPfSms = 152;
constexpr int64_t kPfLeast = int64_t(2700) * kPfSms;
// And what the join waits for where few items are cut over many CTAs: 0.25 us for each piece
// beyond two and query of a warp. `item`: units of the longest item, `units`: of all.
__host__ __device__ inline int64_t pf_pieces(int64_t item, int64_t units, int per) {
  const int64_t all = item * (units < kPfSms ? units : kPfSms);
  if (all < 2 * units || units == 0) return 0;
  const int64_t each = all >> 32 == 0 ? int64_t(uint32_t(all) / uint32_t(units)) : all / units;
  return 25 * kPfSms * (each - 1) * per;
}
// Queries of a warp of the join: as few as all warps can take at once (32 on each SM), in equal
// chunks of a row and kv head's.
constexpr int kPfJoinQueries = 8;
__host__ __device__ inline int pf_join_queries(int64_t rows_heads, int R, int sms) {
  const int64_t at_once = int64_t(sms) * 32, each = (rows_heads * R + at_once - 1) / at_once;
  const int per = each < 1 ? 1 : each > kPfJoinQueries ? kPfJoinQueries : int(each);
  const int chunks = (R + per - 1) / per;
  return (R + chunks - 1) / chunks;
}
// Whether rows of such sizes could share enough of their tables.
__host__ inline bool pf_could(int B, int MB, int bs, int R, int H) {
  return pf_alone(B, int64_t(MB) * bs / kPfTile, R) * H > kPfLeast;
}

// Tiles of an item that begin before its unit x (divided by one of two constants: a division
// of 64 bits by w is a hundred instructions).
__host__ __device__ inline int pf_cut(int64_t x, int w) {
  if (x <= kPfItemUnits) return 0;
  const uint64_t n = uint64_t(x - kPfItemUnits);
  return int(w == kPfOneUnits ? (n + kPfOneUnits - 1) / kPfOneUnits
                              : (n + kPfTwoUnits - 1) / kPfTwoUnits);
}

struct PfArgs {
  const void* q;           // [B, T, H * G, D] bf16
  const uint8_t* pool;     // at the layer
  const float* scales;     // at the layer
  const int32_t* bt;
  const int32_t *sl, *nn;
  void* out;
  const uint8_t* plan;
  size_t plan_bytes;
  float scale_log2;
  int NB, H, G, D, bs, B, T, MB;
  int64_t block_bytes, block_scales;
  float* parts[2];         // [B T H G][D]: of the prefix, of the row's own keys
  float2* stats[2];        // [B T H G]
  float* mid;              // [CTAs][256][D]
  float2* mid_stats;       // [CTAs][256]
  int32_t* err;
  uint64_t wait_ns;
  int stall_row;           // -1, or the row with which a group begins whose keys are withheld (a test)
  int plane0;              // tensor-map plane of (block 0, this layer, keys, head 0)
  int planes_per_block;
};

// The plan as a kernel sees it; `ok` false: not a plan for this call.
struct PfPlan {
  bool ok;
  int NG, NE, nc;
  int64_t W;
  const PrefixGroup* groups;
  const PrefixRow* rows;
  const int64_t* prefix;
  const int32_t* members;
};
__device__ __forceinline__ PfPlan pf_plan(const PfArgs& a, int ctas) {
  PfPlan p;
  const PrefixHeader* h = reinterpret_cast<const PrefixHeader*>(a.plan);
  p.NG = h->NG;
  p.NE = h->NE;
  p.ok = prefix_fits(a.plan, a.plan_bytes, a.B, a.T, a.G, a.H, a.bs, a.MB);
  const PrefixLayout l = prefix_layout(a.B, p.ok ? p.NG : 0, p.ok ? p.NE : 0);
  p.W = p.ok ? h->units : 0;
  p.nc = int(p.W < ctas ? p.W : ctas);
  p.groups = reinterpret_cast<const PrefixGroup*>(a.plan + l.groups);
  p.rows = prefix_row(a.plan, 0);
  p.prefix = reinterpret_cast<const int64_t*>(a.plan + l.prefix);
  p.members = reinterpret_cast<const int32_t*>(a.plan + l.members);
  return p;
}
// First unit of CTA i (W i / nc), in 32 bits where that does.
__device__ __forceinline__ int64_t pf_share(const PfPlan& p, int i) {
  const int64_t n = p.W * i;
  return n >> 32 == 0 ? int64_t(uint32_t(n) / uint32_t(p.nc)) : n / p.nc;
}
// The CTA of unit u: the largest c with W c / nc <= u.
__device__ __forceinline__ int pf_owner(const PfPlan& p, int64_t u) {
  const int64_t n = (u + 1) * p.nc - 1;
  return int((n | p.W) >> 32 == 0 ? int64_t(uint32_t(n) / uint32_t(p.W)) : n / p.W);
}

int launch_pf_attention(const PfArgs& a, const void* pool_base, int64_t planes, int ctas,
                        void* stream);

}  // namespace sv
