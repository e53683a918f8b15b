// Attention of rows whose block tables begin with the same blocks: the plan, the
// split of the work, and the parts that the kernels share.
//
// What is computed is kv_q8_attention's (q8_attn.cuh), without a window. For a group
// of rows the key tiles (128 positions) that every row of it has in common and sees
// whole, the prefix, are read once for all of their queries; what follows is each
// row's own. Softmax sums over disjoint keys join exactly: a part is (m, l, o) with
// m >= about the largest z_j, l = sum 2^(z_j - m), o = sum 2^(z_j - m) v_j in log2
// units, and parts add up as 2^(m_i - M) (l_i, o_i).
//
// Entries: first the groups, then the rows' own keys. A group's queries (all rows of it,
// row by row) are taken in blocks of 256, two M tiles of the tensor core, the last one
// maybe one tile; a row's queries R = T G likewise, but with R <= 32 four consecutive rows,
// with R <= 64 two, share one M tile, a pack: their key tiles follow each other, and a
// tile's probabilities are zero for the other rows of the pack, which are other warps'. (An
// item for each row, with 20 of 128 places in use, spent 15 us each on its beginning and
// end.) An item is (entry, kv head, block). The units of all items form one list, entries
// outermost, then kv heads, blocks, tiles; CTA c of NC takes units [W c / NC,
// W (c + 1) / NC), of each item the tiles that begin there. A piece that begins its item
// leaves its part in the place of its queries (one place for the prefix, one for the row's
// own keys), another one in the place of its CTA, which has at most one such. Everything
// follows from the plan, so the result does not depend on timing.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/specverify.h"
#include "launch.h"
#include "ptx.cuh"

namespace sv {

constexpr int kPfTile = 128;      // keys of a tile, queries of an M tile
constexpr int kPfMaxCtas = 256;   // bound of the work split, for the workspace
constexpr int32_t kPfMagic = 0x70667831;

struct PfHeader {   // 256 bytes
  int32_t magic, B, T, G, H, bs, MB, NG, NE;
  int64_t units;    // W
  int32_t pad[52];
};
static_assert(sizeof(PfHeader) == 256, "the arrays follow it");

struct PfGroup {    // tiles 0: nothing is shared
  int32_t tiles, row, entry, count;  // shared tiles, a row of the group, its members
};
struct PfRow {
  int32_t L, n;       // as the plan found them
  int32_t skip;       // tiles of the group's prefix
  int32_t tiles;      // tiles from there to the end; -1: lengths that are not valid
  int32_t group, at;  // group (-1: none) and the row's place among its members
  int32_t pad[2];
};

// The plan's arrays, by their byte offsets.
struct PfLayout {
  size_t groups, rows, prefix, members, bytes;
};
__host__ __device__ inline PfLayout pf_layout(int B, int NG, int NE) {
  PfLayout l;
  l.groups = sizeof(PfHeader);
  l.rows = l.groups + size_t(NG) * sizeof(PfGroup);
  l.rows = (l.rows + 31) / 32 * 32;
  l.prefix = l.rows + size_t(B) * sizeof(PfRow);
  l.members = l.prefix + (size_t(NG) + B + 1) * 8;
  l.bytes = (l.members + size_t(NE) * 4 + 255) / 256 * 256;
  return l;
}

// Rows of a pack with R queries each.
__host__ __device__ inline int pf_pack(int R) { return R <= 32 ? 4 : R <= 64 ? 2 : 1; }

// What an item costs: its beginning and end (queries, parts), a key tile with two M tiles,
// one with one. The split only needs their proportions (2.4 us a tile with two: 0.5 us each).
constexpr int kPfItemUnits = 16, kPfTwoUnits = 5, kPfOneUnits = 4;
__host__ __device__ inline int64_t pf_item_units(int w, int64_t tiles) {
  return kPfItemUnits + w * tiles;
}
// Units of one kv head of an entry with nq queries and `tiles` key tiles (none: no items).
__host__ __device__ inline int64_t pf_units(int64_t nq, int64_t tiles) {
  const int64_t full = nq / 256;
  const int rest = int(nq % 256);
  if (tiles == 0) return 0;
  return full * pf_item_units(kPfTwoUnits, tiles) +
         (rest > 128 ? pf_item_units(kPfTwoUnits, tiles)
          : rest > 0 ? pf_item_units(kPfOneUnits, tiles)
                     : 0);
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
  const uint32_t* tree;    // null: a chain
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
  int stall_row;           // -1, or the row whose own keys are withheld (a test)
  int plane0;              // tensor-map plane of (block 0, this layer, keys, head 0)
  int planes_per_block;
};

// The plan as a kernel sees it; `ok` false: not a plan for this call.
struct PfPlan {
  bool ok;
  int NG, NE, nc;
  int64_t W;
  const PfGroup* groups;
  const PfRow* rows;
  const int64_t* prefix;
  const int32_t* members;
};
__device__ __forceinline__ PfPlan pf_plan(const PfArgs& a, int ctas) {
  PfPlan p;
  const PfHeader* h = reinterpret_cast<const PfHeader*>(a.plan);
  p.NG = h->NG;
  p.NE = h->NE;
  p.ok = h->magic == kPfMagic && h->B == a.B && h->T == a.T && h->G == a.G && h->H == a.H &&
         h->bs == a.bs && h->MB == a.MB && p.NG >= 0 && p.NE >= 0 && p.NG <= (1 << 20) &&
         p.NE <= (1 << 20) && pf_layout(a.B, p.NG, p.NE).bytes <= a.plan_bytes;
  const PfLayout l = pf_layout(a.B, p.ok ? p.NG : 0, p.ok ? p.NE : 0);
  p.W = p.ok ? h->units : 0;
  p.nc = int(p.W < ctas ? p.W : ctas);
  p.groups = reinterpret_cast<const PfGroup*>(a.plan + l.groups);
  p.rows = reinterpret_cast<const PfRow*>(a.plan + l.rows);
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
