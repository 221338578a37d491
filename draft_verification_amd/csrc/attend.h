// Attention of a step's rows over a paged cache: the plan of a step and what
// its kernels share.
//
// Queries of one key head - the rows of a request times the heads of a group,
// row by row - are taken M at a time: a tile.  A tile's tokens are taken TT at
// a time: units, whose keys and values pass through LDS once for all M
// queries.  Requests differ in length by orders of magnitude, and only the
// device knows them, so the units of all tiles, head after head, are cut into
// equal runs, one per workgroup: a run holds the end of one tile, whole tiles,
// and the beginning of another.  Whole tiles are finished where they are
// computed; the parts of a cut one go to the workspace, and a second launch
// joins them, in their order.
#pragma once

#include <initializer_list>

#include "cache_common.h"
#include "sdv_host.h"

namespace sdv {

constexpr int kAttnThreads = 256;
constexpr uint32_t kPlanMark = 0x5D9A7713u;

// What a plan was made for; the attention call has to say the same.
struct PlanShape {
  uint32_t mark;
  int R, q_max, n_q, n_kv, D, type, bs;
};

struct PlanHead {
  PlanShape shape;
  int causal, window;
  int n_tiles;
  int n_cuts;
  int slices;                // of a cut tile's parts, joined side by side
  int lead;                  // units that the beginning of a tile counts as
  long long total, quota;    // units: of all heads, per workgroup
};

struct Tile {
  int req, q0;       // request; first query, row * group + head of the group
  int u0, units;     // first unit of tokens and how many
  int queries;       // of the request
  int ctx, row0, n;  // tokens, first row and rows of the request
};

// Where a workgroup's run begins: off units into tile `index` (its lead first),
// a copy of which is here, so that a run begins with one read.
struct Start {
  Tile tile;
  int head, index, off, pad;
};

// A tile in parts: runs first .. last have one each.
struct CutTile {
  Tile tile;
  int head, first, last, pad;
};

// How a call is cut up, from what the host knows.
struct Cut {
  bool direct;
  int M, TT, W;            // queries per tile, tokens per unit, workgroups
  long long max_tiles;
  size_t tiles, sums, starts, cuts, ml, part, bytes;   // offsets in the workspace
};

// Whether a wave computes all queries of a tile of M (attend_direct.h): in 4
// bits, where neighbouring channels of a lane share scales and 16 neighbouring
// tokens a block, as long as the output's M x D sums fit its registers.  128
// contexts, one row each: 138 us, 168 with the values passed through LDS; two
// long ones with up to 40 queries a key head: 80 and 112 us.
constexpr bool attn_direct(int D, int M, bool fp4, int bs) {
  return fp4 && bs % 16 == 0 && ((D == 64 && M <= 64) || (D == 128 && M <= 48) || (D == 256 && M <= 16));
}

// Queries per tile: as few as hold those of a request's largest step (a
// workgroup multiplies all M columns, used or not), and at most what the
// registers hold beside the output's sums.  In tiles of 128 throughout, 128
// contexts of one row take 528 us instead of 474, in 4 bits 446 instead of 138,
// of up to 12 rows 294 instead of 286; pieces of prompts in tiles of 256 by
// eight waves 240 instead of 237.
inline int attn_queries(int q_max, int group, int D, bool fp4, int bs) {
  const long long n = (long long)q_max * group;
  for (int M : {16, 32, 48})
    if (n <= M && (attn_direct(D, M, fp4, bs) || M == 32 || (M == 16 && D <= 128))) return M;
  return n <= 64 || D > 128 ? 64 : 128;
}
// Tokens per unit.
constexpr int attn_unit(int D, int M, bool fp4) {
  return fp4 ? (D <= 128 && M < 128 ? 128 : 64) : D <= 128 ? 64 : 32;
}
// Neighbouring tokens that are loaded with one address where they lie in one
// block: all of a wave's quarter of a unit, or, in 4 bits, those of one load
// where the quarter is longer; 0: never.
// (bf16, an address for each piece: 518 instead of 474 us for 128 contexts of
// one row, 263 instead of 229 for pieces of prompts.)
constexpr int attn_span(int D, int M, bool fp4) {
  const int quarter = attn_unit(D, M, fp4) / 4, load = 64 / (D / 32);
  return !fp4 ? quarter : 64 % (D / 32) != 0 ? 0 : load < quarter ? load : quarter;
}

inline Cut attn_cut(int R, int q_max, int n_q, int n_kv, int D, int type, int bs) {
  Cut c;
  const bool fp4 = type == SD_CACHE_FP4;
  c.M = attn_queries(q_max, n_q / n_kv, D, fp4, bs);
  c.direct = attn_direct(D, c.M, fp4, bs);
  c.TT = c.direct ? 128 : attn_unit(D, c.M, fp4);
  // Two workgroups on each of 256 CUs, by their registers and LDS.  (Runs of a
  // half or a quarter, dispatched as others end, are no faster.)
  c.W = 512;
  c.max_tiles = (long long)R * (((long long)q_max * (n_q / n_kv) + c.M - 1) / c.M);
  size_t at = 256;
  auto take = [&](size_t n) {
    const size_t p = at;
    at = sdv_align256(at + n);
    return p;
  };
  c.tiles = take(sizeof(Tile) * (size_t)c.max_tiles);
  c.sums = take(8 * ((size_t)c.max_tiles + 1));
  c.starts = take(sizeof(Start) * ((size_t)c.W + 1));
  c.cuts = take(sizeof(CutTile) * (size_t)c.W);
  c.ml = take(8 * 2 * (size_t)c.W * c.M);
  c.part = take(4 * 2 * (size_t)c.W * c.M * D);
  c.bytes = at;
  return c;
}

struct AttnArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  long long ld_q, ld_out;
  const int32_t* table;
  int32_t* status;
  Cache cache;
  PlanShape shape;
  int max_blocks, n_rows;
  const PlanHead* head;
  const Tile* tiles;
  const Start* starts;
  const CutTile* cuts;
  float2* ml;        // [2 W][M] running maximum and sum of a part
  float* part;       // [2 W][M][D] its values, not divided yet
  float scale2;      // scale * log2(e)
  uint32_t block_tokens;   // n_kv * bs
  uint32_t bs_mul;   // token / bs = token * bs_mul >> bs_shift
  int bs_shift;
  int spans;         // tokens that are loaded together lie in one block
  int once;          // a request is one tile: what is loaded is not needed again
  int group;
  int n_q;
};

SDV_DEV bool same_shape(const PlanShape& x, const PlanShape& y) {
  return x.mark == y.mark && x.R == y.R && x.q_max == y.q_max && x.n_q == y.n_q && x.n_kv == y.n_kv && x.D == y.D &&
         x.type == y.type && x.bs == y.bs;
}

// The plan knows neither the table's width nor the rows of the buffers.
SDV_DEV bool in_range(const AttnArgs& a, const Tile& t) {
  return t.row0 <= a.n_rows - t.n && t.ctx <= (int64_t)a.max_blocks * a.cache.bs;
}

// One launch of the kernel for D, M and the cache's type.
int attend_bf16(hipStream_t stream, int M, int W, const AttnArgs& a);
int attend_fp4(hipStream_t stream, int M, int W, const AttnArgs& a);
int attend_direct(hipStream_t stream, int M, int W, const AttnArgs& a);

}  // namespace sdv
