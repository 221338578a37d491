// sd_attn_plan and sd_cache_attn: how a step's attention is cut up, the entry
// points, and the joining of tiles that were cut.
#include "attend.h"

namespace {

using namespace sdv;

constexpr int kPlanThreads = 1024;
constexpr int kMaxTokens = 0x7FFFFFFF - 256;
// Units that a workgroup takes at least: a shorter run costs more to join than
// it saves.
constexpr int kMinQuota = 2;
// What the beginning of a tile costs, in units: its loads begin from nothing.
// Runs are equal with it (16 requests, pieces of up to 512 rows and single
// rows, 32 query heads on 8 of 128: 235 us, 270 without, 239 with 8 units; 128
// requests of up to 12 rows over 512 to 8192 tokens: 283, 291 and 290 us).
// Where runs are short it would leave workgroups without one: it counts from
// so many times as many units to a run on.
constexpr int kLead = 4, kLeadRuns = 4;

struct PlanArgs {
  const int32_t* row0;
  const int32_t* ell;
  const int32_t* ctx;
  int32_t* status;
  PlanHead* head;
  Tile* tiles;
  long long* sums;
  Start* starts;
  CutTile* cuts;
  PlanShape shape;
  int causal, window, M, TT, W, group;
};

// Exclusive prefix sums over the workgroup; *total gets the sum.
SDV_DEV long long block_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  long long s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long t = __shfl_up(s, o, 64);
    if (lane >= o) s += t;
  }
  __syncthreads();   // part may still be read from the last call
  if (lane == 63) part[wave] = s;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int w = 0; w < waves; ++w) {
    if (w < wave) before += part[w];
    sum += part[w];
  }
  *total = sum;
  return before + s - v;
}

// One workgroup: the tiles of all requests, the units before each of them, and
// where every run begins.  A chain of small reads, once per step: 12 us for 4
// requests, 17 us for 128 (some 60 layers' calls share it).  One thread writes a
// request's tiles: 62 us where a prompt of 8192 rows has 256 of them.
__global__ __launch_bounds__(kPlanThreads) void k_plan(PlanArgs a) {
  __shared__ long long part[kPlanThreads / 64];
  const int R = a.shape.R;
  long long n_tiles = 0, total, mine = 0;
  for (int r0 = 0; r0 < R; r0 += blockDim.x) {
    const int r = r0 + threadIdx.x;
    Tile t = {};
    int count = 0;
    if (r < R) {
      const int ell = a.ell[r];
      t.req = r;
      t.n = ell < 0 ? 0 : ell < a.shape.q_max ? ell + 1 : a.shape.q_max;
      t.ctx = a.ctx[r];
      t.row0 = a.row0[r];
      t.queries = t.n * a.group;
      const bool bad = t.n > 0 && (t.ctx < t.n || t.ctx > kMaxTokens || t.row0 < 0);
      a.status[r] = bad ? SD_ST_BAD_INPUT : 0;
      count = bad ? 0 : (t.queries + a.M - 1) / a.M;
    }
    long long at = n_tiles + block_scan(count, part, &total);
    n_tiles += total;
    for (int j = 0; j < count; ++j) {
      t.q0 = j * a.M;
      const int base = t.ctx - t.n, first = t.q0 / a.group, last = (min(t.q0 + a.M, t.queries) - 1) / a.group;
      const int lo = a.window && base + first + 1 > a.window ? base + first + 1 - a.window : 0;
      const int hi = a.causal ? base + last + 1 : t.ctx;
      t.u0 = lo / a.TT;
      t.units = (hi + a.TT - 1) / a.TT - t.u0;
      mine += t.units;
      a.tiles[at + j] = t;
    }
  }
  block_scan(mine, part, &total);
  const int lead = total * a.shape.n_kv >= (long long)kLeadRuns * kLead * a.W ? kLead : 0;
  __syncthreads();
  long long units = 0;
  for (long long i0 = 0; i0 < n_tiles; i0 += blockDim.x) {
    const long long i = i0 + threadIdx.x;
    const int n = i < n_tiles ? a.tiles[i].units + lead : 0;
    const long long before = units + block_scan(n, part, &total);
    units += total;
    if (i < n_tiles) a.sums[i] = before;
  }
  const long long all = units * a.shape.n_kv;
  long long quota = (all + a.W - 1) / a.W;
  if (quota < kMinQuota) quota = kMinQuota;
  __syncthreads();
  // One thread per run (no more than threads): where it begins, and whether
  // the tile at its end is cut there and began in it.
  const int w = threadIdx.x;
  Start s = {};
  auto start_of = [&](int run) {
    const long long at = run * quota;
    Start x = {};
    if (run >= a.W || at >= all) return x;
    x.head = (int)(at / units);
    const long long rest = at - x.head * units;
    long long lo = 0, hi = n_tiles;   // sums[lo] <= rest < sums[hi]
    while (hi - lo > 1) {
      const long long mid = (lo + hi) >> 1;
      if (a.sums[mid] <= rest) lo = mid;
      else hi = mid;
    }
    x.index = (int)lo;
    x.off = (int)(rest - a.sums[lo]);
    x.tile = a.tiles[lo];
    return x;
  };
  s = start_of(w);
  if (w < a.W) a.starts[w] = s;
  const Start next = start_of(w + 1);
  const bool cut = next.off > lead && next.off - quota <= lead;
  const long long at = block_scan(cut ? 1 : 0, part, &total);
  const long long n_cuts = total;
  int last = 0;
  if (cut) {
    last = (int)(((w + 1) * quota - next.off + lead + next.tile.units - 1) / quota);
    a.cuts[at] = CutTile{next.tile, next.head, w, last, 0};
  }
  block_scan(cut ? last - w + 1 : 0, part, &total);
  if (threadIdx.x == 0) {
    PlanHead h = {};
    h.shape = a.shape;
    h.causal = a.causal;
    h.window = a.window;
    h.n_tiles = (int)n_tiles;
    h.n_cuts = (int)n_cuts;
    // eight parts or more to a slice
    h.slices = 1;
    while (h.slices < 8 && total >= 16 * h.slices * n_cuts) h.slices *= 2;
    h.lead = lead;
    h.total = all;
    h.quota = quota;
    *a.head = h;
  }
}

constexpr int kJoinThreads = 256;
constexpr int kJoinGrid = 2048;

// Joins the parts of cut tiles, in the order of the runs: D / 4 threads to a
// query and a slice of its parts (every slices-th one), slices through LDS.
// With part p's maximum m_p, sum l_p and values o_p, and m the largest m_p:
// out = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.  Two parts a run are
// read at most: 5.5 us for tiles of 16 queries by 128 channels, 17 us for tiles
// of 128 (64 MB at most, most of it still in the caches); latency bounds both.
// With four queries to a thread 32 parts of 48 queries took 10.5 us, one takes
// 5.7; the many tiles of two parts each took 1 us less.
template <int D>
__global__ __launch_bounds__(kJoinThreads) void k_join(AttnArgs a, int M) {
  constexpr int TQ = D / 4, QB = kJoinThreads / TQ;
  __shared__ float4 so[kJoinThreads];
  __shared__ float2 sml[kJoinThreads];
  const PlanHead& p = *a.head;
  if (!same_shape(p.shape, a.shape)) return;
  const int slices = p.slices <= QB ? p.slices : QB >= 8 ? 8 : 4;   // QB is 4 at least
  const int per = QB / slices, jobs = (M + per - 1) / per;
  const int mine = threadIdx.x / TQ, d = threadIdx.x % TQ * 4, slice = mine / per;
  for (long long job = blockIdx.x; job < (long long)p.n_cuts * jobs; job += gridDim.x) {
    const CutTile c = a.cuts[job / jobs];
    const Tile& t = c.tile;
    if (!in_range(a, t)) continue;   // the same for all threads
    const int q = (int)(job % jobs) * per + mine % per, qi = t.q0 + q;
    const bool in = q < M && qi < t.queries;
    float top = -__builtin_huge_valf(), l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float2& ml, const float4& v) {
      const float to = fmaxf(top, ml.x), ref = to == -__builtin_huge_valf() ? 0.f : to;
      const float f = fast_exp2(top - ref), h = fast_exp2(ml.x - ref);
      top = to;
      l = l * f + ml.y * h;
      o.x = o.x * f + v.x * h, o.y = o.y * f + v.y * h;
      o.z = o.z * f + v.z * h, o.w = o.w * f + v.w * h;
    };
    if (slice < slices) {
#pragma unroll 4
      for (int k = c.first + slice; k <= c.last; k += slices) {
        const int64_t slot = (int64_t)(k == c.first ? 2 * k + 1 : 2 * k) * M + (in ? q : 0);   // column 0 is always a query
        add(a.ml[slot], *(const float4*)(a.part + slot * D + d));
      }
    }
    if (slices > 1) {
      so[threadIdx.x] = o;
      sml[threadIdx.x] = make_float2(top, l);
      __syncthreads();
      if (slice == 0)
        for (int k = 1; k < slices; ++k) add(sml[threadIdx.x + k * per * TQ], so[threadIdx.x + k * per * TQ]);
      __syncthreads();
    }
    if (slice > 0 || !in) continue;
    const int row = qi / a.group, head = c.head * a.group + qi - row * a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *(uint2*)(a.out + (int64_t)(t.row0 + row) * a.ld_out + (int64_t)head * D + d) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (a.lse && d == 0)
      a.lse[(int64_t)(t.row0 + row) * a.n_q + head] =
          l == 0.f ? -__builtin_huge_valf() : (top + __log2f(l)) * 0.69314718055994531f;
  }
}

bool head_dim(int D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

int check_shape(int R, int q_max, int n_q, int n_kv, int D, int type) {
  if (R < 0 || q_max < 1 || n_kv < 1 || n_q < 1 || n_q % n_kv != 0 || D < 1) return SD_EINVAL;
  if (type != SD_CACHE_BF16 && type != SD_CACHE_FP4) return SD_EINVAL;
  if (!head_dim(D) || n_q > SD_MAX_HEADS) return SD_EUNSUPPORTED;
  if ((long long)R * q_max * (n_q / n_kv) > kMaxTokens) return SD_EUNSUPPORTED;
  return SD_OK;
}

bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }
bool off256(const void* p) { return ((uintptr_t)p & 255) != 0; }

}  // namespace

extern "C" size_t sd_attn_workspace_size(int R, int q_max, int n_q, int n_kv, int D) {
  if (check_shape(R, q_max, n_q, n_kv, D, SD_CACHE_BF16) != SD_OK) return 0;
  // tiles of 4 bits are as wide or narrower, and as many
  return attn_cut(R, q_max, n_q, n_kv, D, SD_CACHE_BF16, 1).bytes;
}

extern "C" int sd_attn_plan(hipStream_t stream, int R, int q_max, int n_q, int n_kv, int D, int cache_type,
                            int block_size, const int32_t* row0, const int32_t* ell, const int32_t* ctx_len, int causal, int window,
                            int32_t* status, void* workspace, size_t workspace_bytes) {
  const int rc = check_shape(R, q_max, n_q, n_kv, D, cache_type);
  if (rc != SD_OK) return rc;
  if (block_size < 1 || (causal != 0 && causal != 1) || window < 0) return SD_EINVAL;
  if (R == 0) return SD_OK;
  if (!row0 || !ell || !ctx_len || !status || !workspace || off256(workspace)) return SD_EINVAL;
  const Cut c = attn_cut(R, q_max, n_q, n_kv, D, cache_type, block_size);
  if (workspace_bytes < c.bytes) return SD_ERANGE;
  const Span written[] = {span(status, 4ll * R), span(workspace, (long long)c.bytes)};
  const Span read[] = {span(row0, 4ll * R), span(ell, 4ll * R), span(ctx_len, 4ll * R)};
  if (overlap(written, read)) return SD_EINVAL;
  char* ws = (char*)workspace;
  PlanArgs a = {};
  a.row0 = row0, a.ell = ell, a.ctx = ctx_len, a.status = status;
  a.head = (PlanHead*)ws, a.tiles = (Tile*)(ws + c.tiles), a.sums = (long long*)(ws + c.sums);
  a.starts = (Start*)(ws + c.starts), a.cuts = (CutTile*)(ws + c.cuts);
  a.shape = PlanShape{kPlanMark, R, q_max, n_q, n_kv, D, cache_type, block_size};
  a.causal = causal, a.window = window, a.M = c.M, a.TT = c.TT, a.W = c.W, a.group = n_q / n_kv;
  SDV_TRY_LAUNCH(launch(k_plan, dim3(1), dim3(kPlanThreads), 0, stream, a));
  return SD_OK;
}

extern "C" int sd_cache_attn(hipStream_t stream, int R, int q_max, int n_q, int n_kv, int D, int n_rows,
                             const uint16_t* q, long long ld_q, int cache_type, int block_size, int n_blocks,
                             const void* k_cache, const void* v_cache, const uint8_t* k_scale,
                             const uint8_t* v_scale, const int32_t* block_table, int max_blocks, float scale,
                             uint16_t* out, long long ld_out, float* lse, int32_t* status, void* workspace,
                             size_t workspace_bytes) {
  const int rc = check_shape(R, q_max, n_q, n_kv, D, cache_type);
  if (rc != SD_OK) return rc;
  if (n_rows < 0 || block_size < 1 || n_blocks < 0 || max_blocks < 0) return SD_EINVAL;
  if (!(scale > 0.0f && scale * kLog2e < __builtin_huge_valf())) return SD_EINVAL;
  if ((long long)block_size * max_blocks > kMaxTokens || (long long)n_blocks * block_size > (1ll << 40) ||
      (long long)n_kv * block_size > kMaxTokens)
    return SD_EUNSUPPORTED;
  if (R == 0 || n_rows == 0) return SD_OK;
  const long long width = (long long)n_q * D;
  if (!q || !out || !k_cache || !v_cache || !block_table || !status || !workspace || n_blocks < 1) return SD_EINVAL;
  if (cache_type == SD_CACHE_FP4 && (!k_scale || !v_scale || off16(k_scale) || off16(v_scale))) return SD_EINVAL;
  if (off16(q) || off16(out) || off16(k_cache) || off16(v_cache) || off256(workspace)) return SD_EINVAL;
  if (ld_q < width || ld_q % 8 != 0 || ld_out < width || ld_out % 8 != 0) return SD_EINVAL;
  const Cut c = attn_cut(R, q_max, n_q, n_kv, D, cache_type, block_size);
  if (workspace_bytes < c.bytes) return SD_ERANGE;
  const bool fp4 = cache_type == SD_CACHE_FP4;
  const long long tokens = (long long)n_blocks * block_size * n_kv;
  const long long side = fp4 ? tokens * (D / 2) : tokens * D * 2;
  const Span written[] = {span(out, n_rows, width * 2, ld_out * 2), span(lse, 4ll * n_rows * n_q), span(status, 4ll * R),
                          span(workspace, (long long)c.bytes)};
  const Span read[] = {span(q, n_rows, width * 2, ld_q * 2), span(k_cache, side), span(v_cache, side),
                       span(fp4 ? k_scale : nullptr, tokens * (D / 32)),
                       span(fp4 ? v_scale : nullptr, tokens * (D / 32)), span(block_table, 4ll * R * max_blocks)};
  if (overlap(written, read)) return SD_EINVAL;
  char* ws = (char*)workspace;
  AttnArgs a = {};
  a.q = q, a.out = out, a.lse = lse, a.ld_q = ld_q, a.ld_out = ld_out, a.table = block_table, a.status = status;
  a.cache = Cache{(void*)k_cache, (void*)v_cache, (uint8_t*)k_scale, (uint8_t*)v_scale, n_kv, block_size, n_blocks, 1.0 / block_size};
  a.shape = PlanShape{kPlanMark, R, q_max, n_q, n_kv, D, cache_type, block_size};
  a.max_blocks = max_blocks, a.n_rows = n_rows;
  a.head = (const PlanHead*)ws, a.tiles = (const Tile*)(ws + c.tiles), a.starts = (const Start*)(ws + c.starts);
  a.cuts = (const CutTile*)(ws + c.cuts);
  a.ml = (float2*)(ws + c.ml), a.part = (float*)(ws + c.part);
  a.scale2 = scale * kLog2e;
  // token * ceil(2^(31 + s) / bs) >> (31 + s), 2^s >= bs: exact below 2^31
  int s = 0;
  while ((1ll << s) < block_size) ++s;
  a.bs_mul = (uint32_t)(((1ull << (31 + s)) + block_size - 1) / block_size);
  a.bs_shift = 31 + s;
  a.group = n_q / n_kv, a.n_q = n_q, a.block_tokens = (uint32_t)(n_kv * block_size);
  const int span = attn_span(D, c.M, fp4);
  // Then streaming loads win: 128 contexts, one row each, 474 us, 528 with
  // cached ones; up to 12 rows each, 286 and 320 us.
  a.once = (long long)q_max * (n_q / n_kv) <= c.M;
  a.spans = span > 0 && block_size % span == 0;
  const int done = c.direct ? attend_direct(stream, c.M, c.W, a) : fp4 ? attend_fp4(stream, c.M, c.W, a) : attend_bf16(stream, c.M, c.W, a);
  if (done != SD_OK) return done;
#define SDV_JOIN(DD) \
  case DD: SDV_TRY_LAUNCH(launch(k_join<DD>, dim3(kJoinGrid), dim3(kJoinThreads), 0, stream, a, c.M)); return SD_OK;
  switch (D) {
    SDV_JOIN(64)
    SDV_JOIN(96)
    SDV_JOIN(128)
    SDV_JOIN(192)
    SDV_JOIN(256)
  }
#undef SDV_JOIN
  return SD_EUNSUPPORTED;
}
