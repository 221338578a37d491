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

struct PlanArgs {
  const int32_t* row0;
  const int32_t* ell;
  const int32_t* ctx;
  int32_t* status;
  PlanHead* head;
  Tile* tiles;
  long long* sums;
  Start* starts;
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
// where every run begins.
__global__ __launch_bounds__(kPlanThreads) void k_plan(PlanArgs a) {
  __shared__ long long part[kPlanThreads / 64];
  const int R = a.shape.R;
  long long n_tiles = 0, total;
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
      a.tiles[at + j] = t;
    }
  }
  __syncthreads();
  long long units = 0;
  for (long long i0 = 0; i0 < n_tiles; i0 += blockDim.x) {
    const long long i = i0 + threadIdx.x;
    const int n = i < n_tiles ? a.tiles[i].units : 0;
    const long long before = units + block_scan(n, part, &total);
    units += total;
    if (i < n_tiles) a.sums[i] = before;
  }
  const long long all = units * a.shape.n_kv;
  long long quota = (all + a.W - 1) / a.W;
  if (quota < kMinQuota) quota = kMinQuota;
  __syncthreads();
  for (int w = threadIdx.x; w <= a.W; w += blockDim.x) {
    const long long at = w * quota;
    Start s = {0, 0, 0};
    if (at < all) {
      s.head = (int)(at / units);
      const long long rest = at - s.head * units;
      long long lo = 0, hi = n_tiles;   // sums[lo] <= rest < sums[hi]
      while (hi - lo > 1) {
        const long long mid = (lo + hi) >> 1;
        if (a.sums[mid] <= rest) lo = mid;
        else hi = mid;
      }
      s.tile = (int)lo;
      s.off = (int)(rest - a.sums[lo]);
    }
    a.starts[w] = s;
  }
  if (threadIdx.x == 0) {
    PlanHead h = {};
    h.shape = a.shape;
    h.causal = a.causal;
    h.window = a.window;
    h.n_tiles = (int)n_tiles;
    h.per_head = units;
    h.total = all;
    h.quota = quota;
    *a.head = h;
  }
}

// Joins the parts of the tile that run w began and did not finish; D / 4
// threads to a query.
template <int D>
__global__ __launch_bounds__(256) void k_join(AttnArgs a, int M) {
  constexpr int TQ = D / 4, QB = 256 / TQ;
  const PlanHead& p = *a.head;
  if (!same_shape(p.shape, a.shape)) return;
  const int w = blockIdx.x, q = blockIdx.y * QB + threadIdx.x / TQ, d = threadIdx.x % TQ * 4;
  const long long quota = p.quota, end = (w + 1) * quota;
  if (end >= p.total) return;
  const Start s = a.starts[w + 1];
  if (s.off == 0 || s.off > quota) return;   // no tile is cut here, or a run before began it
  const Tile t = a.tiles[s.tile];
  if (!in_range(a, t)) return;
  const int qi = t.q0 + q;
  if (threadIdx.x >= QB * TQ || q >= M || qi >= t.queries) return;
  const int last = (int)((end - s.off + t.units - 1) / quota);   // the run that ends it
  auto slot = [&](int k) { return (int64_t)(k == w ? 2 * w + 1 : 2 * k) * M + q; };
  float top = -__builtin_huge_valf();
  for (int k = w; k <= last; ++k) top = fmaxf(top, a.ml[slot(k)].x);
  const float ref = top == -__builtin_huge_valf() ? 0.f : top;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = w; k <= last; ++k) {
    const float2 ml = a.ml[slot(k)];
    const float f = fast_exp2(ml.x - ref);
    const float4 v = *(const float4*)(a.part + slot(k) * D + d);
    l += ml.y * f;
    o.x += v.x * f, o.y += v.y * f, o.z += v.z * f, o.w += v.w * f;
  }
  const int i = qi / a.group, head = s.head * a.group + qi - i * a.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *(uint2*)(a.out + (int64_t)(t.row0 + i) * a.ld_out + (int64_t)head * D + d) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (a.lse && d == 0)
    a.lse[(int64_t)(t.row0 + i) * a.n_q + head] =
        l == 0.f ? -__builtin_huge_valf() : (top + __log2f(l)) * 0.69314718055994531f;
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
  return attn_cut(R, q_max, n_q, n_kv, D).bytes;
}

extern "C" int sd_attn_plan(hipStream_t stream, int R, int q_max, int n_q, int n_kv, int D, int cache_type,
                            const int32_t* row0, const int32_t* ell, const int32_t* ctx_len, int causal, int window,
                            int32_t* status, void* workspace, size_t workspace_bytes) {
  const int rc = check_shape(R, q_max, n_q, n_kv, D, cache_type);
  if (rc != SD_OK) return rc;
  if ((causal != 0 && causal != 1) || window < 0) return SD_EINVAL;
  if (R == 0) return SD_OK;
  if (!row0 || !ell || !ctx_len || !status || !workspace || off256(workspace)) return SD_EINVAL;
  const Cut c = attn_cut(R, q_max, n_q, n_kv, D);
  if (workspace_bytes < c.bytes) return SD_ERANGE;
  const Span written[] = {span(status, 4ll * R), span(workspace, (long long)c.bytes)};
  const Span read[] = {span(row0, 4ll * R), span(ell, 4ll * R), span(ctx_len, 4ll * R)};
  if (overlap(written, read)) return SD_EINVAL;
  char* ws = (char*)workspace;
  PlanArgs a = {};
  a.row0 = row0, a.ell = ell, a.ctx = ctx_len, a.status = status;
  a.head = (PlanHead*)ws, a.tiles = (Tile*)(ws + c.tiles), a.sums = (long long*)(ws + c.sums);
  a.starts = (Start*)(ws + c.starts);
  a.shape = PlanShape{kPlanMark, R, q_max, n_q, n_kv, D, cache_type};
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
  if (!(scale > 0.0f && scale < __builtin_huge_valf())) return SD_EINVAL;
  if ((long long)block_size * max_blocks > kMaxTokens || (long long)n_blocks * block_size > (1ll << 40) ||
      (long long)n_kv * block_size > kMaxTokens)
    return SD_EUNSUPPORTED;
  if (R == 0 || n_rows == 0) return SD_OK;
  const long long width = (long long)n_q * D;
  if (!q || !out || !k_cache || !v_cache || !block_table || !status || !workspace || n_blocks < 1) return SD_EINVAL;
  if (cache_type == SD_CACHE_FP4 && (!k_scale || !v_scale)) return SD_EINVAL;
  if (off16(q) || off16(out) || off16(k_cache) || off16(v_cache) || off256(workspace)) return SD_EINVAL;
  if (ld_q < width || ld_q % 8 != 0 || ld_out < width || ld_out % 8 != 0) return SD_EINVAL;
  const Cut c = attn_cut(R, q_max, n_q, n_kv, D);
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
  a.cache = Cache{(void*)k_cache, (void*)v_cache, (uint8_t*)k_scale, (uint8_t*)v_scale, n_kv, block_size, n_blocks};
  a.shape = PlanShape{kPlanMark, R, q_max, n_q, n_kv, D, cache_type};
  a.max_blocks = max_blocks, a.n_rows = n_rows;
  a.head = (const PlanHead*)ws, a.tiles = (const Tile*)(ws + c.tiles), a.starts = (const Start*)(ws + c.starts);
  a.ml = (float2*)(ws + c.ml), a.part = (float*)(ws + c.part);
  a.scale2 = scale * kLog2e;
  // token * ceil(2^(31 + s) / bs) >> (31 + s), 2^s >= bs: exact below 2^31
  int s = 0;
  while ((1ll << s) < block_size) ++s;
  a.bs_mul = (uint32_t)(((1ull << (31 + s)) + block_size - 1) / block_size);
  a.bs_shift = 31 + s;
  a.group = n_q / n_kv, a.n_q = n_q, a.block_tokens = (uint32_t)(n_kv * block_size);
  const int done = fp4 ? attend_fp4(stream, c.M, c.W, a) : attend_bf16(stream, c.M, c.W, a);
  if (done != SD_OK) return done;
#define SDV_JOIN(DD)                                                                                   \
  case DD: {                                                                                           \
    constexpr int kQueries = 256 / (DD / 4);                                                           \
    const dim3 grid((unsigned)c.W, (unsigned)((c.M + kQueries - 1) / kQueries));                       \
    SDV_TRY_LAUNCH(launch(k_join<DD>, grid, dim3(256), 0, stream, a, c.M));                            \
    return SD_OK;                                                                                      \
  }
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
