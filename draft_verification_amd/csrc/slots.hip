// sd_slot_reserve and sd_slot_commit: the verify batch's rows and the paged
// cache's slots, before the target's pass and after verification.
//
// The scheduler fixes how many tokens of each request the target scores
// (DSpark summary, "2.2 hardware-aware prefix scheduler"); token slots are
// reserved for all of them and cut back afterwards to what was accepted
// (LightSpec article, system section).  Neither may wait for the host, so
// both steps are prefix sums over the requests on the device.
#include "sdv_host.h"
#include "verify_common.h"

namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWaves = kScanThreads / 64;
constexpr int kFillThreads = 256;

// Exclusive prefix sum over the workgroup; *total gets the sum.
SDV_DEV int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(s, o, 64);
    if (lane >= o) s += t;
  }
  __syncthreads();   // part may still be read from the last call
  if (lane == 63) part[wave] = s;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kScanWaves; ++w) {
    const int p = part[w];
    if (w < wave) before += p;
    sum += p;
  }
  *total = sum;
  return before + s - v;
}

SDV_DEV int blocks_of(int64_t n, int bs) { return (int)((n + bs - 1) / bs); }

struct ReserveArgs {
  const int64_t* seq_len;
  const int32_t* ell;
  const int32_t* free_list;
  const int32_t* free_count;
  const int32_t* x0;
  const int32_t* tokens;
  int32_t* table;
  int32_t* ell_out;
  int32_t* row0;
  int32_t* cu_rows;
  int32_t* ctx_len;
  int32_t* batch;
  int32_t* free_out;
  int32_t* row_req;
  int32_t* row_pos;
  int64_t* row_slot;
  int32_t* row_token;
  int32_t* status;
  int32_t* ws_first;   // [R] index in the free list of the request's first new block, counting down
  int32_t* ws_base;    // [R] tokens in the cache, or -1
  int32_t* ws_cu;      // [R + 1]
  int R, q_max, bs, max_blocks, n_blocks, max_rows, padded, ld_tokens;
};

__global__ __launch_bounds__(kScanThreads) void k_reserve_scan(ReserveArgs a) {
  __shared__ int part[kScanWaves];
  const int64_t cap = (int64_t)a.bs * a.max_blocks;
  const int F = sdv::clampi(*a.free_count, 0, a.n_blocks);
  int want_before = 0, need_before = 0, rows_before = 0, taken = 0;
  for (int t = 0; t < a.R; t += kScanThreads) {
    const int r = t + threadIdx.x;
    int64_t len = 0;
    int asked = 0, st = 0;
    if (r < a.R) {
      len = a.seq_len[r];
      asked = min(a.ell[r], a.q_max - 1) + 1;
      if (asked < 0) asked = 0;
      if (len < 0 || len > cap) {
        st = SD_ST_BAD_INPUT;
        len = 0;
        asked = 0;
      }
    }
    int want = (int)(asked < cap - len ? asked : cap - len);
    int total;
    int before = block_scan(want, part, &total) + want_before;
    want_before += total;
    if (!a.padded) want = sdv::clampi(a.max_rows - before, 0, want);
    const int h0 = blocks_of(len, a.bs);
    const int need = blocks_of(len + want, a.bs) - h0;
    before = block_scan(need, part, &total) + need_before;
    need_before += total;
    const int got = sdv::clampi(F - before, 0, need);
    const int64_t room = (int64_t)(h0 + got) * a.bs - len;
    const int n = (int)(want < room ? want : room);
    const int first = F - 1 - before;
    before = block_scan(n, part, &total) + rows_before;
    rows_before += total;
    block_scan(got, part, &total);
    taken += total;
    if (r < a.R) {
      if (n < asked) st |= SD_ST_NO_SLOT;
      const bool bad = (st & SD_ST_BAD_INPUT) != 0;
      a.ws_first[r] = first;
      a.ws_base[r] = (int32_t)len;
      a.ws_cu[r] = before;
      a.ell_out[r] = n - 1;
      a.row0[r] = a.padded ? r * a.q_max : min(before, a.max_rows - 1);
      a.cu_rows[r] = before;
      a.ctx_len[r] = bad ? 0 : (int32_t)(len + n);
      a.status[r] = st;
    }
  }
  if (threadIdx.x == 0) {
    a.ws_cu[a.R] = rows_before;
    a.cu_rows[a.R] = rows_before;
    *a.batch = rows_before;
    *a.free_out = F - taken;
  }
}

// One thread per row of the buffers: its request, position, slot and token;
// the first row of a new block also enters the block into the table.
__global__ __launch_bounds__(kFillThreads) void k_reserve_rows(ReserveArgs a) {
  const int e = blockIdx.x * kFillThreads + threadIdx.x;
  if (e >= a.max_rows) return;
  int r, i = 0;
  bool live;
  if (a.padded) {
    r = e / a.q_max;
    i = e - r * a.q_max;
    live = r < a.R && i < a.ws_cu[r + 1] - a.ws_cu[r];
  } else {   // the request whose rows hold e: ws_cu[r] <= e < ws_cu[r + 1]
    live = e < a.ws_cu[a.R];
    int lo = 0, hi = a.R;   // ws_cu[lo] <= e < ws_cu[hi]
    while (live && hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.ws_cu[mid] <= e) lo = mid;
      else hi = mid;
    }
    r = lo;
    if (live) i = e - a.ws_cu[r];
  }
  if (!live) {
    a.row_req[e] = -1;
    a.row_pos[e] = -1;
    a.row_slot[e] = -1;
    if (a.row_token) a.row_token[e] = -1;
    return;
  }
  const int len = a.ws_base[r], pos = len + i;
  const int b = pos / a.bs, off = pos - b * a.bs;
  const int h0 = (len + a.bs - 1) / a.bs;
  int block;
  if (b < h0) {
    block = a.table[(int64_t)r * a.max_blocks + b];
  } else {
    block = a.free_list[a.ws_first[r] - (b - h0)];
    if (off == 0) a.table[(int64_t)r * a.max_blocks + b] = block;
  }
  const bool good = block >= 0 && block < a.n_blocks;
  if (!good) atomicOr(&a.status[r], SD_ST_BAD_INPUT);
  a.row_req[e] = r;
  a.row_pos[e] = pos;
  a.row_slot[e] = good ? (int64_t)block * a.bs + off : -1;
  if (a.row_token) {
    const int32_t* t = a.tokens + (int64_t)r * a.ld_tokens;
    a.row_token[e] = a.x0 ? (i == 0 ? a.x0[r] : t[i - 1]) : t[i];
  }
}

struct CommitArgs {
  const int64_t* seq_len;
  const int32_t* ell;
  const int32_t* n_acc;
  const int32_t* out_tokens;
  const int32_t* x0;
  const int32_t* release;
  const int32_t* keep;
  const int32_t* table;
  int32_t* status;
  int32_t* free_list;
  const int32_t* free_count;
  int64_t* seq_out;
  int32_t* x0_out;
  int32_t* n_new;
  int32_t* free_out;
  int32_t* ws;   // [R][3]: first surplus block, how many, where they go
  int R, q_max, bs, max_blocks, n_blocks;
};

__global__ __launch_bounds__(kScanThreads) void k_commit_scan(CommitArgs a) {
  __shared__ int part[kScanWaves];
  const int64_t cap = (int64_t)a.bs * a.max_blocks;
  const int F = sdv::clampi(*a.free_count, 0, a.n_blocks);
  int before_all = 0;
  for (int t = 0; t < a.R; t += kScanThreads) {
    const int r = t + threadIdx.x;
    int kept = 0, give = 0;
    if (r < a.R) {
      const int64_t len = a.seq_len[r];
      const int L = a.ell[r], st = a.status ? a.status[r] : 0;
      const int q = L < 0 ? 0 : L + 1;
      int64_t len1 = len;
      int adv = 0, acc = 0;
      if (len < 0 || len > cap || L >= a.q_max || len + q > cap) {
        if (a.status) a.status[r] = st | SD_ST_BAD_INPUT;
      } else {
        acc = sdv::clampi(a.n_acc[r], 0, q ? L : 0);
        adv = q && !(st & (SD_ST_NONFINITE | SD_ST_ZERO_Z)) ? acc + 1 : 0;
        const bool done = a.release && a.release[r];
        const int held = blocks_of(len + q, a.bs);
        len1 = done ? 0 : len + adv;
        kept = done ? sdv::clampi(a.keep ? a.keep[r] : 0, 0, held) : blocks_of(len1, a.bs);
        give = held - kept;
      }
      a.seq_out[r] = len1;
      a.n_new[r] = adv;
      if (a.x0_out) a.x0_out[r] = adv ? a.out_tokens[(int64_t)r * a.q_max + acc] : a.x0[r];
    }
    int total;
    const int before = block_scan(give, part, &total) + before_all;
    before_all += total;
    if (r < a.R) {
      // more blocks than the pool has: the accounting was broken before
      if (give && (int64_t)F + before + give > a.n_blocks && a.status) a.status[r] |= SD_ST_BAD_INPUT;
      a.ws[3 * r] = kept;
      a.ws[3 * r + 1] = give;
      a.ws[3 * r + 2] = F + before;
    }
  }
  if (threadIdx.x == 0) *a.free_out = (int)((int64_t)F + before_all < a.n_blocks ? F + before_all : a.n_blocks);
}

__global__ __launch_bounds__(kFillThreads) void k_commit_move(CommitArgs a) {
  const int r = blockIdx.x;
  const int kept = a.ws[3 * r], give = a.ws[3 * r + 1], to = a.ws[3 * r + 2];
  for (int i = threadIdx.x; i < give; i += kFillThreads)
    if ((int64_t)to + i < a.n_blocks) a.free_list[to + i] = a.table[(int64_t)r * a.max_blocks + kept + i];
}

}  // namespace

extern "C" size_t sd_slot_reserve_workspace_size(int R) {
  return R < 0 ? 0 : sdv_align256((size_t)(3 * (size_t)R + 1) * sizeof(int32_t));
}

extern "C" int sd_slot_reserve(hipStream_t stream, int R, int q_max, int block_size, int max_blocks,
                               int n_blocks, int max_rows, int padded, const int64_t* seq_len,
                               const int32_t* ell, const int32_t* x0, const int32_t* tokens, int ld_tokens,
                               int32_t* block_table, const int32_t* free_list, const int32_t* free_count,
                               int32_t* ell_out, int32_t* row0, int32_t* cu_rows, int32_t* ctx_len,
                               int32_t* batch, int32_t* free_left, int32_t* row_req, int32_t* row_pos,
                               int64_t* row_slot, int32_t* row_token, int32_t* status, void* workspace,
                               size_t workspace_bytes) {
  if (R < 0 || q_max < 1 || block_size < 1 || max_blocks < 1 || n_blocks < 0 || max_rows < 0) return SD_EINVAL;
  if (padded != 0 && padded != 1) return SD_EINVAL;
  const long long lim = 0x7FFFFFFFLL - kFillThreads;
  if ((long long)block_size * max_blocks > lim || (long long)R * q_max > lim || (long long)R * max_blocks > lim ||
      max_rows > lim)
    return SD_EUNSUPPORTED;
  if (R == 0) return SD_OK;
  if (padded ? max_rows < R * q_max : max_rows < 1) return SD_ERANGE;
  if (!seq_len || !ell || !block_table || (n_blocks > 0 && !free_list) || !free_count || !ell_out || !row0 || !cu_rows ||
      !ctx_len || !batch || !free_left || !row_req || !row_pos || !row_slot || !status)
    return SD_EINVAL;
  if (row_token && !tokens && !(x0 && q_max == 1)) return SD_EINVAL;
  if (row_token && ld_tokens < (x0 ? q_max - 1 : q_max)) return SD_ERANGE;
  if (!workspace || workspace_bytes < sd_slot_reserve_workspace_size(R)) return SD_ERANGE;
  if (((uintptr_t)workspace & 7) != 0) return SD_EINVAL;
  ReserveArgs a;
  a.seq_len = seq_len;
  a.ell = ell;
  a.free_list = free_list;
  a.free_count = free_count;
  a.x0 = x0;
  a.tokens = tokens;
  a.table = block_table;
  a.ell_out = ell_out;
  a.row0 = row0;
  a.cu_rows = cu_rows;
  a.ctx_len = ctx_len;
  a.batch = batch;
  a.free_out = free_left;
  a.row_req = row_req;
  a.row_pos = row_pos;
  a.row_slot = row_slot;
  a.row_token = row_token;
  a.status = status;
  a.ws_first = (int32_t*)workspace;
  a.ws_base = a.ws_first + R;
  a.ws_cu = a.ws_base + R;
  a.R = R;
  a.q_max = q_max;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.n_blocks = n_blocks;
  a.max_rows = max_rows;
  a.padded = padded;
  a.ld_tokens = ld_tokens;
  SDV_TRY_LAUNCH(sdv::launch(k_reserve_scan, dim3(1), dim3(kScanThreads), 0, stream, a));
  SDV_TRY_LAUNCH(sdv::launch(k_reserve_rows, dim3((max_rows + kFillThreads - 1) / kFillThreads),
                             dim3(kFillThreads), 0, stream, a));
  return SD_OK;
}

extern "C" size_t sd_slot_commit_workspace_size(int R) {
  return R < 0 ? 0 : sdv_align256(3 * (size_t)R * sizeof(int32_t));
}

extern "C" int sd_slot_commit(hipStream_t stream, int R, int q_max, int block_size, int max_blocks,
                              int n_blocks, const int64_t* seq_len, const int32_t* ell,
                              const int32_t* n_accepted, const int32_t* out_tokens, const int32_t* x0,
                              const int32_t* release, const int32_t* keep, const int32_t* block_table,
                              int32_t* free_list, const int32_t* free_count, int32_t* status,
                              int64_t* seq_len_out, int32_t* x0_out, int32_t* n_new, int32_t* free_count_out,
                              void* workspace, size_t workspace_bytes) {
  if (R < 0 || q_max < 1 || block_size < 1 || max_blocks < 1 || n_blocks < 0) return SD_EINVAL;
  const long long lim = 0x7FFFFFFFLL - kFillThreads;
  if ((long long)block_size * max_blocks > lim || (long long)R * max_blocks > lim || (long long)R * q_max > lim)
    return SD_EUNSUPPORTED;
  if ((long long)R * kFillThreads > 0xFFFFFFFFLL) return SD_EUNSUPPORTED;  // work-items of one launch
  if (R == 0) return SD_OK;
  if (!seq_len || !ell || !n_accepted || !block_table || (n_blocks > 0 && !free_list) || !free_count ||
      !seq_len_out || !n_new || !free_count_out)
    return SD_EINVAL;
  if (x0_out && (!out_tokens || !x0)) return SD_EINVAL;
  if (!workspace || workspace_bytes < sd_slot_commit_workspace_size(R)) return SD_ERANGE;
  if (((uintptr_t)workspace & 7) != 0) return SD_EINVAL;
  CommitArgs a;
  a.seq_len = seq_len;
  a.ell = ell;
  a.n_acc = n_accepted;
  a.out_tokens = out_tokens;
  a.x0 = x0;
  a.release = release;
  a.keep = keep;
  a.table = block_table;
  a.status = status;
  a.free_list = free_list;
  a.free_count = free_count;
  a.seq_out = seq_len_out;
  a.x0_out = x0_out;
  a.n_new = n_new;
  a.free_out = free_count_out;
  a.ws = (int32_t*)workspace;
  a.R = R;
  a.q_max = q_max;
  a.bs = block_size;
  a.max_blocks = max_blocks;
  a.n_blocks = n_blocks;
  SDV_TRY_LAUNCH(sdv::launch(k_commit_scan, dim3(1), dim3(kScanThreads), 0, stream, a));
  SDV_TRY_LAUNCH(sdv::launch(k_commit_move, dim3(R), dim3(kFillThreads), 0, stream, a));
  return SD_OK;
}
