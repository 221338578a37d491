// sd_slot_reserve and sd_slot_commit: the verify batch's rows and the paged
// cache's slots, before the target's pass and after verification.
//
// The scheduler fixes how many tokens of each request the target scores
// (DSpark summary, "2.2 hardware-aware prefix scheduler"); token slots are
// reserved for all of them and cut back afterwards to what was accepted
// (LightSpec article, system section).  Neither may wait for the host, so
// both steps are prefix sums over the requests on the device.
//
// They read and write some 60 bytes per request and 20 per row, so a verify
// batch is bound by its chain of dependent loads (count and lengths, scan,
// blocks, rows: 3.7 us for 4 requests), and long pieces of prompts by the
// rows' stores (640 k rows, 13 MB: 9 us).
#include "sdv_host.h"
#include "verify_common.h"

namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWaves = kScanThreads / 64;
constexpr int kFillThreads = 256;
// Up to these requests every workgroup repeats the scan and keeps it in LDS:
// one launch (512 requests with up to 17 rows: 6.0 us, 8.0 us in two launches;
// 4 requests: 3.7 and 4.3 us; commit 4.8 and 5.9 us, 2.8 and 3.7 us).
constexpr int kOneLaunchRequests = 1024;
constexpr int kOneLaunchGrid = 1024;      // (640 k rows: 9.0 us, 15.6 us with 256 workgroups)
constexpr int kCommitRequests = 4;        // per workgroup (512 requests: 5.9 us, 8: 6.5 us, 16: 6.8 us)
// Requests per thread of such a scan: 1 up to 256 requests, 2 up to 512, else
// 4, so that one pass covers them all (reserve, 1 / 2 / 4 per thread: 64
// requests 5.3 / 5.5 / 5.9 us, 512: 7.2 / 6.1 / 6.4 us, 1024: 7.1 / 5.7 / 5.2 us).

// As many waves as the requests fill, up to a workgroup.
unsigned scan_threads(int R) { return R >= kScanThreads ? kScanThreads : (unsigned)(R + 63) / 64 * 64; }

// Exclusive prefix sums over the workgroup of two counts below 2^31, one in
// each half of a word (their sums stay below 2^31: the halves do not mix);
// *total gets the sums.
SDV_DEV uint64_t block_scan(uint64_t v, uint64_t* part, uint64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  uint64_t s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t t = __shfl_up((unsigned long long)s, o, 64);
    if (lane >= o) s += t;
  }
  if (waves == 1) {
    *total = __shfl((unsigned long long)s, 63, 64);
    return s - v;
  }
  __syncthreads();   // part may still be read from the last call
  if (lane == 63) part[wave] = s;
  __syncthreads();
  uint64_t before = 0, sum = 0;
  for (int w = 0; w < waves; ++w) {
    const uint64_t p = part[w];
    if (w < wave) before += p;
    sum += p;
  }
  *total = sum;
  return before + s - v;
}
SDV_DEV uint64_t two(int hi, int lo) { return (uint64_t)(uint32_t)hi << 32 | (uint32_t)lo; }
SDV_DEV int hi_of(uint64_t v) { return (int)(v >> 32); }
SDV_DEV int lo_of(uint64_t v) { return (int)(uint32_t)v; }

// Blocks that hold n positions; n and bs below 2^31 - 256 as all positions are.
SDV_DEV int blocks_of(int n, int bs) { return (int)(((unsigned)n + (unsigned)bs - 1u) / (unsigned)bs); }

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
  int32_t* ws_base;    // [R] tokens in the cache
  int32_t* ws_cu;      // [R + 1]
  int R, q_max, bs, max_blocks, n_blocks, max_rows, padded, ld_tokens;
};

SDV_DEV void no_row(const ReserveArgs& a, int e) {
  a.row_req[e] = -1;
  a.row_pos[e] = -1;
  a.row_slot[e] = -1;
  if (a.row_token) a.row_token[e] = -1;
}

struct Reserved {
  int len;     // tokens in the cache
  int n;       // rows
  int row;     // rows of the requests before
  int first;   // index in the free list of the first new block, counting down
  int st;
};

// What each request gets, kItems requests per thread, whose loads are
// requested together.  Three quantities depend on the requests before: the
// rows that fit the buffers, the blocks that are left, and where the rows
// begin.  Each is a prefix sum; the last two are one while the blocks suffice.
// emit(r, Reserved) is called by one thread per request; every thread gets
// the totals.
template <int kItems, typename Emit>
SDV_DEV void reserve_scan(const ReserveArgs& a, uint64_t* part, int* rows, int* free_left, Emit emit) {
  const int64_t cap = (int64_t)a.bs * a.max_blocks;
  const int F = sdv::clampi(*a.free_count, 0, a.n_blocks);
  const bool may_cut = !a.padded && a.max_rows < a.R * a.q_max;   // rows may not fit the buffers
  int want_before = 0, need_before = 0, rows_before = 0;
  for (int t = 0; t < a.R; t += blockDim.x * kItems) {
    const int r0 = t + threadIdx.x * kItems;
    int64_t len[kItems];
    int asked[kItems], want[kItems], h0[kItems], need[kItems], n[kItems], st[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      len[k] = r0 + k < a.R ? a.seq_len[r0 + k] : 0;
      asked[k] = r0 + k < a.R ? a.ell[r0 + k] : -1;
    }
    int wants = 0, needs = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      asked[k] = max(min(asked[k], a.q_max - 1) + 1, 0);
      st[k] = 0;
      if (len[k] < 0 || len[k] > cap) {
        st[k] = SD_ST_BAD_INPUT;
        len[k] = 0;
        asked[k] = 0;
      }
      want[k] = (int)(asked[k] < cap - len[k] ? asked[k] : cap - len[k]);
      wants += want[k];
    }
    uint64_t total;
    if (may_cut) {
      int before = lo_of(block_scan(two(0, wants), part, &total)) + want_before;
      want_before += lo_of(total);
      wants = 0;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int wished = want[k];
        want[k] = sdv::clampi(a.max_rows - before, 0, wished);
        before += wished;
        wants += want[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      h0[k] = blocks_of((int)len[k], a.bs);
      need[k] = blocks_of((int)len[k] + want[k], a.bs) - h0[k];
      n[k] = want[k];
      needs += need[k];
    }
    const uint64_t pre = block_scan(two(needs, wants), part, &total);
    int spoken = hi_of(pre) + need_before, before = lo_of(pre);
    need_before += hi_of(total);
    if (need_before > F) {   // the blocks run out in this tile or did before
      int sum = 0, taken = spoken;
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        const int got = sdv::clampi(F - taken, 0, need[k]);
        const int64_t room = (int64_t)(h0[k] + got) * a.bs - len[k];
        n[k] = (int)(want[k] < room ? want[k] : room);
        taken += need[k];
        sum += n[k];
      }
      before = lo_of(block_scan(two(0, sum), part, &total));
    }
    before += rows_before;
    rows_before += lo_of(total);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (n[k] < asked[k]) st[k] |= SD_ST_NO_SLOT;
      if (r0 + k < a.R) emit(r0 + k, Reserved{(int)len[k], n[k], before, F - 1 - spoken, st[k]});
      before += n[k];
      spoken += need[k];
    }
  }
  *rows = rows_before;
  *free_left = F - min(F, need_before);
}

SDV_DEV void reserve_out(const ReserveArgs& a, int r, const Reserved& q) {
  a.ell_out[r] = q.n - 1;
  a.row0[r] = a.padded ? r * a.q_max : min(q.row, a.max_rows - 1);
  a.cu_rows[r] = q.row;
  a.ctx_len[r] = (q.st & SD_ST_BAD_INPUT) ? 0 : q.len + q.n;
}

// One row of a request: its position's slot and its token.
SDV_DEV void fill_row(const ReserveArgs& a, int e, int r, int i, int len, int first) {
  const int pos = len + i, b = (int)((unsigned)pos / (unsigned)a.bs), off = pos - b * a.bs;
  const int h0 = blocks_of(len, a.bs);
  const int block = b < h0 ? a.table[(int64_t)r * a.max_blocks + b] : a.free_list[first - (b - h0)];
  a.row_req[e] = r;
  a.row_pos[e] = pos;
  a.row_slot[e] = block >= 0 && block < a.n_blocks ? (int64_t)block * a.bs + off : -1;
  if (a.row_token) {
    const int32_t* t = a.tokens + (int64_t)r * a.ld_tokens;
    a.row_token[e] = a.x0 ? (i == 0 ? a.x0[r] : t[i - 1]) : t[i];
  }
}

// The new blocks of a request into its table, by one wave; true where one of
// the blocks of its rows is outside the pool.
SDV_DEV bool enter_blocks(const ReserveArgs& a, int r, int len, int n, int first) {
  const int lane = threadIdx.x & 63, h0 = blocks_of(len, a.bs);
  const int got = blocks_of(len + n, a.bs) - h0;
  int32_t* table = a.table + (int64_t)r * a.max_blocks + h0;
  bool bad = false;
  if (lane == 0 && n > 0 && len % a.bs != 0) {   // rows begin inside a block
    const int b = table[-1];
    bad = b < 0 || b >= a.n_blocks;
  }
  for (int k = lane; k < got; k += 64) {
    const int b = a.free_list[first - k];
    bad |= b < 0 || b >= a.n_blocks;
    table[k] = b;
  }
  return __ballot(bad) != 0;
}

// One launch: every workgroup repeats the scan (a few thousand words from
// cache, no second launch to wait for), then its waves take requests and its
// threads rows.  No output may be an input here unless the grid is one
// workgroup.
template <int kItems>
__global__ __launch_bounds__(kFillThreads) void k_reserve_all(ReserveArgs a) {
  __shared__ uint64_t part[kScanWaves];
  __shared__ int cu[kOneLaunchRequests + 1], len[kOneLaunchRequests], first[kOneLaunchRequests];
  __shared__ uint8_t st[kOneLaunchRequests];
  int rows, left;
  reserve_scan<kItems>(a, part, &rows, &left, [&](int r, const Reserved& q) {
    cu[r] = q.row;
    len[r] = q.len;
    first[r] = q.first;
    st[r] = (uint8_t)q.st;
  });
  if (threadIdx.x == 0) cu[a.R] = rows;
  __syncthreads();   // and free_count has been read by all
  const int waves = gridDim.x * (kFillThreads / 64);
  for (int r = blockIdx.x * (kFillThreads / 64) + (threadIdx.x >> 6); r < a.R; r += waves) {
    const Reserved q{len[r], cu[r + 1] - cu[r], cu[r], first[r], st[r]};
    const bool bad = enter_blocks(a, r, q.len, q.n, q.first);
    if ((threadIdx.x & 63) == 0) {
      reserve_out(a, r, q);
      a.status[r] = q.st | (bad ? SD_ST_BAD_INPUT : 0);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.cu_rows[a.R] = rows;
    *a.batch = rows;
    *a.free_out = left;
  }
  for (int64_t e64 = (int64_t)blockIdx.x * kFillThreads + threadIdx.x; e64 < a.max_rows;
       e64 += (int64_t)gridDim.x * kFillThreads) {
    const int e = (int)e64;
    int lo = 0, i;
    if (a.padded) {
      lo = e / a.q_max;
      i = e - lo * a.q_max;
      if (lo >= a.R || i >= cu[lo + 1] - cu[lo]) {
        no_row(a, e);
        continue;
      }
    } else {
      if (e >= rows) {
        no_row(a, e);
        continue;
      }
      int hi = a.R;   // cu[lo] <= e < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= e) lo = mid;
        else hi = mid;
      }
      i = e - cu[lo];
    }
    fill_row(a, e, lo, i, len[lo], first[lo]);
  }
}

// Two launches, for more requests or outputs in the place of inputs: the scan,
// then the rows.
template <int kItems>
__global__ __launch_bounds__(kScanThreads) void k_reserve_scan(ReserveArgs a) {
  __shared__ uint64_t part[kScanWaves];
  int rows, left;
  reserve_scan<kItems>(a, part, &rows, &left, [&](int r, const Reserved& q) {
    a.ws_first[r] = q.first;
    a.ws_base[r] = q.len;
    a.ws_cu[r] = q.row;
    reserve_out(a, r, q);
    a.status[r] = q.st;
  });
  __syncthreads();   // free_out may be free_count, which every thread has read now
  if (threadIdx.x == 0) {
    a.ws_cu[a.R] = rows;
    a.cu_rows[a.R] = rows;
    *a.batch = rows;
    *a.free_out = left;
  }
}

// One wave per request for its blocks, and one thread per row.
__global__ __launch_bounds__(kFillThreads) void k_reserve_rows(ReserveArgs a) {
  const int e = blockIdx.x * kFillThreads + threadIdx.x;
  const int w = e >> 6, waves = gridDim.x * (kFillThreads / 64);
  for (int r = w; r < a.R; r += waves) {
    const int row = a.ws_cu[r];
    if (enter_blocks(a, r, a.ws_base[r], a.ws_cu[r + 1] - row, a.ws_first[r]) && (e & 63) == 0)
      a.status[r] |= SD_ST_BAD_INPUT;
  }
  if (e >= a.max_rows) return;
  int r, i = 0;
  bool live;
  if (a.padded) {
    r = e / a.q_max;
    i = e - r * a.q_max;
    live = r < a.R && i < a.ws_cu[r + 1] - a.ws_cu[r];
  } else {   // the request whose rows hold e: ws_cu[r] <= e < ws_cu[r + 1]
    live = e < a.ws_cu[a.R];
    int lo = 0, hi = a.R;
    while (live && hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.ws_cu[mid] <= e) lo = mid;
      else hi = mid;
    }
    r = lo;
    if (live) i = e - a.ws_cu[r];
  }
  if (live) fill_row(a, e, r, i, a.ws_base[r], a.ws_first[r]);
  else no_row(a, e);
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

// Statuses whose step is repeated: rows that could not be verified, or that a
// call before verification left out.
constexpr int kHeld = SD_ST_NONFINITE | SD_ST_ZERO_Z | SD_ST_BAD_INPUT;

struct Committed {
  int64_t len;   // tokens that stay
  int n_new;
  int acc;
  int kept;      // blocks that stay
  int give;      // blocks that go back ...
  int to;        // ... and where in the free list
  bool bad;
};

// What becomes of each request, kItems per thread; emit(r, Committed) by one thread per request,
// every thread gets the new count.
template <int kItems, typename Emit>
SDV_DEV void commit_scan(const CommitArgs& a, uint64_t* part, int* free_out, Emit emit) {
  const int64_t cap = (int64_t)a.bs * a.max_blocks;
  const int F = sdv::clampi(*a.free_count, 0, a.n_blocks);
  int before_all = 0;
  for (int t = 0; t < a.R; t += blockDim.x * kItems) {
    const int r0 = t + threadIdx.x * kItems;
    Committed c[kItems];
    int64_t len[kItems];
    int L[kItems], st[kItems], acc[kItems], done[kItems], keep[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {   // all requested together
      const bool in = r0 + k < a.R;
      len[k] = in ? a.seq_len[r0 + k] : 0;
      L[k] = in ? a.ell[r0 + k] : -1;
      acc[k] = in ? a.n_acc[r0 + k] : 0;
      st[k] = in && a.status ? a.status[r0 + k] : 0;
      done[k] = in && a.release ? a.release[r0 + k] : 0;
      keep[k] = in && a.keep ? a.keep[r0 + k] : 0;
    }
    int gives = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int q = L[k] < 0 || L[k] >= a.q_max ? 0 : L[k] + 1;
      c[k] = Committed{len[k], 0, 0, 0, 0, 0, false};
      if (len[k] < 0 || len[k] > cap || L[k] >= a.q_max || len[k] + q > cap) {
        c[k].bad = true;
      } else {
        c[k].acc = sdv::clampi(acc[k], 0, q ? L[k] : 0);
        c[k].n_new = q && !(st[k] & kHeld) ? c[k].acc + 1 : 0;
        const int held = blocks_of((int)len[k] + q, a.bs);
        c[k].len = done[k] ? 0 : len[k] + c[k].n_new;
        c[k].kept = done[k] ? sdv::clampi(keep[k], 0, held) : blocks_of((int)c[k].len, a.bs);
        c[k].give = held - c[k].kept;
      }
      gives += c[k].give;
    }
    uint64_t total;
    int to = F + lo_of(block_scan(two(0, gives), part, &total)) + before_all;
    before_all += lo_of(total);
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      c[k].to = to;
      to += c[k].give;
      // more blocks than the pool has: the accounting was broken before
      if (c[k].give && to > a.n_blocks) c[k].bad = true;
      if (r0 + k < a.R) emit(r0 + k, c[k]);
    }
  }
  *free_out = (int)((int64_t)F + before_all < a.n_blocks ? F + before_all : a.n_blocks);
}

SDV_DEV void commit_out(const CommitArgs& a, int r, const Committed& c) {
  a.seq_out[r] = c.len;
  a.n_new[r] = c.n_new;
  if (a.x0_out) a.x0_out[r] = c.n_new ? a.out_tokens[(int64_t)r * a.q_max + c.acc] : a.x0[r];
  if (c.bad && a.status) a.status[r] |= SD_ST_BAD_INPUT;
}

// The blocks of a request back to the free list, by one wave.
SDV_DEV void give_back(const CommitArgs& a, int r, int kept, int give, int to) {
  const int32_t* table = a.table + (int64_t)r * a.max_blocks + kept;
  for (int i = threadIdx.x & 63; i < give; i += 64)
    if ((int64_t)to + i < a.n_blocks) a.free_list[to + i] = table[i];
}

// One launch: every workgroup repeats the scan and keeps the requests of its
// waves.  No output may be an input unless the grid is one workgroup, but for
// the status: a workgroup that already sees the bit that another one adds
// (commit_out) comes to the same result.  A request out of range is so with
// and without the bit.  One that gives back more than the pool holds (to +
// give > n_blocks) would give back more yet if it were held; those after it
// drop their blocks either way, for their `to` is past the pool in both, and
// the count is the pool's.  Its own outputs come from the one workgroup that
// writes its status, by the thread that has read it.
template <int kItems>
__global__ __launch_bounds__(kFillThreads) void k_commit_all(CommitArgs a) {
  __shared__ uint64_t part[kScanWaves];
  __shared__ int kept[kOneLaunchRequests], give[kOneLaunchRequests], to[kOneLaunchRequests];
  int left;
  commit_scan<kItems>(a, part, &left, [&](int r, const Committed& c) {
    kept[r] = c.kept;
    give[r] = c.give;
    to[r] = c.to;
    if (r % gridDim.x == blockIdx.x) commit_out(a, r, c);
  });
  __syncthreads();
  for (int r = blockIdx.x + (threadIdx.x >> 6) * gridDim.x; r < a.R; r += gridDim.x * (kFillThreads / 64))
    if (give[r]) give_back(a, r, kept[r], give[r], to[r]);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_out = left;
}

// Two launches, for more requests or outputs in the place of inputs.
template <int kItems>
__global__ __launch_bounds__(kScanThreads) void k_commit_scan(CommitArgs a) {
  __shared__ uint64_t part[kScanWaves];
  int left;
  commit_scan<kItems>(a, part, &left, [&](int r, const Committed& c) {
    a.ws[3 * r] = c.kept;
    a.ws[3 * r + 1] = c.give;
    a.ws[3 * r + 2] = c.to;
    commit_out(a, r, c);
  });
  __syncthreads();   // free_out may be free_count, which every thread has read now
  if (threadIdx.x == 0) *a.free_out = left;
}

__global__ __launch_bounds__(kFillThreads) void k_commit_move(CommitArgs a) {
  const int r = blockIdx.x * (kFillThreads / 64) + (threadIdx.x >> 6);
  if (r < a.R) give_back(a, r, a.ws[3 * r], a.ws[3 * r + 1], a.ws[3 * r + 2]);
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
  if (padded ? max_rows < R * q_max : (R > 0 && max_rows < 1)) return SD_ERANGE;
  if (!free_count || !cu_rows || !batch || !free_left) return SD_EINVAL;
  if (max_rows > 0 && (!row_req || !row_pos || !row_slot)) return SD_EINVAL;
  if (R > 0 && (!seq_len || !ell || !block_table || (n_blocks > 0 && !free_list) || !ell_out || !row0 || !ctx_len ||
                !status))
    return SD_EINVAL;
  if (R > 0 && row_token && !tokens && !(x0 && q_max == 1)) return SD_EINVAL;
  if (R > 0 && row_token && ld_tokens < (x0 ? q_max - 1 : q_max)) return SD_ERANGE;
  if (!workspace || workspace_bytes < sd_slot_reserve_workspace_size(R)) return SD_ERANGE;
  if (((uintptr_t)workspace & 7) != 0) return SD_EINVAL;
  using sdv::span;
  const long long per = 4LL * R;   // bytes of an int32 per request
  const sdv::Span written[] = {
      span(block_table, per * max_blocks), span(ell_out, per), span(row0, per), span(cu_rows, per + 4),
      span(ctx_len, per), span(batch == cu_rows + R ? nullptr : batch, 4), span(free_left, 4), span(row_req, 4LL * max_rows),
      span(row_pos, 4LL * max_rows), span(row_slot, 8LL * max_rows), span(row_token, 4LL * max_rows),
      span(status, per), span(workspace, 3 * per + 4)};
  const sdv::Span read[] = {
      span(seq_len, 2 * per), span(ell == ell_out ? nullptr : ell, per), span(row_token ? x0 : nullptr, per),
      span(row_token ? tokens : nullptr, R, 4LL * (x0 ? q_max - 1 : q_max), 4LL * ld_tokens),
      span(free_list, 4LL * n_blocks), span(free_count == free_left ? nullptr : free_count, 4)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
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
  // a thread per row and, as far as the grid goes, a wave per request
  const int row_wgs = (max_rows + kFillThreads - 1) / kFillThreads, req_wgs = R < 16384 ? (R + 3) / 4 : 4096;
  const unsigned wgs = (unsigned)(row_wgs > req_wgs ? row_wgs : (req_wgs > 1 ? req_wgs : 1));
  // an output in an input's place (without requests only the count is read, and stays)
  const bool over = R > 0 && (ell_out == ell || free_left == free_count);
  if (R <= kOneLaunchRequests && (!over || wgs == 1)) {
    const auto k = R <= kFillThreads ? k_reserve_all<1> : (R <= 2 * kFillThreads ? k_reserve_all<2> : k_reserve_all<4>);
    SDV_TRY_LAUNCH(sdv::launch(k, dim3(wgs < kOneLaunchGrid ? wgs : kOneLaunchGrid), dim3(kFillThreads), 0, stream, a));
    return SD_OK;
  }
  SDV_TRY_LAUNCH(sdv::launch(R <= kScanThreads ? k_reserve_scan<1> : k_reserve_scan<4>, dim3(1),
                             dim3(scan_threads(R)), 0, stream, a));
  SDV_TRY_LAUNCH(sdv::launch(k_reserve_rows, dim3(wgs), dim3(kFillThreads), 0, stream, a));
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
  if ((long long)block_size * max_blocks > lim || (long long)R * max_blocks + n_blocks > lim ||
      (long long)R * q_max > lim)
    return SD_EUNSUPPORTED;
  if (!free_count || !free_count_out) return SD_EINVAL;
  if (R > 0 && (!seq_len || !ell || !n_accepted || !block_table || (n_blocks > 0 && !free_list) || !seq_len_out ||
                !n_new))
    return SD_EINVAL;
  if (R > 0 && x0_out && (!out_tokens || !x0)) return SD_EINVAL;
  if (!workspace || workspace_bytes < sd_slot_commit_workspace_size(R)) return SD_ERANGE;
  if (((uintptr_t)workspace & 7) != 0) return SD_EINVAL;
  using sdv::span;
  const long long per = 4LL * R;   // bytes of an int32 per request
  const sdv::Span written[] = {span(free_list, 4LL * n_blocks), span(status, per),  span(seq_len_out, 2 * per),
                               span(x0_out, per),               span(n_new, per),   span(free_count_out, 4),
                               span(workspace, 3 * per)};
  const sdv::Span read[] = {
      span(seq_len == seq_len_out ? nullptr : seq_len, 2 * per), span(ell, per), span(n_accepted, per),
      span(x0_out ? out_tokens : nullptr, per * q_max), span(x0_out && x0 != x0_out ? x0 : nullptr, per),
      span(release, per), span(keep, per), span(block_table, per * max_blocks),
      span(free_count == free_count_out ? nullptr : free_count, 4)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
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
  const unsigned wgs = R > 0 ? (unsigned)((R + kCommitRequests - 1) / kCommitRequests) : 1;
  const bool over = seq_len_out == seq_len || free_count_out == free_count || (x0_out && x0_out == x0);
  if (R <= kOneLaunchRequests && (!over || wgs == 1)) {
    const auto k = R <= kFillThreads ? k_commit_all<1> : (R <= 2 * kFillThreads ? k_commit_all<2> : k_commit_all<4>);
    SDV_TRY_LAUNCH(sdv::launch(k, dim3(wgs), dim3(kFillThreads), 0, stream, a));
    return SD_OK;
  }
  SDV_TRY_LAUNCH(sdv::launch(R <= kScanThreads ? k_commit_scan<1> : k_commit_scan<4>, dim3(1),
                             dim3(scan_threads(R)), 0, stream, a));
  SDV_TRY_LAUNCH(sdv::launch(k_commit_move, dim3((R + 3) / 4), dim3(kFillThreads), 0, stream, a));
  return SD_OK;
}
