// sd_logit_shape and sd_token_counts: the target rows of a verification step
// with the request's penalties, biases and grammar masks applied, and the
// token counts behind the penalties.
//
// Verification is lossless with respect to the target rows it is given
// (speculative-decoding history page, "1.1 mechanism"), so everything a
// request asks of the target's distribution has to be in those rows before
// sd_verify reads them.  Row i of a request scores the token after the drafts
// x_1..x_i, so those drafts count as written there, although they are not in
// the request's state until they are accepted.
#include "sdv_host.h"
#include "verify_common.h"

namespace {

constexpr int kShapeThreads = 64;
constexpr int kVecTokens = 8;                              // tokens per thread: one mask byte
constexpr int kShapeChunk = kShapeThreads * kVecTokens;    // tokens per workgroup
// A batch with fewer (request, chunk) waves, two rounds of what the chip holds
// at this kernel's registers, splits its rows over more (64 requests with 9
// rows, V = 32000: 13.1 us in 3 groups, 17.2 us unsplit, 13.9 us in 5; 4
// requests with 5 rows, V = 1000: 3.8 and 7.5 us; 16 requests with 9 rows, V =
// 151936: 12.4 us, 16.5 us with half as many waves).  One that fills the chip
// anyway gains 1 % at most by a split and is left whole: its state is read once.
constexpr long long kFullWaves = 16384;
// Beyond this the rows do not stay in the 256 MB last-level cache: they are
// streamed past it and wait for their masks (512 requests, V = 151936: 426 us
// streamed, 560 us not; 64 requests, V = 32000: 14.5 and 13.1 us).
constexpr double kCacheBytes = 128 << 20;
constexpr int kWholeLanes = 32;   // (grammars in place: 63 us, 71 us vector by vector; penalties: 227 and 223 us)

struct ShapeArgs {
  const char* logits;
  char* out;
  const int32_t* row0;
  const int32_t* ell;
  const int32_t* draft;
  const float* rep;
  const float* freq;
  const float* pres;
  const uint32_t* seen;
  const int32_t* counts;
  const int32_t* slot;
  const int64_t* bias_off;
  const int32_t* bias_tok;
  const float* bias_val;
  const uint32_t* mask;
  const int32_t* mask_row0;
  int32_t* status;
  int64_t n_bias;
  int64_t ld_bytes;
  int gmax, V, n_ch, n_rows, n_slots, ld_seen, ld_counts, ld_mask, n_mask_rows;
  int group;   // rows of a request per workgroup
};

// Eight consecutive logits as they lie in memory; a value is changed in its
// place, so the others keep their bits.
template <bool BF16>
struct Oct;
template <>
struct Oct<true> {
  static constexpr int kBytes = 16;
  uint4 q;
  template <bool NT>
  SDV_DEV void load(const char* p) { q = NT ? sdv::ld_nt(p) : *(const uint4*)p; }
  template <bool NT>
  SDV_DEV void store(char* p) const {
    if (NT) sdv::st_nt(p, q);
    else *(uint4*)p = q;
  }
  SDV_DEV uint32_t& word(int k) { return k == 0 ? q.x : (k == 1 ? q.y : (k == 2 ? q.z : q.w)); }
  SDV_DEV float get(int e) { return e & 1 ? sdv::bf16hi(word(e >> 1)) : sdv::bf16lo(word(e >> 1)); }
  SDV_DEV void set(int e, float x) {
    const uint32_t h = __builtin_bit_cast(uint16_t, (__bf16)x);   // nearest-even in one instruction
    uint32_t& w = word(e >> 1);
    w = e & 1 ? (w & 0xFFFFu) | (h << 16) : (w & 0xFFFF0000u) | h;
  }
  // -inf wherever the bit of `allowed` is 0
  SDV_DEV void keep(unsigned allowed) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned two = allowed >> (2 * k);
      const uint32_t m = ((two & 1u) ? 0xFFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
      uint32_t& w = word(k);
      w = (w & m) | (0xFF80FF80u & ~m);
    }
  }
};
template <>
struct Oct<false> {
  static constexpr int kBytes = 32;
  uint4 q[2];
  template <bool NT>
  SDV_DEV void load(const char* p) {
    q[0] = NT ? sdv::ld_nt(p) : ((const uint4*)p)[0];
    q[1] = NT ? sdv::ld_nt(p + 16) : ((const uint4*)p)[1];
  }
  template <bool NT>
  SDV_DEV void store(char* p) const {
    if (NT) {
      sdv::st_nt(p, q[0]);
      sdv::st_nt(p + 16, q[1]);
    } else {
      ((uint4*)p)[0] = q[0];
      ((uint4*)p)[1] = q[1];
    }
  }
  SDV_DEV uint32_t& word(int e) {
    uint4& v = q[e >> 2];
    return (e & 3) == 0 ? v.x : ((e & 3) == 1 ? v.y : ((e & 3) == 2 ? v.z : v.w));
  }
  SDV_DEV float get(int e) { return __uint_as_float(word(e)); }
  SDV_DEV void set(int e, float x) { word(e) = __float_as_uint(x); }
  SDV_DEV void keep(unsigned allowed) {
#pragma unroll
    for (int e = 0; e < 8; ++e) word(e) = (allowed >> e) & 1u ? word(e) : 0xFF800000u;
  }
};

// What a request asks for, and whether its device-side arguments are in range.
struct Request {
  int n;       // rows
  int row0, srow, m0;
  int64_t b0, b1;
  float rep, freq, pres;
  bool pen, ok;
};
SDV_DEV Request read_request(const ShapeArgs& a, int r) {
  Request q;   // requested together
  q.n = min(a.ell[r], a.gmax) + 1;
  q.row0 = a.row0[r];
  q.rep = a.rep ? a.rep[r] : 1.0f;
  q.freq = a.freq ? a.freq[r] : 0.0f;
  q.pres = a.pres ? a.pres[r] : 0.0f;
  q.srow = a.slot ? a.slot[r] : r;
  q.m0 = a.mask_row0 ? a.mask_row0[r] : -1;
  q.b0 = a.bias_off ? a.bias_off[r] : 0;
  q.b1 = a.bias_off ? a.bias_off[r + 1] : 0;
  const float inf = __builtin_huge_valf();
  q.pen = q.rep != 1.0f || q.freq != 0.0f || q.pres != 0.0f;
  q.ok = q.row0 >= 0 && (int64_t)q.row0 + q.n <= a.n_rows;
  q.ok = q.ok && q.rep > 0.0f && q.rep < inf && fabsf(q.freq) < inf && fabsf(q.pres) < inf;
  q.ok = q.ok && (!q.pen || (q.srow >= 0 && q.srow < a.n_slots));
  q.ok = q.ok && (q.m0 < 0 || (int64_t)q.m0 + q.n <= a.n_mask_rows);
  q.ok = q.ok && q.b0 >= 0 && q.b0 <= q.b1 && q.b1 <= a.n_bias;
  return q;
}

// What a lane holds for its eight tokens v0..v0+7.
struct Tokens {
  unsigned seen = 0;               // by the state, then by the drafts so far
  float c[kVecTokens] = {};        // written how often; up to 2^24 exact
  unsigned biased = 0;
  float bias[kVecTokens] = {};

  SDV_DEV void read_counts(const ShapeArgs& a, int srow, int v0) {
    if (!seen || !a.counts) return;
    const int4* p = (const int4*)(a.counts + (int64_t)srow * a.ld_counts + v0);
    const int4 p0 = p[0], p1 = p[1];
    const int k[kVecTokens] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int e = 0; e < kVecTokens; ++e) c[e] = (seen >> e) & 1 ? (float)k[e] : 0.0f;
  }
  SDV_DEV void write(int t, int v0) {   // token t counts as written
#pragma unroll
    for (int e = 0; e < kVecTokens; ++e)
      if (t == v0 + e) {
        c[e] += 1.0f;
        seen |= 1u << e;
      }
  }
  // The terms of the tokens in `hit`, of which those in `met` are seen.
  template <typename O>
  SDV_DEV void apply(const Request& q, unsigned hit, unsigned met, O& x) const {
#pragma unroll
    for (int e = 0; e < kVecTokens; ++e)
      if ((hit >> e) & 1) {
        float y = x.get(e);
        if ((met >> e) & 1) {
          // (the division as it is: a reciprocal and one step of correction, which
          // needs cases of its own where they underflow, took 13.3 us where
          // this takes 13.1, for 64 requests at V = 32000)
          y = y > 0.0f ? y / q.rep : y * q.rep;
          y = fmaf(-q.freq, c[e], y) - (c[e] > 0.0f ? q.pres : 0.0f);
        }
        if ((biased >> e) & 1) y += bias[e];
        x.set(e, y);
      }
  }
};

// The request's status: a draft or a bias entry outside the vocabulary.
SDV_DEV void report(const ShapeArgs& a, int r, const int32_t* drafts, int n, int bad) {
  const int lane = threadIdx.x;
  if (drafts)
    for (int i = lane; i < n - 1; i += kShapeThreads) bad |= drafts[i] < 0 || drafts[i] >= a.V;
  const bool any = __ballot(bad != 0) != 0;
  if (lane == 0) a.status[r] = any ? SD_ST_BAD_TOKEN : 0;
}

// l -> the row's logit with the request's terms (see read_request, Tokens):
// elementwise, so bound by the bytes of the rows.  One wave per (request,
// chunk of 512 tokens, group of rows); a lane owns eight consecutive tokens
// (16 bytes of bf16, one byte of a bitmap) in every row of the group, so the
// request's state is read once and stays in registers while the rows stream
// past, and no other lane's data is needed: workgroups of one wave were
// fastest (448 us, 455 us with two and 481 us with four waves).  NT: a batch
// that does not fit the last-level cache.
// Measured: 512 requests with up to 17 rows each, V = 151936 bf16, out of
// place, every term: 426 us for 2.46 GB of memory traffic, 5.8 TB/s (a copy of
// 2 GiB with streaming accesses reaches 6.5, torch's 4.9); grammars in place,
// 128 requests, V = 129280: 56-63 us by the share of masked rows, 0.30 GB,
// 4.7 TB/s (partial lines); penalties alone, 512 requests with histories of up
// to 1500 tokens: 227 us in place, 0.36 GB (single 16-byte pieces of lines),
// 518 us out of place; fp32 out of place, 256 requests, penalties: 642 us, 3.2
// GB, 4.9 TB/s.
template <bool BF16, bool NT, bool COPY>
__global__ __launch_bounds__(kShapeThreads) void k_logit_shape(ShapeArgs a) {
  // rows whose loads are issued together (large batch out of place: 1: 440 us,
  // 2: 426 us, 4: 422 us with more registers; grammars in place 1: 66 us, 2: 67
  // us, 4: 63 us; 64 requests at V = 32000 1: 13.1 us, 2: 14.1 us)
  constexpr int kRows = NT ? (COPY ? 2 : 4) : 1;
  __shared__ int last[kShapeChunk];   // 1 + index of a token's last bias entry
  const int r = blockIdx.x / a.n_ch, ch = blockIdx.x % a.n_ch;
  const int tid = threadIdx.x;
  const Request q = read_request(a, r);
  const int n = q.n, row0 = q.row0, m0 = q.m0;
  const int i0 = blockIdx.y * a.group, i1 = min(n, i0 + a.group);
  const bool tell = ch == 0 && i0 == 0;      // this wave reports the request's status
  if (i0 >= i1) {
    if (tell && tid == 0) a.status[r] = 0;
    return;
  }
  if (!q.ok) {   // uniform over the request's waves: none of its rows is written
    if (tell && tid == 0) a.status[r] = SD_ST_BAD_INPUT;
    return;
  }

  const int v0 = ch * kShapeChunk + tid * kVecTokens;
  const bool mine = v0 < a.V;
  const int m_all = mine ? i1 - i0 : 0;   // rows of this lane
  const char* src = a.logits + ((int64_t)row0 + i0) * a.ld_bytes + (int64_t)v0 * (Oct<BF16>::kBytes / kVecTokens);
  char* dst = a.out + (src - a.logits);
  const int64_t mask_step = (int64_t)a.ld_mask * 4;
  const uint8_t* mask =
      m0 >= 0 ? (const uint8_t*)(a.mask + ((int64_t)m0 + i0) * a.ld_mask) + (v0 >> 3) : nullptr;
  unsigned allowed[kRows];
  Oct<BF16> x[kRows];
  // A large batch is bound by bytes: a row's logits wait for its mask, and
  // what is neither read nor kept is not loaded.  A small one is bound by the
  // chain of loads: the first rows are requested here, with the state.
  auto fetch_mask = [&](int i) {
#pragma unroll
    for (int k = 0; k < kRows; ++k) allowed[k] = mask && i + k < m_all ? mask[(i + k) * mask_step] : 0xFFu;
  };
  auto fetch_all = [&](int i) {
#pragma unroll
    for (int k = 0; k < kRows; ++k)
      if (i + k < m_all) x[k].template load<NT>(src + (i + k) * a.ld_bytes);
  };
  if (!NT) {
    fetch_mask(0);
    fetch_all(0);
  }
  Tokens tk;
  if (q.pen && mine) tk.seen = ((const uint8_t*)(a.seen + (int64_t)q.srow * a.ld_seen))[v0 >> 3];

  // a draft before the row counts as written; most chunks hold none of them
  const int32_t* const drafts = q.pen && a.draft ? a.draft + (int64_t)r * a.gmax : nullptr;
  bool here = false;
  if (drafts)
    for (int i = tid; i < i1 - 1; i += kShapeThreads) here |= (unsigned)drafts[i] / kShapeChunk == (unsigned)ch;
  const int32_t* const draft = __ballot(here) ? drafts : nullptr;

  int bad = 0;
  if (q.b1 > q.b0) {
#pragma unroll
    for (int e = 0; e < kVecTokens; ++e) last[e * kShapeThreads + tid] = 0;
    __syncthreads();
    const int nb = (int)(q.b1 - q.b0);
    for (int i = tid; i < nb; i += kShapeThreads) {
      const int t = a.bias_tok[q.b0 + i];
      if (t < 0 || t >= a.V) bad = 1;
      else if (t / kShapeChunk == ch) atomicMax(&last[t % kShapeChunk], i + 1);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kVecTokens; ++e) {
      const int i = last[tid * kVecTokens + e];
      if (i > 0) {
        tk.bias[e] = a.bias_val[q.b0 + i - 1];
        tk.biased |= 1u << e;
      }
    }
  }
  // in place, most chunks of a request without a mask hold nothing to change
  if (!COPY && !mask && !draft && !tell && !__ballot(tk.seen | tk.biased)) return;
  tk.read_counts(a, q.srow, v0);
  if (draft)
    for (int i = 0; i < i0; ++i) tk.write(draft[i], v0);

  for (int i = 0; i < m_all; i += kRows) {
    if (NT) fetch_mask(i);
    // the tokens met before each row; the draft before it is new in it
    unsigned met[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      met[k] = k ? met[k - 1] : tk.seen;
      if (draft && i + k > 0 && i + k < m_all) {
        const int t = draft[i0 + i + k - 1];
        if ((t >> 3) == (v0 >> 3)) met[k] |= 1u << (t & 7);
      }
    }
    // In place a wave writes its whole 1 KB of a row back once many lanes are
    // touched: full lines, where single vectors would be merged in memory.
    unsigned touched[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      touched[k] = met[k] | tk.biased | (allowed[k] ^ 0xFFu);
      if (!COPY && __popcll(__ballot(touched[k] != 0)) >= kWholeLanes) touched[k] = 1;
    }
    if (NT) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (i + k < m_all && allowed[k] != 0 && (COPY || touched[k]))
          x[k].template load<NT>(src + (i + k) * a.ld_bytes);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (i + k >= m_all) break;
      if (draft && i + k > 0 && met[k]) tk.write(draft[i0 + i + k - 1], v0);
      const unsigned hit = (met[k] | tk.biased) & allowed[k];
      if (hit) tk.apply(q, hit, met[k], x[k]);
      if (allowed[k] != 0xFFu) x[k].keep(allowed[k]);
      if (COPY || touched[k]) x[k].template store<NT>(dst + (i + k) * a.ld_bytes);
    }
    if (!NT) {
      fetch_mask(i + kRows);
      fetch_all(i + kRows);
    }
  }
  if (tell) report(a, r, drafts, n, bad);
}

// ---------------------------------------------------------------------------
// Token counts.

struct CountArgs {
  const int32_t* tokens;
  const int64_t* start;
  const int32_t* length;
  const int32_t* prompt_len;
  const int32_t* slot;
  const int32_t* reset;
  uint32_t* seen;
  int32_t* counts;
  int32_t* status;
  int64_t n_tokens;
  int R, V, width, n_slots, ld_seen, ld_counts;
  int chunk;   // tokens per workgroup of k_count_own
};

// The request's tokens and state row; false where they are out of range.
SDV_DEV bool count_row(const CountArgs& a, int r, int64_t* at, int* n, int* srow) {
  *at = a.start ? a.start[r] : (int64_t)r * a.width;
  *n = a.length ? a.length[r] : a.width;
  *srow = a.slot ? a.slot[r] : r;
  if (*n < 0) *n = 0;
  if ((!a.start || a.width > 0) && *n > a.width) return false;   // a list ends with its row
  return *srow >= 0 && *srow < a.n_slots && *at >= 0 && *at <= a.n_tokens && *n <= a.n_tokens - *at;
}

constexpr int kCountThreads = 256;

// Short lists (a step's accepted tokens) without a reset: atomics on the
// state, whose order does not matter to whole numbers.
__global__ __launch_bounds__(kCountThreads) void k_count_add(CountArgs a) {
  const int r = blockIdx.x;
  int64_t at;
  int n, srow;
  const bool ok = count_row(a, r, &at, &n, &srow);
  if (blockIdx.y == 0 && threadIdx.x == 0) a.status[r] = ok ? 0 : SD_ST_BAD_INPUT;
  if (!ok) return;
  const int prompt = a.prompt_len ? a.prompt_len[r] : 0;
  uint32_t* seen = a.seen + (int64_t)srow * a.ld_seen;
  int32_t* counts = a.counts ? a.counts + (int64_t)srow * a.ld_counts : nullptr;
  const int64_t step = (int64_t)gridDim.y * kCountThreads;
  for (int64_t i = blockIdx.y * kCountThreads + threadIdx.x; i < n; i += step) {
    const int t = a.tokens[at + i];
    if (t < 0 || t >= a.V) continue;
    atomicOr(&seen[t >> 5], 1u << (t & 31));
    if (counts && i >= prompt) atomicAdd(&counts[t], 1);
  }
}

// Resets of very many requests: the rows cleared first.
__global__ __launch_bounds__(kCountThreads) void k_count_clear(CountArgs a) {
  const int r = blockIdx.x;
  int64_t at;
  int n, srow;
  if (!count_row(a, r, &at, &n, &srow) || !a.reset[r]) return;
  const int first = blockIdx.y * kCountThreads + threadIdx.x, step = gridDim.y * kCountThreads;
  for (int w = first; w < (a.V + 31) / 32; w += step) a.seen[(int64_t)srow * a.ld_seen + w] = 0;
  if (a.counts)
    for (int v = first; v < a.V; v += step) a.counts[(int64_t)srow * a.ld_counts + v] = 0;
}

// With resets, where a state row is written whole, and for long lists one
// workgroup owns a range of the vocabulary in one state row: it counts in LDS
// the tokens of every list entered into that row, then writes the range once,
// coalesced (without a reset: adds to what the lists touch).  A word of LDS
// holds a token's count and, in its top bit, that it was seen.  Every range
// reads the whole list; long lists are bound by the instructions of that
// filter (and wait for the ranges of the longest), short ones by the writing.
// Measured at V = 151936: 96 lists of up to 131072 tokens 26 us (252 us with a
// clearing pass and atomics on the state, 1.8 ms where half of a list is one
// token, here 34 us); one list of 131072 tokens 14.6 us; 256 lists of at most
// 100 tokens 32 us, 5.0 TB/s.  A call that has `reset` pays for the ranges also
// where no request resets (512 lists of up to 17 tokens: 51 us, 2.4 us added by
// atomics without it).
constexpr int kOwnThreads = 1024;
constexpr int kOwnLoads = 16;            // 4: 30 us, 8: 27 us for the 96 lists
constexpr int kOwnMaxChunk = 32768;      // 128 KB of the 160 KB of LDS
// Lists below this mean length are entered in half as large ranges, two
// workgroups per CU (256 short lists: 32 against 39 us; the 96 long ones
// above: 28 against 27 us).
constexpr int kOwnLongList = 8192;
// Without a reset, from this mean length on (64 lists of 4096 tokens: atomics
// 24 us, ranges 16 us; of 512 tokens: 4.7 and 11 us; one list of 131072: 272
// and 16.6 us).
constexpr int kOwnMinList = 4096;
// The search for shared state rows grows with the square of the requests
// (8192 requests at V = 4000: 71 us, 38 us cleared first and added to).
constexpr int kOwnMaxRequests = 4096;
constexpr uint32_t kSeenBit = 0x80000000u;

// Enter n tokens into the workgroup's range: MARK sets the seen bit, else the
// count grows.  `spare` are 64 more words for the tokens of other ranges, one
// per lane, so that the common path has no branch.
template <bool MARK>
SDV_DEV void enter_tokens(uint32_t* cell, uint32_t* spare, const int32_t* tokens, int n, int v0, int width) {
  const int tid = threadIdx.x, lane = tid & 63;
  auto add = [&](uint32_t* at, uint32_t k) {
    if (MARK) atomicOr(at, kSeenBit);
    else atomicAdd(at, k);
  };
  auto one = [&](int tok) {
    const unsigned t = (unsigned)tok - (unsigned)v0;   // a negative token is past every range
    add(t < (unsigned)width ? cell + t : spare + lane, 1u);
  };
  // a wave takes kOwnLoads * 64 tokens in a row at a time, requested together:
  // a list is one chain of loads otherwise
  const int wave0 = (tid >> 6) * (kOwnLoads * 64) + lane;
  const int full = n - n % (kOwnLoads * kOwnThreads);
  for (int i = 0; i < full; i += kOwnLoads * kOwnThreads) {
    int tok[kOwnLoads];
#pragma unroll
    for (int k = 0; k < kOwnLoads; ++k) tok[k] = tokens[i + wave0 + k * 64];
    // a stretch of one token would queue the wave's lanes at one word
    const int tok0 = __builtin_amdgcn_readfirstlane(tok[0]);
    if (__ballot(tok[0] == tok0) == ~0ull) {
#pragma unroll
      for (int k = 0; k < kOwnLoads; ++k) {
        const unsigned t0 = (unsigned)tok0 - (unsigned)v0;
        const uint64_t with = __ballot(tok[k] == tok0);
        if (tok[k] != tok0) one(tok[k]);
        else if (t0 < (unsigned)width && lane == __builtin_ctzll(with)) add(cell + t0, (uint32_t)__popcll(with));
      }
    } else {
#pragma unroll
      for (int k = 0; k < kOwnLoads; ++k) one(tok[k]);
    }
  }
  for (int64_t i = full + tid; i < n; i += 4 * kOwnThreads) {
    int tok[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) tok[k] = i + k * kOwnThreads < n ? tokens[i + k * kOwnThreads] : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) one(tok[k]);
  }
}

__global__ __launch_bounds__(kOwnThreads) void k_count_own(CountArgs a) {
  extern __shared__ uint32_t cell[];
  __shared__ int shared_row, reset_row;
  const int r = blockIdx.x, v0 = blockIdx.y * a.chunk;
  const int tid = threadIdx.x, width = min(a.chunk, a.V - v0);
  int64_t at;
  int n, srow;
  const bool ok = count_row(a, r, &at, &n, &srow);
  if (v0 == 0 && tid == 0) a.status[r] = ok ? 0 : SD_ST_BAD_INPUT;
  if (!ok) return;
  if (tid == 0) {
    shared_row = 0;
    reset_row = a.reset && a.reset[r];
  }
  for (int v = tid; v < a.chunk; v += kOwnThreads) cell[v] = 0;
  __syncthreads();
  // the first of the requests that share a state row enters them all
  if (a.slot)
    for (int q = tid; q < a.R; q += kOwnThreads)
      if (q != r && a.slot[q] == srow) {
        int64_t at_q;
        int n_q, s_q;
        if (count_row(a, q, &at_q, &n_q, &s_q)) {
          atomicOr(&shared_row, q < r ? 2 : 1);
          if (a.reset && a.reset[q]) reset_row = 1;
        }
      }
  __syncthreads();
  if (shared_row & 2) return;
  const bool clear = reset_row;
  // a prompt's tokens are marked, the others counted
  auto enter = [&](int64_t from, int len, int prompt) {
    const int cut = a.counts ? sdv::clampi(prompt, 0, len) : len;
    enter_tokens<true>(cell, cell + a.chunk, a.tokens + from, cut, v0, width);
    enter_tokens<false>(cell, cell + a.chunk, a.tokens + from + cut, len - cut, v0, width);
  };
  enter(at, n, a.prompt_len ? a.prompt_len[r] : 0);
  if (shared_row & 1)
    for (int q = r + 1; q < a.R; ++q) {
      int64_t at_q;
      int n_q, s_q;
      if (count_row(a, q, &at_q, &n_q, &s_q) && s_q == srow) enter(at_q, n_q, a.prompt_len ? a.prompt_len[q] : 0);
    }
  __syncthreads();
  // four tokens per lane (V, and so a range, is a multiple of 8); eight lanes'
  // bits make a word of the bitmap
  uint32_t* seen = a.seen + (int64_t)srow * a.ld_seen + v0 / 32;
  int32_t* counts = a.counts ? a.counts + (int64_t)srow * a.ld_counts + v0 : nullptr;
  for (int v = 4 * tid; v < (width + 255) / 256 * 256; v += 4 * kOwnThreads) {
    const bool in = v < width;
    const uint4 w = in ? *(const uint4*)&cell[v] : make_uint4(0, 0, 0, 0);
    uint32_t b = ((w.x != 0) | (w.y != 0) << 1 | (w.z != 0) << 2 | (w.w != 0) << 3) << (4 * (tid & 7));
    b |= __shfl_xor(b, 1, 64);
    b |= __shfl_xor(b, 2, 64);
    b |= __shfl_xor(b, 4, 64);
    if (!in) continue;
    if ((tid & 7) == 0) {
      uint32_t* s = seen + v / 32;
      if (clear) *s = b;
      else if (b) *s |= b;
    }
    if (!counts) continue;
    const sdv::u32x4 k = {w.x & ~kSeenBit, w.y & ~kSeenBit, w.z & ~kSeenBit, w.w & ~kSeenBit};
    if (clear) {
      __builtin_nontemporal_store(k, (sdv::u32x4*)(counts + v));
    } else if (k.x | k.y | k.z | k.w) {
      sdv::u32x4* p = (sdv::u32x4*)(counts + v);
      *p += k;
    }
  }
}

template <bool BF16>
hipError_t launch_shape(bool nt, bool copy, dim3 g, dim3 b, hipStream_t stream, const ShapeArgs& a) {
  if (nt)
    return copy ? sdv::launch(k_logit_shape<BF16, true, true>, g, b, 0, stream, a)
                : sdv::launch(k_logit_shape<BF16, true, false>, g, b, 0, stream, a);
  return copy ? sdv::launch(k_logit_shape<BF16, false, true>, g, b, 0, stream, a)
              : sdv::launch(k_logit_shape<BF16, false, false>, g, b, 0, stream, a);
}

}  // namespace

extern "C" int sd_logit_shape(hipStream_t stream, int R, int gamma_max, int V, int ld, int dtype,
                              const void* logits, void* out, int n_rows, const int32_t* row0,
                              const int32_t* ell, const int32_t* draft_tokens, const float* repetition,
                              const float* frequency, const float* presence, const uint32_t* seen,
                              int ld_seen, const int32_t* counts, int ld_counts, int n_slots,
                              const int32_t* slot, const int64_t* bias_off, const int32_t* bias_tok,
                              const float* bias_val, long long n_bias, const uint32_t* mask, int ld_mask,
                              int n_mask_rows, const int32_t* mask_row0, int32_t* status) {
  if (R < 0 || gamma_max < 0 || V < 8 || (V % 8) != 0 || ld < V || (ld % 8) != 0 || n_rows < 0)
    return SD_EINVAL;
  if (gamma_max > SD_MAX_GAMMA || V > SD_MAX_VOCAB) return SD_EUNSUPPORTED;
  if (dtype != SD_DTYPE_F32 && dtype != SD_DTYPE_BF16) return SD_EINVAL;
  if (R == 0) return SD_OK;
  if (!logits || !out || !row0 || !ell || !status) return SD_EINVAL;
  if ((((uintptr_t)logits) & 15) != 0 || (((uintptr_t)out) & 15) != 0) return SD_EINVAL;
  const int words = (V + 31) / 32;
  const bool pen = repetition || frequency || presence;
  if (pen && !seen) return SD_EINVAL;
  if ((frequency || presence) && !counts) return SD_EINVAL;
  if (pen && (n_slots < 1 || ld_seen < words)) return SD_EINVAL;
  if (counts && (ld_counts < V || (ld_counts % 4) != 0 || (((uintptr_t)counts) & 15) != 0)) return SD_EINVAL;
  if (bias_off && (n_bias < 0 || (n_bias > 0 && (!bias_tok || !bias_val)))) return SD_EINVAL;
  if (bias_off && n_bias > (1 << 30)) return SD_EUNSUPPORTED;
  if (mask && !mask_row0) return SD_EINVAL;
  if (mask_row0 && (n_mask_rows < 0 || (n_mask_rows > 0 && (!mask || ld_mask < words)))) return SD_EINVAL;
  ShapeArgs a;
  a.logits = (const char*)logits;
  a.out = (char*)out;
  a.row0 = row0;
  a.ell = ell;
  a.draft = draft_tokens;
  a.rep = repetition;
  a.freq = frequency;
  a.pres = presence;
  a.seen = seen;
  a.counts = counts;
  a.slot = slot;
  a.bias_off = bias_off;
  a.bias_tok = bias_tok;
  a.bias_val = bias_val;
  a.mask = mask;
  a.mask_row0 = mask_row0;
  a.status = status;
  a.n_bias = bias_off ? n_bias : 0;
  a.ld_bytes = (int64_t)ld * (dtype == SD_DTYPE_BF16 ? 2 : 4);
  a.gmax = gamma_max;
  a.V = V;
  a.n_ch = (V + kShapeChunk - 1) / kShapeChunk;
  a.n_rows = n_rows;
  a.n_slots = n_slots;
  a.ld_seen = ld_seen;
  a.ld_counts = ld_counts;
  a.ld_mask = ld_mask;
  a.n_mask_rows = n_mask_rows;
  const long long items = (long long)R * a.n_ch;
  const int rows = gamma_max + 1;
  const bool copy = out != logits;
  const bool nt = (double)R * rows * a.ld_bytes * (copy ? 2 : 1) > kCacheBytes;
  const long long spare = kFullWaves / (items > 0 ? items : 1);   // waves a request's rows may be split over
  const int most = spare < 1 ? 1 : (spare < rows ? (int)spare : rows);
  a.group = (rows + most - 1) / most;
  const int groups = (rows + a.group - 1) / a.group;   // each with rows of its own
  if (items * groups > 0xFFFFFFFFLL / kShapeThreads) return SD_EUNSUPPORTED;  // work-items of one launch
  using sdv::span;
  const long long es = dtype == SD_DTYPE_BF16 ? 2 : 4;
  const sdv::Span written[] = {span(out, n_rows, V * es, ld * es), span(status, 4LL * R)};
  const sdv::Span read[] = {
      span(logits == out ? nullptr : logits, n_rows, V * es, ld * es), span(row0, 4LL * R), span(ell, 4LL * R),
      span(draft_tokens, 4LL * R * gamma_max), span(repetition, 4LL * R), span(frequency, 4LL * R),
      span(presence, 4LL * R), span(pen ? seen : nullptr, n_slots, 4LL * words, 4LL * ld_seen),
      span(pen ? counts : nullptr, n_slots, 4LL * V, 4LL * ld_counts), span(slot, 4LL * R),
      span(bias_off, 8LL * (R + 1LL)), span(bias_off ? bias_tok : nullptr, 4 * n_bias),
      span(bias_off ? bias_val : nullptr, 4 * n_bias),
      span(mask_row0 ? mask : nullptr, n_mask_rows, 4LL * words, 4LL * ld_mask), span(mask_row0, 4LL * R)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
  const dim3 g((unsigned)items, groups), b(kShapeThreads);
  hipError_t e;
  if (dtype == SD_DTYPE_BF16)
    e = launch_shape<true>(nt, copy, g, b, stream, a);
  else
    e = launch_shape<false>(nt, copy, g, b, stream, a);
  SDV_TRY_LAUNCH(e);
  return SD_OK;
}

extern "C" int sd_token_counts(hipStream_t stream, int R, int V, const int32_t* tokens, long long n_tokens,
                               int width, const int64_t* start, const int32_t* length,
                               const int32_t* prompt_len, const int32_t* slot, const int32_t* reset,
                               uint32_t* seen, int ld_seen, int32_t* counts, int ld_counts, int n_slots,
                               int32_t* status) {
  if (R < 0 || V < 8 || (V % 8) != 0 || n_tokens < 0 || width < 0) return SD_EINVAL;
  if (V > SD_MAX_VOCAB) return SD_EUNSUPPORTED;
  if (R == 0) return SD_OK;
  if (!seen || !status || n_slots < 1 || ld_seen < (V + 31) / 32) return SD_EINVAL;
  if (n_tokens > 0 && !tokens) return SD_EINVAL;
  if (counts && (ld_counts < V || (ld_counts % 4) != 0 || (((uintptr_t)counts) & 15) != 0)) return SD_EINVAL;
  if (start && !length) return SD_EINVAL;
  if (!start && (long long)R * width > n_tokens) return SD_ERANGE;
  if ((long long)R * kCountThreads > 0xFFFFFFFFLL) return SD_EUNSUPPORTED;
  using sdv::span;
  const sdv::Span written[] = {span(seen, n_slots, (V + 31) / 32 * 4LL, 4LL * ld_seen),
                               span(counts, n_slots, 4LL * V, 4LL * ld_counts), span(status, 4LL * R)};
  const sdv::Span read[] = {span(tokens, n_tokens < 1LL << 60 ? 4 * n_tokens : 1LL << 62),
                            span(start, 8LL * R), span(length, 4LL * R), span(prompt_len, 4LL * R),
                            span(slot, 4LL * R), span(reset, 4LL * R)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
  CountArgs a;
  a.tokens = tokens;
  a.start = start;
  a.length = length;
  a.prompt_len = prompt_len;
  a.slot = slot;
  a.reset = reset;
  a.seen = seen;
  a.counts = counts;
  a.status = status;
  a.n_tokens = n_tokens;
  a.V = V;
  a.width = width;
  a.n_slots = n_slots;
  a.ld_seen = ld_seen;
  a.ld_counts = ld_counts;
  a.R = R;
  // the lengths are on the device: what a list can hold on average
  const long long room = start ? n_tokens / R : width;
  const long long mean = start && width > 0 && width < room ? width : room;
  // workgroups per request: 2048 in all, as far as the work goes
  auto split = [&](long long work, long long each) {
    const long long fill = (2048 + R - 1) / R, need = (work + each - 1) / each;
    return (unsigned)(need < 1 ? 1 : (need < fill ? need : fill));
  };
  const int most = mean < kOwnLongList ? kOwnMaxChunk / 2 : kOwnMaxChunk;
  a.chunk = V < most ? (V + 63) / 64 * 64 : most;
  const int n_ch = (V + a.chunk - 1) / a.chunk;
  if ((reset || mean >= kOwnMinList) && R <= kOwnMaxRequests &&
      (long long)R * n_ch * kOwnThreads <= 0xFFFFFFFFLL) {   // work-items of one launch
    const size_t lds = (a.chunk + 64) * sizeof(uint32_t);
    if (lds > 64 * 1024)
      SDV_TRY_LAUNCH(hipFuncSetAttribute((const void*)k_count_own, hipFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)lds));
    SDV_TRY_LAUNCH(sdv::launch(k_count_own, dim3(R, n_ch), dim3(kOwnThreads), lds, stream, a));
    return SD_OK;
  }
  if (reset)
    SDV_TRY_LAUNCH(sdv::launch(k_count_clear, dim3(R, split(V, kCountThreads)), dim3(kCountThreads), 0, stream, a));
  SDV_TRY_LAUNCH(sdv::launch(k_count_add, dim3(R, split(width > 0 || !start ? width : n_tokens, kCountThreads)),
                             dim3(kCountThreads), 0, stream, a));
  return SD_OK;
}
