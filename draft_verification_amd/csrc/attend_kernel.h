// The attention kernel: see attend.h for how a step's work is cut up.
//
// Scores are formed transposed, S^T = K Q^T (tokens are the matrix
// instruction's rows, queries its columns).  A lane then holds, for one query,
// four neighbouring tokens of each 16, and that is the operand layout that
// O^T = V^T P^T takes its P^T in (which token stands at which place of the sum
// is free as long as V^T agrees): the weights go from one product into the
// next without leaving their registers.  A query's running maximum and sum are
// the same lane's, two exchanges with the other lane groups join them, and the
// rescaling of O^T is a product by a lane's own number.  V^T comes from LDS by
// transposing reads, four tokens of one channel to a lane.
#pragma once

#include "attend.h"

namespace sdv {
namespace attn {

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) uint16_t* LdsPtr;

// A value that is the same for the whole wave, in scalar registers.
template <typename T>
SDV_DEV T uniform(const T& v) {
  constexpr int kWords = sizeof(T) / 4;
  struct W {
    int w[kWords];
  } x = __builtin_bit_cast(W, v);
#pragma unroll
  for (int i = 0; i < kWords; ++i) x.w[i] = __builtin_amdgcn_readfirstlane(x.w[i]);
  return __builtin_bit_cast(T, x);
}

// 16 bytes per lane straight into LDS, from `to` of the wave on, lane after
// lane.  Not the builtin: the compiler then waits for all loads in flight
// before any later read of LDS, also of the other buffer.  (m0 is the compiler's to
// set before each use, and nothing else here uses it.)  Nothing but LDS is
// written; the callers wait (vmcnt) before the barrier that shows it to others.
SDV_DEV void load_to_lds(const void* from, const uint16_t* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(LdsPtr)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory");
}

SDV_DEV float max_over_groups(float v) {   // over lanes l, l ^ 16, l ^ 32, l ^ 48
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
SDV_DEV float sum_over_groups(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// D channels; NT times 16 queries per wave; WT waves share a tile's queries
// and take TT / WT tokens of a unit each, the other waves take other queries.
template <int D, int NT, int WT, bool kFp4>
struct Kernel {
  static constexpr int TT = D <= 128 ? 64 : 32;
  static constexpr int WQ = 4 / WT;
  static constexpr int M = WQ * NT * 16;
  static constexpr int TW = TT / WT;          // tokens of a wave
  static constexpr int NS = TW / 16;
  static constexpr int KS = D / 32;           // steps of the sum over channels
  static constexpr int ND = D / 16;           // rows of O^T, 16 at a time
  static constexpr int CH = D / 8;            // chunks of 16 bytes in a token's row
  static constexpr int kSide = TT * D;        // elements of one side of a unit
  static constexpr int kLoads = TT * CH / kAttnThreads;      // chunks of a thread, one side
  static constexpr int kGroups = TT * (D / 32);              // of 32 channels, one side
  static constexpr int kRow = kFp4 ? D / 2 : D * 2;          // bytes of a token, without scales
  static constexpr int kAhead = kFp4 ? 2 : 1;                // units requested before they are needed
  static constexpr int kTokens = kFp4 ? 1 : kLoads;          // tokens whose blocks a thread looks up
  static_assert(TW >= 16 && TT * CH % kAttnThreads == 0 && kGroups <= kAttnThreads, "unit");

  // A token's chunks are stored at c ^ swizzle(t), so that the rows that one
  // read touches (16 of keys; 4 of values, two chunks each) lie in different
  // banks.  It changes the lowest bits of c alone: a lane has one address for
  // each value of those (kPeriodK steps of keys, kPeriodV rows of values), and
  // the rest are constants.
  static SDV_DEV int swz_k(int t) { return CH % 8 == 0 ? t & 7 : t & 3; }
  static SDV_DEV int swz_v(int t) { return CH % 8 == 0 ? (t & 3) << 1 : (t & 1) << 1; }
  static constexpr int kPeriodK = CH % 8 == 0 ? 2 : 1, kPeriodV = CH % 8 == 0 ? 4 : 2;

  struct Shared {
    uint16_t kv[2][2][kSide];     // two units of keys and values
    float ml[WT > 1 ? (WT - 1) * M * 2 : 1];
    int bad[2];                   // the unit has a block outside the pool
  };

  const AttnArgs& a;
  Shared& sh;
  const int tid, lane, wave, l16, g, wq, wt;

  int at_k[kPeriodK], at_v[kPeriodV];   // elements from the start of a side

  // The tile at hand
  int q0, queries, ctx, row0, n, h, req;
  const char* k_head;             // the head's keys and values in block 0
  const char* v_head;
  const int32_t* table;           // the request's row
  bool causal;
  int window;
  b16x8 qf[NT][KS];
  f32x4 o[ND][NT];
  float m[NT], l[NT];
  int hi[NT], lo[NT];
  int all_hi, all_lo;             // tokens in [all_lo, all_hi) are seen by every query of the tile

  SDV_DEV Kernel(const AttnArgs& args, Shared& shared)
      : a(args), sh(shared), tid(threadIdx.x), lane(tid & 63), wave(__builtin_amdgcn_readfirstlane(tid >> 6)),
        l16(lane & 15), g(lane >> 4), wq(wave / WT), wt(wave % WT) {
#pragma unroll
    for (int i = 0; i < kPeriodK; ++i) at_k[i] = (wt * TW + l16) * D + ((i * 4 + g) ^ swz_k(l16)) * 8;
    const int row = 4 * g + (l16 >> 2);
#pragma unroll
    for (int i = 0; i < kPeriodV; ++i)
      at_v[i] = (wt * TW + row) * D + ((2 * i + ((l16 & 3) >> 1)) ^ swz_v(row)) * 8 + (l16 & 1) * 4;
  }

  SDV_DEV int block_of(int token) const { return (int)((uint64_t)(uint32_t)token * a.bs_mul >> a.bs_shift); }

  SDV_DEV void begin(const Tile& t, int head) {
    q0 = t.q0, queries = t.queries, ctx = t.ctx, row0 = t.row0, n = t.n, req = t.req, h = head;
    const int64_t first = (int64_t)h * a.cache.bs;
    k_head = (const char*)a.cache.k + first * kRow;
    v_head = (const char*)a.cache.v + first * kRow;
    table = a.table + (int64_t)req * a.max_blocks;
    const int G = a.group, base = ctx - n;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = q0 + (wq * NT + nt) * 16 + l16;
      const bool in = qi < queries;
      const int i = (in ? qi : q0) / G;
      const uint16_t* q = a.q + (int64_t)(row0 + i) * a.ld_q + (int64_t)(h * G + (in ? qi - i * G : 0)) * D + g * 8;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        b16x8 z = {};
        qf[nt][ks] = in ? *(const b16x8*)(q + ks * 32) : z;
      }
      hi[nt] = causal ? base + i + 1 : ctx;
      lo[nt] = window ? base + i + 1 - window : 0;
      m[nt] = -__builtin_huge_valf();
      l[nt] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int last = (min(q0 + M, queries) - 1) / G;
    all_hi = causal ? base + q0 / G + 1 : ctx;
    all_lo = window ? base + last + 1 - window : 0;
  }

  // ---- loading a unit -----------------------------------------------------
  // The blocks of a thread's tokens are looked up one unit before they are used.
  SDV_DEV int token_of(int u, int j) const {
    const int row = kFp4 ? tid / (D / 32) : (j * kAttnThreads + tid) / CH;
    return min(u * TT + row, ctx - 1);       // past the end: the last one again, and masked
  }
  SDV_DEV void look_up(int u, int (&blk)[kTokens]) const {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) blk[j] = table[block_of(token_of(u, j))];
  }
  // The token of this thread's piece j, counted from the head's first in block 0.
  SDV_DEV int64_t token_at(int u, int j, int blk, bool& bad) const {
    const int tok = token_of(u, j);
    const bool ok = (unsigned)blk < (unsigned)a.cache.n_blocks;
    bad |= !ok;
    return (int64_t)((uint64_t)(uint32_t)(ok ? blk : 0) * a.block_tokens + (uint32_t)(tok - block_of(tok) * a.cache.bs));
  }

  SDV_DEV void note_bad(bool bad, int buf) {
    if (__builtin_expect(bad, 0)) {
      sh.bad[buf] = 1;
      atomicOr(a.status + req, SD_ST_BAD_INPUT);
    }
  }

  // bf16: straight into LDS, a wave's 64 lanes one KB at a time.
  SDV_DEV void load_bf16(int u, int buf, const int (&blk)[kTokens]) {
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int x = j * kAttnThreads + tid, row = x / CH, c = x % CH;
      const int64_t at = token_at(u, j, blk[j < kTokens ? j : 0], bad) * kRow;
      const int base = (j * kAttnThreads + wave * 64) * 8;
      load_to_lds(k_head + at + (c ^ swz_k(row)) * 16, sh.kv[buf][0] + base);
      load_to_lds(v_head + at + (c ^ swz_v(row)) * 16, sh.kv[buf][1] + base);
    }
    note_bad(bad, buf);
  }

  // 4 bits: a group of 32 channels of each side into registers, and from
  // there, as bf16, into LDS.
  struct Codes {
    uint4 k, v;
    uint32_t ks, vs;
    bool bad;
  };
  SDV_DEV void load_fp4(int u, Codes& c, const int (&blk)[kTokens]) const {
    c.bad = false;
    if (tid < kGroups) {
      const int64_t at = token_at(u, 0, blk[0], c.bad) * (D / 32) + tid % (D / 32);
      const int64_t first = (int64_t)h * a.cache.bs * (D / 32);
      c.k = ((const uint4*)k_head)[at];
      c.v = ((const uint4*)v_head)[at];
      c.ks = a.cache.k_scale[first + at];
      c.vs = a.cache.v_scale[first + at];
    }
  }
  SDV_DEV void put_fp4(const Codes& c, int buf) {
    if (tid < kGroups) {
      const int row = tid / (D / 32), first = tid % (D / 32) * 4;
      const uint32_t kw[4] = {c.k.x, c.k.y, c.k.z, c.k.w}, vw[4] = {c.v.x, c.v.y, c.v.z, c.v.w};
      const float ks = fp4_scale(c.ks), vs = fp4_scale(c.vs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *(uint4*)(sh.kv[buf][0] + row * D + ((first + i) ^ swz_k(row)) * 8) = fp4_to_bf16(kw[i], ks);
        *(uint4*)(sh.kv[buf][1] + row * D + ((first + i) ^ swz_v(row)) * 8) = fp4_to_bf16(vw[i], vs);
      }
    }
    note_bad(c.bad, buf);
  }

  // ---- one unit -----------------------------------------------------------
  SDV_DEV u32x2 v_part(const uint16_t* v, int s, int d) const {   // tokens 16 s + 4 g .. + 3 of channel 16 d + l16
    const uint16_t* p = v + at_v[d % kPeriodV] + s * 16 * D + d / kPeriodV * kPeriodV * 16;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)p));
  }

  SDV_DEV void unit(int u, int buf) {
    const uint16_t* kk = sh.kv[buf][0];
    const uint16_t* vv = sh.kv[buf][1];
    f32x4 s[NS][NT];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[i][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const b16x8 kf = *(const b16x8*)(kk + at_k[ks % kPeriodK] + i * 16 * D + ks / kPeriodK * kPeriodK * 32);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[i][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[nt][ks], s[i][nt], 0, 0, 0);
      }
    }
    const bool bad = sh.bad[buf] != 0;
    // the same for all waves, as is what follows from it
    const bool masked = bad || (u + 1) * TT > all_hi || u * TT < all_lo;
    uint64_t ok = ~0ull;
    bool fault = false;   // values that are not finite beside masked weights
    if (masked) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t from = (uint32_t)(u * TT + wt * TW + 4 * g) - (uint32_t)lo[nt];   // the lane's first token
        const uint32_t span = (uint32_t)hi[nt] - (uint32_t)lo[nt];
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (from + (i * 16 + e) >= span) s[i][nt][e] = -__builtin_huge_valf();
      }
      if (__builtin_expect(bad, 0)) {
        const int blk = table[block_of(min(u * TT + lane % TT, ctx - 1))];
        ok = __ballot((unsigned)blk < (unsigned)a.cache.n_blocks);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (!(ok >> (wt * TW + i * 16 + 4 * g + e) & 1)) s[i][nt][e] = -__builtin_huge_valf();
      }
      int odd = 0;
      for (int x = tid; x < TT * CH; x += kAttnThreads) {
        const uint4 w = *(const uint4*)(vv + x * 8);
        odd |= not_finite(w.x) | not_finite(w.y) | not_finite(w.z) | not_finite(w.w);
      }
      fault = __syncthreads_or(odd) != 0;
    }
    // The maximum that the weights are taken against moves only where a score
    // is 2^8 times over it: what it does to the sums is exact to rounding
    // either way, and most units then rescale nothing.
    bool move = false;
    float top[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x = -__builtin_huge_valf();
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x = fmaxf(x, s[i][nt][e]);
      top[nt] = max_over_groups(x) * a.scale2;
      move |= top[nt] > m[nt] + 8.f;
    }
    if (__ballot(move) != 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float to = fmaxf(m[nt], top[nt]);
        const float f = to == -__builtin_huge_valf() ? 1.f : fast_exp2(m[nt] - to);
        m[nt] = to;
        l[nt] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][nt] *= f;
      }
    }
    uint32_t p[NS][NT][2];   // weights, two tokens to a word
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ref = m[nt] == -__builtin_huge_valf() ? 0.f : m[nt];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = fast_exp2(fmaf(s[i][nt][e], a.scale2, -ref));
          l[nt] += w[e];
        }
        // Rounded to bf16 for the matrix cores: 2^-9 of each weight, and the
        // errors of different tokens do not add up.
        p[i][nt][0] = pack_bf16(w[0], w[1]);
        p[i][nt][1] = pack_bf16(w[2], w[3]);
      }
    }
    if (__builtin_expect(fault, 0)) {
      // 0 * inf and 0 * NaN of masked tokens must not reach a sum: values that
      // are not finite are added here, for the queries that see their tokens,
      // and taken out before the product.
      add_faults(u, ok, vv, p);
      __syncthreads();
      for (int x = tid; x < TT * D; x += kAttnThreads)
        if ((sh.kv[buf][1][x] & 0x7F80u) == 0x7F80u) sh.kv[buf][1][x] = 0;
      __syncthreads();
    }
    accumulate(vv, p);
  }

  static SDV_DEV int not_finite(uint32_t w) {   // either half of a word
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
  }

  SDV_DEV void accumulate(const uint16_t* vv, const uint32_t (&p)[NS][NT][2]) {
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      if constexpr (NS == 1) {
        const u32x2 v = v_part(vv, 0, d);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[d][nt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
              __builtin_bit_cast(s16x4, v), __builtin_bit_cast(s16x4, u32x2{p[0][nt][0], p[0][nt][1]}), o[d][nt], 0, 0,
              0);
      } else {
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
          const u32x2 x = v_part(vv, i, d), y = v_part(vv, i + 1, d);
          const uint4 v = make_uint4(x[0], x[1], y[0], y[1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            o[d][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(b16x8, v),
                __builtin_bit_cast(b16x8, make_uint4(p[i][nt][0], p[i][nt][1], p[i + 1][nt][0], p[i + 1][nt][1])),
                o[d][nt], 0, 0, 0);
        }
      }
    }
  }

  // Token by token, as this is rare and its code has to be small.
  SDV_DEV void add_faults(int u, uint64_t ok, const uint16_t* vv, const uint32_t (&p)[NS][NT][2]) {
#pragma unroll 1
    for (int at = 0; at < TW; ++at) {
      const int s = at >> 4, from = at >> 2 & 3, e = at & 3, row = wt * TW + at;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < NS; ++i) w = s == i ? (e & 2 ? p[i][nt][1] : p[i][nt][0]) : w;
        w = __shfl((int)w, from * 16 + l16, 64);     // of the lane group that holds the token
        const float weight = e & 1 ? bf16hi(w) : bf16lo(w);
        const bool see = (uint32_t)(u * TT + row) - (uint32_t)lo[nt] < (uint32_t)hi[nt] - (uint32_t)lo[nt] &&
                         (ok >> row & 1);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const int c = 2 * d + (g >> 1);
          const uint2 v = *(const uint2*)(vv + row * D + (c ^ swz_v(row)) * 8 + (g & 1) * 4);
          const float x[4] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y)};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (see && !(__builtin_fabsf(x[i]) < __builtin_huge_valf())) o[d][nt][i] += weight * x[i];
        }
      }
    }
  }

  // ---- the end of a run's part of a tile ----------------------------------
  // Waves that took other tokens of the same queries are joined in LDS.
  SDV_DEV void join_waves() {
    float* ob = (float*)sh.kv;                       // [WT - 1][M][D]
    float* mb = sh.ml;
    static_assert((WT - 1) * M * D * 4 <= (int)sizeof(sh.kv), "join");
    __syncthreads();                                 // the last unit has been read by all
    if (wt > 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = (wq * NT + nt) * 16 + l16;
        float* to = ob + ((int64_t)(wt - 1) * M + col) * D;
#pragma unroll
        for (int d = 0; d < ND; ++d) *(f32x4*)(to + ((d * 16 + 4 * g) ^ ((l16 & 7) << 2))) = o[d][nt];
        if (g == 0) {
          mb[((wt - 1) * M + col) * 2] = m[nt];
          mb[((wt - 1) * M + col) * 2 + 1] = l[nt];
        }
      }
    }
    __syncthreads();
    if (wt == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = (wq * NT + nt) * 16 + l16;
        float top = m[nt];
#pragma unroll
        for (int w = 0; w < WT - 1; ++w) top = fmaxf(top, mb[(w * M + col) * 2]);
        const float ref = top == -__builtin_huge_valf() ? 0.f : top;
        float f = fast_exp2(m[nt] - ref);
        l[nt] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[d][nt] *= f;
#pragma unroll
        for (int w = 0; w < WT - 1; ++w) {
          f = fast_exp2(mb[(w * M + col) * 2] - ref);
          l[nt] += mb[(w * M + col) * 2 + 1] * f;
          const float* from = ob + ((int64_t)w * M + col) * D;
#pragma unroll
          for (int d = 0; d < ND; ++d) o[d][nt] += *(const f32x4*)(from + ((d * 16 + 4 * g) ^ ((l16 & 7) << 2))) * f;
        }
        m[nt] = top;
      }
    }
    __syncthreads();                                 // the buffers are free again
  }

  SDV_DEV void end(int slot) {                       // slot < 0: the tile is whole
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt] = sum_over_groups(l[nt]);
    if constexpr (WT > 1) join_waves();
    if (WT > 1 && wt > 0) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = (wq * NT + nt) * 16 + l16, qi = q0 + col;
      if (qi >= queries) continue;
      if (slot < 0) {
        const int i = qi / a.group, head = h * a.group + qi - i * a.group;
        const float inv = l[nt] == 0.f ? 0.f : 1.f / l[nt];
        uint16_t* to = a.out + (int64_t)(row0 + i) * a.ld_out + (int64_t)head * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const f32x4 v = o[d][nt] * inv;
          *(uint2*)(to + d * 16) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        }
        if (a.lse && g == 0)
          a.lse[(int64_t)(row0 + i) * a.n_q + head] =
              l[nt] == 0.f ? -__builtin_huge_valf() : (m[nt] + __log2f(l[nt])) * 0.69314718055994531f;
      } else {
        float* to = a.part + ((int64_t)slot * M + col) * D + 4 * g;
#pragma unroll
        for (int d = 0; d < ND; ++d) *(f32x4*)(to + d * 16) = o[d][nt];
        if (g == 0) a.ml[(int64_t)slot * M + col] = make_float2(m[nt], l[nt]);
      }
    }
  }

  // Units [u, u + n) of the tile at hand.
  SDV_DEV void units(int u, int n) {
    if (tid < 2) sh.bad[tid] = 0;
    __syncthreads();
    if constexpr (!kFp4) {
      int blk[kTokens];
      look_up(u, blk);
      load_bf16(u, 0, blk);
      if (n > 1) look_up(u + 1, blk);
      for (int i = 0; i < n; ++i) {
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): this unit is in LDS
        __syncthreads();                      // ... for every wave, and the other buffer has been read
        if (i + 1 < n) {
          load_bf16(u + i + 1, (i + 1) & 1, blk);
          if (i + 2 < n) look_up(u + i + 2, blk);
        }
        unit(u + i, i & 1);
      }
    } else {
      int blk[kAhead + 1][kTokens];
      Codes c[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) look_up(u + i, blk[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < n) load_fp4(u + i, c[i], blk[i]);
      if (kAhead < n) look_up(u + kAhead, blk[kAhead]);
      for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          const int i = i0 + e;
          if (i < n) {                          // the same for all waves
            put_fp4(c[e], i & 1);
            if (i + kAhead < n) {
              load_fp4(u + i + kAhead, c[e], blk[kAhead]);
              if (i + kAhead + 1 < n) look_up(u + i + kAhead + 1, blk[kAhead]);
            }
            __syncthreads();                    // the unit is in LDS; the one before has been read by all
            unit(u + i, i & 1);
          }
        }
      }
    }
    __syncthreads();
  }
};

template <int D, int NT, int WT, bool kFp4>
__global__ __launch_bounds__(kAttnThreads, 2) void k_attend(AttnArgs a) {
  using K = Kernel<D, NT, WT, kFp4>;
  __shared__ typename K::Shared sh;
  const PlanHead& p = *a.head;
  // Neighbouring runs read the same tokens where a request has several tiles:
  // they go to the same eighth of the chip, which shares a cache.
  const int per = (int)gridDim.x / 8, w = (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8;
  if (!same_shape(p.shape, a.shape)) return;
  const long long quota = p.quota, total = p.total;
  long long at = w * quota;
  const long long end = at + quota < total ? at + quota : total;
  if (at >= end) return;
  K k(a, sh);
  k.causal = p.causal != 0;
  k.window = p.window;
  Start s = uniform(a.starts[w]);
  const int n_tiles = p.n_tiles;
  while (at < end) {
    const Tile t = uniform(a.tiles[s.tile]);
    const long long room = end - at;
    const int left = t.units - s.off, n = left < room ? left : (int)room;
    if (in_range(a, t)) {
      k.begin(t, s.head);
      k.units(t.u0 + s.off, n);
      // a part that begins its tile goes to the run's second place, others to its first
      k.end(n == t.units ? -1 : s.off == 0 ? 2 * w + 1 : 2 * w);
    } else if (threadIdx.x == 0) {
      atomicOr(a.status + t.req, SD_ST_BAD_INPUT);
    }
    at += n;
    s.off = 0;
    if (++s.tile == n_tiles) {
      s.tile = 0;
      ++s.head;
    }
  }
}

template <bool kFp4>
int launch_attend(hipStream_t stream, int M, int W, const AttnArgs& a) {
  const dim3 grid((unsigned)W), block(kAttnThreads);
#define SDV_ATTN(...) SDV_TRY_LAUNCH(sdv::launch(k_attend<__VA_ARGS__, kFp4>, grid, block, 0, stream, a))
#define SDV_ATTN_SMALL(D)                                  \
  case D:                                                  \
    if (M == 16) SDV_ATTN(D, 1, 4);                        \
    else if (M == 32) SDV_ATTN(D, 1, 2);                   \
    else if (M == 64) SDV_ATTN(D, 2, 2);                   \
    else SDV_ATTN(D, 2, 1);                                \
    return SD_OK;
#define SDV_ATTN_LARGE(D)                                  \
  case D:                                                  \
    if (M == 32) SDV_ATTN(D, 1, 2);                        \
    else SDV_ATTN(D, 1, 1);                                \
    return SD_OK;
  switch (a.shape.D) {
    SDV_ATTN_SMALL(64)
    SDV_ATTN_SMALL(96)
    SDV_ATTN_SMALL(128)
    SDV_ATTN_LARGE(192)
    SDV_ATTN_LARGE(256)
  }
#undef SDV_ATTN_LARGE
#undef SDV_ATTN_SMALL
#undef SDV_ATTN
  return SD_EUNSUPPORTED;
}

}  // namespace attn
}  // namespace sdv
