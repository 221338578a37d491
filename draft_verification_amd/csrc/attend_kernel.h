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

#include <type_traits>

#include "attend.h"

namespace sdv {
namespace attn {

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(4))) int32_t* ConstPtr;   // read by scalar loads

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
// before any later read of LDS, also of the other buffer.  Nothing but LDS and m0
// is written; the callers wait (vmcnt) before the barrier that shows it to
// others.
// Between m0 and its use there has to be one instruction, between a scalar base
// that a vector instruction wrote (a lane's value, or one kept in a lane) and its
// use five: the compiler sees to neither inside assembly.
template <bool kOnce>   // read once: streaming
SDV_DEV void load_to_lds(const void* base, uint32_t off, uint32_t to) {   // base: the same for the wave
  if constexpr (kOnce)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(to), "v"(off), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(base)
                 : "memory", "m0");
}
template <bool kOnce>
SDV_DEV void load_to_lds(const void* from, uint32_t to) {
  if constexpr (kOnce)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(to), "v"(from)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from)
                 : "memory", "m0");
}
// ... and 4 bytes per lane.
SDV_DEV void load_word_to_lds(const void* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from)
               : "memory", "m0");
}
SDV_DEV uint32_t lds_at(const void* p) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p; }

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

// What every form of the kernel keeps of a tile: D channels, NT times 16
// queries of a wave, 16 NS of its tokens at a time, of each 16 of which lane
// group g has kByGroup g + kByPlace e, e < 4.
template <int D, int NT, int NS, bool kFp4, bool kWide, int kByGroup = 4, int kByPlace = 1>
struct Queries {
  static constexpr int KS = D / 32;           // steps of the sum over channels
  static constexpr int ND = D / 16;           // rows of O^T, 16 at a time
  static constexpr int DG = D / 32;           // groups of 32 channels
  static constexpr int kRow = kFp4 ? D / 2 : D * 2;          // bytes of a token, without scales

  const AttnArgs& a;
  const int tid, lane, wave, l16, g;
  // The tile at hand
  int q0, queries, ctx, row0, n, h, req;
  const char* k_head;             // the head's keys and values in block 0
  const char* v_head;
  const uint8_t* ks_head;
  const uint8_t* vs_head;
  const int32_t* table;           // the request's row
  bool causal;
  int window;
  int turn;                       // which of a CU's two workgroups this is likely to be
  b16x8 qf[NT][KS];
  f32x4 o[ND][NT];
  float m[NT], l[NT];
  int hi[NT], lo[NT];
  int all_hi, all_lo;             // tokens in [all_lo, all_hi) are seen by every query of the tile

  SDV_DEV explicit Queries(const AttnArgs& args)
      : a(args), tid(threadIdx.x), lane(tid & 63), wave(__builtin_amdgcn_readfirstlane(tid >> 6)), l16(lane & 15),
        g(lane >> 4) {}

  // Which eight channels (times 8) a lane multiplies at a step: any order will
  // do if queries and keys agree.  Of keys in 4 bits a lane takes D / 4
  // neighbours, one wide read and one or two scales, where D / 4 is whole
  // groups or parts of one.
  static SDV_DEV int eighth(int ks, int g) { return kWide ? KS * g + ks : 4 * ks + g; }

  SDV_DEV int block_of(int token) const { return (int)((uint64_t)(uint32_t)token * a.bs_mul >> a.bs_shift); }
  // Tokens are counted from the head's first in block 0.
  SDV_DEV uint64_t place(int tok, int blk, bool& bad) const {
    const bool ok = (unsigned)blk < (unsigned)a.cache.n_blocks;
    bad |= !ok;
    return (uint64_t)(uint32_t)(ok ? blk : 0) * a.block_tokens + (uint32_t)(tok - block_of(tok) * a.cache.bs);
  }

  // M queries of the tile; this wave's begin at column `col`.
  SDV_DEV void begin(const Tile& t, int head, int col, int M) {
    q0 = t.q0, queries = t.queries, ctx = t.ctx, row0 = t.row0, n = t.n, req = t.req, h = head;
    const int64_t first = (int64_t)h * a.cache.bs;
    k_head = (const char*)a.cache.k + first * kRow;
    v_head = (const char*)a.cache.v + first * kRow;
    if (kFp4) {
      ks_head = a.cache.k_scale + first * DG;
      vs_head = a.cache.v_scale + first * DG;
    }
    table = a.table + (int64_t)req * a.max_blocks;
    const int G = a.group, base = ctx - n;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = q0 + col + nt * 16 + l16;
      const bool in = qi < queries;
      const int i = (in ? qi : q0) / G;
      const uint16_t* q = a.q + (int64_t)(row0 + i) * a.ld_q + (int64_t)(h * G + (in ? qi - i * G : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        b16x8 z = {};
        qf[nt][ks] = in ? *(const b16x8*)(q + eighth(ks, g) * 8) : z;
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

  SDV_DEV bool sees(int tok, int nt) const {
    return (uint32_t)tok - (uint32_t)lo[nt] < (uint32_t)hi[nt] - (uint32_t)lo[nt];
  }

  // Scores of 16 NS tokens from `first` on that their query does not see.
  SDV_DEV void mask(int first, f32x4 (&s)[NS][NT]) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t from = (uint32_t)(first + kByGroup * g) - (uint32_t)lo[nt];   // the lane's first token
      const uint32_t span = (uint32_t)hi[nt] - (uint32_t)lo[nt];
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (from + (i * 16 + kByPlace * e) >= span) s[i][nt][e] = -__builtin_huge_valf();
    }
  }
  // ... and of those outside the pool; returns which of the tokens are in it.
  // The request is told of those that a row of the tile (M queries) sees: the
  // others that lie in its units, behind a window, need no block.
  SDV_DEV uint64_t mask_pool(int first, int i0, int M, f32x4 (&s)[NS][NT]) const {
    const int tok = first + i0 * 16 + lane, blk = table[block_of(min(tok, ctx - 1))];
    const uint64_t ok = __ballot((unsigned)blk < (unsigned)a.cache.n_blocks);
    const int base = ctx - n, to = causal ? base + (min(q0 + M, queries) - 1) / a.group + 1 : ctx;
    const int from = window ? base + q0 / a.group + 1 - window : 0;
    const uint64_t seen = __ballot(tok >= from && tok < to);
    if ((~ok & seen) != 0 && lane == 0) atomicOr(a.status + req, SD_ST_BAD_INPUT);
#pragma unroll
    for (int i = 0; i < 4 && i < NS; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (i0 + i < NS && !(ok >> (i * 16 + kByGroup * g + kByPlace * e) & 1)) s[i0 + i < NS ? i0 + i : 0][nt][e] = -__builtin_huge_valf();
    return ok;
  }

  // The maximum that the weights are taken against moves only where a score
  // is 2^8 times over it: what it does to the sums is exact to rounding
  // either way, and most units then rescale nothing.
  SDV_DEV void move_maximum(const f32x4 (&s)[NS][NT]) {
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
  }

  // The weights, two tokens to a word.
  SDV_DEV void weights(const f32x4 (&s)[NS][NT], u32x2 (&p)[NT][NS]) {
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
        // Rounded to bf16 for the matrix cores: up to 2^-8 of each weight, and
        // the errors of different tokens do not add up.
        p[nt][i] = u32x2{pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])};
      }
    }
  }

  // Of the queries above all: what is on its way where a loop begins, the
  // compiler waits for in every turn.
  static SDV_DEV void wait_all() { __builtin_amdgcn_s_waitcnt(0x0f70); }
};

// D channels; NT times 16 queries per wave; WT waves share a tile's queries
// and take TT / WT tokens of a unit each, the other waves take other queries.
// Units pass through LDS.
template <int D, int NT, int WT, bool kFp4>
struct Kernel : Queries<D, NT, attn_unit(D, 64 / WT * NT, kFp4) / WT / 16, kFp4, kFp4 && (D == 64 || D == 128 || D == 256)> {
  static constexpr int WQ = 4 / WT;
  static constexpr int M = WQ * NT * 16;
  static constexpr int TT = attn_unit(D, M, kFp4);
  static constexpr int TW = TT / WT;          // tokens of a wave
  static constexpr int NS = TW / 16;
  static constexpr bool kWide = kFp4 && (D == 64 || D == 128 || D == 256);
  using Base = Queries<D, NT, NS, kFp4, kWide>;
  using Base::a, Base::tid, Base::lane, Base::wave, Base::l16, Base::g;
  using Base::q0, Base::queries, Base::ctx, Base::row0, Base::h, Base::req, Base::table;
  using Base::k_head, Base::v_head, Base::ks_head, Base::vs_head;
  using Base::qf, Base::o, Base::m, Base::l, Base::all_hi, Base::all_lo;
  using Base::KS, Base::ND, Base::DG, Base::kRow, Base::block_of, Base::place, Base::wait_all;
  static constexpr int CH = D / 8;            // chunks of 16 bytes in a token's row
  static constexpr int RW = TT / 4;           // tokens of a unit that a wave loads, next to each other
  static constexpr int kPer = kFp4 ? DG : CH;                // pieces of 16 bytes in a token's row
  static constexpr int kPieces = (RW * kPer + 63) / 64;      // of a lane, one side of a unit
  static constexpr int kSpan = attn_span(D, M, kFp4);        // tokens that share one look-up of their block
  static constexpr int kSpans = kFp4 ? kPieces : 1;          // of a wave
  static_assert(TW % 16 == 0 && (kFp4 || RW * CH % 64 == 0), "unit");
  // A wave's spans are its tokens: a longer one would begin inside another's,
  // and end behind its block.
  static_assert(kSpan == 0 || kSpan * kSpans == RW, "spans");

  // A token's chunks of 16 bytes are stored at c ^ swizzle(t), so that what one
  // access touches at a time (16 tokens of keys; 8 of values, two chunks each)
  // lies in different ones of the 64 banks, 16 chunks wide.  bf16 rows of 16
  // chunks begin at the same bank, of 8 or 24 at every second one's, of 12 at
  // every fourth's.  It changes the lowest bits of c alone: a lane has one
  // address for each value of those (kPeriodK steps of keys, kPeriodV rows of
  // values), the rest are constants.
  static constexpr int kRowsPerBanks = CH % 16 == 0 ? 1 : CH % 8 == 0 ? 2 : 4;
  static SDV_DEV int swz_k(int t) {
    if (kRowsPerBanks == 1) return t & 15;
    if (kRowsPerBanks == 2) return t & 7;
    const int x = t >> 2 & 3;
    return ((x ^ x >> 1) & 1) << 1 | x >> 1;
  }
  static SDV_DEV int swz_v(int t) {
    if (kRowsPerBanks == 1) return (t & 7) << 1;
    if (kRowsPerBanks == 2) return (t >> 1 & 3) << 1;
    return (t >> 2 & 1) << 1;
  }
  static constexpr int kPeriodK = 4 / kRowsPerBanks, kPeriodV = 8 / kRowsPerBanks;
  // Keys in 4 bits stay so in LDS, D / 32 chunks to a token.
  static SDV_DEV int swz_codes(int t) {
    if (D == 64) return t >> 3 & 1;
    if (D == 128) {
      const int x = t >> 2 & 3;
      return ((x ^ x >> 1) & 1) << 1 | x >> 1;
    }
    if (D == 256) return (t >> 1 & 1) | (t >> 1 & 4);
    return 0;
  }

  // bf16: two units.  4 bits: one, its values as bf16, its keys as they are.
  struct Units {
    uint16_t k[2][TT * D], v[2][TT * D];
  };
  static constexpr int kValuesAt = 2 * TT * D * 2;   // bytes
  struct Unit4 {
    uint16_t v[1][TT * D];
    uint8_t k[TT * D / 2], ks[TT * DG];
  };
  struct Shared {
    alignas(1024) std::conditional_t<kFp4, Unit4, Units> kv;
    float ml[WT > 1 ? (WT - 1) * M * 2 : 1];
    int bad[2];                   // the unit has a block outside the pool
  };

  Shared& sh;
  const int wq, wt;
  int at_k[kPeriodK], at_v[kPeriodV];   // elements from the start of a side

  SDV_DEV Kernel(const AttnArgs& args, Shared& shared) : Base(args), sh(shared), wq(wave / WT), wt(wave % WT) {
#pragma unroll
    for (int i = 0; i < kPeriodK; ++i) at_k[i] = (wt * TW + l16) * D + ((i * 4 + g) ^ swz_k(l16)) * 8;
    const int row = 4 * g + (l16 >> 2);
#pragma unroll
    for (int i = 0; i < kPeriodV; ++i)
      at_v[i] = (wt * TW + row) * D + ((2 * i + ((l16 & 3) >> 1)) ^ swz_v(row)) * 8 + (l16 & 1) * 4;
  }

  SDV_DEV void begin(const Tile& t, int head) { Base::begin(t, head, wq * NT * 16, M); }

  // ---- loading a unit -----------------------------------------------------
  // Blocks are looked up a unit before they are used.  Where neighbouring
  // tokens that are loaded together lie in one block (its size a multiple of
  // kSpan), one scalar look-up and one address serve the wave, and lanes differ
  // by constants; else each piece has its own.
  struct Blocks {
    int of[kPieces];
  };
  SDV_DEV int piece(int j) const { return kFp4 ? min(j * 64 + lane, RW * kPer - 1) : j * 64 + lane; }
  SDV_DEV int row_of(int j) const { return wave * RW + piece(j) / kPer; }
  SDV_DEV int token_of(int u, int j) const { return min(u * TT + row_of(j), ctx - 1); }   // past the end: masked
  SDV_DEV int span_of(int u, int j) const {
    return min(u * TT + wave * RW + j * kSpan, (ctx - 1) / kSpan * kSpan);
  }
  SDV_DEV Blocks look_up(int u) const {
    Blocks b;
    if (kSpan > 0 && a.spans) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        b.of[j] = j < kSpans ? ((const ConstPtr)table)[block_of(span_of(u, j))] : b.of[0];
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) b.of[j] = table[block_of(token_of(u, j))];
      // Loads into registers that may still be on their way would have the
      // compiler wait for all loads where the paths meet again.
      if (!kFp4) __builtin_amdgcn_s_waitcnt(0x0f70);
    }
    return b;
  }
  SDV_DEV void note_bad(bool bad, int buf) {
    if (__builtin_expect(bad, 0)) sh.bad[buf] = 1;
  }

  // bf16: one side straight into LDS, a wave's 64 lanes one KB at a time.
  template <bool kValues>
  SDV_DEV void load_side(int u, int buf, const Blocks& b) {
    bool bad = false;
    const char* head = kValues ? v_head : k_head;
    const uint32_t to = __builtin_amdgcn_readfirstlane(
        lds_at(&sh) + (kValues ? kValuesAt : 0) + buf * (TT * D * 2) + wave * (RW * D * 2));
    if (a.spans) {
      const char* from = head + place(span_of(u, 0), __builtin_amdgcn_readfirstlane(b.of[0]), bad) * kRow;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int x = j * 64 + lane, swz = kValues ? swz_v(row_of(j)) : swz_k(row_of(j));
        const uint32_t off = x / CH * kRow + ((x % CH) ^ swz) * 16;
        if (a.once) load_to_lds<true>(from, off, to + j * 1024);
        else load_to_lds<false>(from, off, to + j * 1024);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int c = (j * 64 + lane) % CH, swz = kValues ? swz_v(row_of(j)) : swz_k(row_of(j));
        load_to_lds<false>(head + place(token_of(u, j), b.of[j], bad) * kRow + (c ^ swz) * 16, to + j * 1024);
      }
    }
    if (!kValues) note_bad(bad, buf);
  }

  // 4 bits: groups of 32 channels into registers, and from there into LDS.
  struct Codes {
    u32x4 k[kPieces], v[kPieces];
    uint32_t ks[kPieces], vs[kPieces];
    bool bad;
  };
  SDV_DEV void load_codes(int u, Codes& c, const Blocks& b) const {
    c.bad = false;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (kSpan > 0 && a.spans) {
        const uint64_t at = place(span_of(u, j), __builtin_amdgcn_readfirstlane(b.of[j]), c.bad) * DG;
        const uint32_t mine = min(lane, RW * kPer - 1);   // lanes past the wave's pieces stay in its block
        c.k[j] = ((const u32x4*)k_head + at)[mine];
        c.v[j] = ((const u32x4*)v_head + at)[mine];
        c.ks[j] = (ks_head + at)[mine];
        c.vs[j] = (vs_head + at)[mine];
      } else {
        const uint64_t at = place(token_of(u, j), b.of[j], c.bad) * DG + piece(j) % DG;
        c.k[j] = ((const u32x4*)k_head)[at];
        c.v[j] = ((const u32x4*)v_head)[at];
        c.ks[j] = ks_head[at];
        c.vs[j] = vs_head[at];
      }
    }
  }
  static SDV_DEV u32x4 turned(u32x4 w, int by) {   // element i ^ by
    if (by & 1) w = w.yxwz;
    if (by & 2) w = w.zwxy;
    return w;
  }
  static SDV_DEV u32x4 values(uint32_t codes, float scale) {
    const uint4 v = fp4_to_bf16(codes, scale);
    return u32x4{v.x, v.y, v.z, v.w};
  }
  SDV_DEV void put_codes(const Codes& c) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int x = j * 64 + lane;
      if (RW * DG % 64 != 0 && x >= RW * DG) continue;
      const int row = wave * RW + x / DG, q = x % DG;
      *(u32x4*)(sh.kv.k + row * kRow + (q ^ swz_codes(row)) * 16) = c.k[j];
      sh.kv.ks[row * DG + q] = (uint8_t)c.ks[j];
      // Eight neighbouring lanes write at a time: each begins at a chunk of its
      // group that lies in other banks than theirs.  (12 cycles a store, 20
      // where all begin at the first)
      const int turn = D == 256 ? q >> 1 : D == 128 ? q >> 1 : D == 64 ? row & 1 : 0;
      const u32x4 w = turned(c.v[j], turn);
      const float scale = fp4_scale(c.vs[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *(u32x4*)(sh.kv.v[0] + row * D + ((4 * q + (i ^ turn)) ^ swz_v(row)) * 8) = values(w[i], scale);
    }
    note_bad(c.bad, 0);
  }

  // ---- one unit -----------------------------------------------------------
  SDV_DEV u32x2 v_part(const uint16_t* v, int s, int d) const {   // tokens 16 s + 4 g .. + 3 of channel 16 d + l16
    const uint16_t* p = v + at_v[d % kPeriodV] + s * 16 * D + d / kPeriodV * kPeriodV * 16;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4*)p));
  }
  // Keys of tokens 16 i .. + 15 of the wave, as they lie in LDS.
  struct Keys {
    b16x8 as[kFp4 ? 1 : KS];
    uint32_t codes[kFp4 ? KS : 1];
    float scale[kFp4 ? DG : 1];
  };
  SDV_DEV void load_keys(int buf, int i, Keys& k) const {
    if constexpr (!kFp4) {
      const uint16_t* kk = sh.kv.k[buf];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        k.as[ks] = *(const b16x8*)(kk + at_k[ks % kPeriodK] + i * 16 * D + ks / kPeriodK * kPeriodK * 32);
    } else {
      const int row = wt * TW + i * 16 + l16;
      const uint8_t* from = sh.kv.k + row * kRow;
      if constexpr (D == 64) {
        const u32x2 w = *(const u32x2*)(from + ((g >> 1) ^ swz_codes(l16)) * 16 + (g & 1) * 8);
        k.codes[0] = w[0], k.codes[1] = w[1];
        k.scale[0] = fp4_scale(sh.kv.ks[row * DG + (g >> 1)]);
      } else if constexpr (kWide) {
#pragma unroll
        for (int x = 0; x < KS / 4; ++x) {
          const u32x4 w = *(const u32x4*)(from + ((KS / 4 * g + x) ^ swz_codes(l16)) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) k.codes[4 * x + e] = w[e];
          k.scale[x] = fp4_scale(sh.kv.ks[row * DG + KS / 4 * g + x]);
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          k.codes[ks] = *(const uint32_t*)(from + (4 * ks + g) * 4);
          k.scale[ks] = fp4_scale(sh.kv.ks[row * DG + ks]);
        }
      }
    }
  }
  static SDV_DEV b16x8 key(const Keys& k, int ks) {
    if constexpr (!kFp4) return k.as[ks];
    else return __builtin_bit_cast(b16x8, values(k.codes[ks], k.scale[kWide ? ks / 4 : ks]));
  }

  // S^T of a unit: the wave's tokens by its queries.
  SDV_DEV void scores(int buf, f32x4 (&s)[NS][NT]) const {
    Keys k[2];
    load_keys(buf, 0, k[0]);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if (i + 1 < NS) load_keys(buf, i + 1, k[(i + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);   // all requested before the first is waited for
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[i][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const b16x8 kf = key(k[i & 1], ks);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[i][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[nt][ks], s[i][nt], 0, 0, 0);
      }
    }
  }

  // Values of kRows rows of O^T at a time, so that one set is on its way while
  // another is multiplied, and the first while the weights are formed.
  static constexpr int kRows = NS >= 4 ? (ND % 4 == 0 ? 4 : 3) : ND <= 8 ? ND : ND % 8 == 0 ? 8 : 6;
  static_assert(ND % kRows == 0, "rows");
  SDV_DEV void load_values(const uint16_t* vv, int first, u32x2 (&vf)[kRows][NS]) const {
#pragma unroll
    for (int d = 0; d < kRows; ++d)
#pragma unroll
      for (int i = 0; i < NS; ++i) vf[d][i] = v_part(vv, i, first + d);
  }

  // Masks, weights and O^T of unit u, whose values are in vv; bad: it has a
  // block outside the pool.
  SDV_DEV void weigh(int u, uint16_t* vv, bool bad, f32x4 (&s)[NS][NT]) {
    u32x2 vf[2][kRows][NS];
    load_values(vv, 0, vf[0]);
    __builtin_amdgcn_sched_barrier(0);
    // the same for all waves, as is what follows from it
    const bool masked = bad || (u + 1) * TT > all_hi || u * TT < all_lo;
    uint64_t ok[2] = {~0ull, ~0ull};
    bool fault = false;   // values that are not finite beside masked weights
    if (masked) {
      this->mask(u * TT + wt * TW, s);
      if (__builtin_expect(bad, 0)) {
        ok[0] = this->mask_pool(u * TT + wt * TW, 0, M, s);
        if (NS > 4) ok[1] = this->mask_pool(u * TT + wt * TW, 4, M, s);
      }
      int odd = 0;
      for (int x = tid; x < TT * CH; x += kAttnThreads) {
        const u32x4 w = *(const u32x4*)(vv + x * 8);
        odd |= not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
      }
      fault = __syncthreads_or(odd) != 0;
    }
    this->move_maximum(s);
    u32x2 p[NT][NS];
    this->weights(s, p);
    if (__builtin_expect(fault, 0)) {
      // 0 * inf and 0 * NaN of masked tokens must not reach a sum: values that
      // are not finite are added here, for the queries that see their tokens,
      // and taken out before the product.
      add_faults(u, ok, vv);
      __syncthreads();
      for (int x = tid; x < TT * D; x += kAttnThreads)
        if ((vv[x] & 0x7F80u) == 0x7F80u) vv[x] = 0;
      __syncthreads();
      load_values(vv, 0, vf[0]);
    }
#pragma unroll
    for (int r = 0; r < ND / kRows; ++r) {
      if (r + 1 < ND / kRows) load_values(vv, (r + 1) * kRows, vf[(r + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < kRows; ++d)
#pragma unroll
        for (int i = 0; i < NS; i += 2)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            f32x4& to = o[r * kRows + d][nt];
            const u32x2 v0 = vf[r & 1][d][i];
            if constexpr (NS == 1) {
              to = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, v0),
                                                             __builtin_bit_cast(s16x4, p[nt][0]), to, 0, 0, 0);
            } else {
              const u32x2 v1 = vf[r & 1][d][i + 1];
              to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(b16x8, u32x4{v0[0], v0[1], v1[0], v1[1]}),
                  __builtin_bit_cast(b16x8, u32x4{p[nt][i][0], p[nt][i][1], p[nt][i + 1][0], p[nt][i + 1][1]}), to, 0,
                  0, 0);
            }
          }
    }
  }

  static SDV_DEV int not_finite(uint32_t w) {   // either half of a word
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
  }

  // Token by token, as this is rare and its code has to be small.  Infinities
  // and NaN outlast any weight, so none is needed.
  SDV_DEV void add_faults(int u, const uint64_t (&ok)[2], const uint16_t* vv) {
#pragma unroll 1
    for (int i = 0; i < TW; ++i) {
      const int row = wt * TW + i;
      if (!((i < 64 ? ok[0] : ok[1]) >> (i & 63) & 1)) continue;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool see = this->sees(u * TT + row, nt);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const int c = 2 * d + (g >> 1);
          const uint2 v = *(const uint2*)(vv + row * D + (c ^ swz_v(row)) * 8 + (g & 1) * 4);
          o[d][nt] += f32x4{fault_of(v.x << 16, see), fault_of(v.x & 0xFFFF0000u, see), fault_of(v.y << 16, see),
                            fault_of(v.y & 0xFFFF0000u, see)};
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  static SDV_DEV float fault_of(uint32_t bits, bool see) {
    return __uint_as_float(see && (bits & 0x7F800000u) == 0x7F800000u ? bits : 0u);
  }

  // ---- the end of a run's part of a tile ----------------------------------
  // Waves that took other tokens of the same queries are joined in LDS.
  SDV_DEV void join_waves() {
    float* ob = (float*)&sh.kv;                      // [WT - 1][M][D]
    float* mb = sh.ml;
    static_assert(((WT - 1) * M * D * 4) <= (int)sizeof(sh.kv), "join");
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
          for (int d = 0; d < ND; ++d) {
            o[d][nt] += *(const f32x4*)(from + ((d * 16 + 4 * g) ^ ((l16 & 7) << 2))) * f;
            if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // not all of them in registers at a time
          }
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
    if constexpr (kFp4) {
      // One unit is on its way into registers while another is computed.
      const int last = u + n - 1;
      Codes c;
      Blocks b = look_up(u);
      load_codes(u, c, b);
      b = look_up(min(u + 1, last));
      wait_all();
      for (int i = 0; i < n; ++i) {
        if (i > 0) __syncthreads();            // the last unit has been read by all
        put_codes(c);
        load_codes(min(u + i + 1, last), c, b);
        b = look_up(min(u + i + 2, last));
        __syncthreads();                       // this one is in LDS
        const bool bad = __builtin_amdgcn_readfirstlane(sh.bad[0]) != 0;
        f32x4 s[NS][NT];
        scores(0, s);
        weigh(u + i, sh.kv.v[0], bad, s);
      }
    } else {
      // Keys are asked for two units ahead of their use, values one and a half:
      // each side's buffer is given away as soon as all waves have read it, and
      // a wait leaves what is behind it on its way.  In the order of issue: keys
      // 0, values 0, keys 1, values 1, ...
      Blocks b1 = look_up(u), b2 = look_up(u + (n > 1));
      wait_all();   // for the queries, while the blocks are looked up
      load_side<false>(u, 0, b1);
      load_side<true>(u, 0, b1);
      b1 = b2;
      if (n > 1) load_side<false>(u + 1, 1, b1);
      for (int i = 0; i < n; ++i) {
        const bool more = i + 1 < n;
        if (i + 2 < n) b2 = look_up(u + i + 2);
        wait_loads(more ? 2 * kPieces : kPieces);   // keys i are here
        __syncthreads();                            // ... for all, and values i - 1 have been read
        const bool bad = __builtin_amdgcn_readfirstlane(sh.bad[i & 1]) != 0;
        if (more) load_side<true>(u + i + 1, (i + 1) & 1, b1);
        f32x4 s[NS][NT];
        scores(i & 1, s);
        wait_loads(more ? 2 * kPieces : 0);         // values i are here
        __syncthreads();                            // ... for all, and keys i have been read
        if (i + 2 < n) load_side<false>(u + i + 2, i & 1, b2);
        b1 = b2;
        weigh(u + i, sh.kv.v[i & 1], bad, s);
      }
    }
    __syncthreads();
  }
  // Until at most so many of the loads into LDS, the newest, are on their way
  // (other loads that the compiler issues in between only make it stricter).
  static SDV_DEV void wait_loads(int left) {
    static_assert(2 * kPieces <= 15, "the count's low bits");
    if (left == 0) __builtin_amdgcn_s_waitcnt(0x0f70);
    else if (left == kPieces) __builtin_amdgcn_s_waitcnt(0x0f70 | (kFp4 ? 0 : kPieces));
    else __builtin_amdgcn_s_waitcnt(0x0f70 | (kFp4 ? 0 : 2 * kPieces));
  }
};

// The tiles of a workgroup's run.
template <typename K>
SDV_DEV void run_tiles(const AttnArgs& a, typename K::Shared& sh) {
  const PlanHead& p = *a.head;
  // Neighbouring runs read the same tokens where a request has several tiles:
  // they go to the same eighth of the chip, which shares a cache.
  const int per = (int)gridDim.x / 8, w = (int)(blockIdx.x % 8) * per + (int)blockIdx.x / 8;
  if (!same_shape(p.shape, a.shape)) return;
  const long long quota = p.quota, total = p.total;
  long long at = w * quota;
  long long end = at + quota < total ? at + quota : total;
  if (at >= end) return;
  K k(a, sh);
  k.causal = p.causal != 0;
  k.window = p.window;
  k.turn = (int)(blockIdx.x / (gridDim.x / 2));
  const int n_tiles = p.n_tiles, lead = p.lead;
  // Where requests have several tiles, the one that begins in this run and ends
  // in another comes first: runs of a request are then at the same tokens at
  // about the same time, and more of them are found in the cache that they
  // share (16 requests with pieces of up to 512 rows, 8 key heads of 128: 226
  // us, 237 in the tiles' order).
  Start s = {};
  if (!a.once && w + 1 < (int)gridDim.x) s = uniform(a.starts[w + 1]);
  bool begins = s.off > lead && s.off - quota <= lead;
  if (begins) end -= s.off;
  else s = uniform(a.starts[w]);
  for (;;) {
    const Tile& t = s.tile;
    const long long room = end - at;
    const int left = lead + t.units - s.off, take = left < room ? left : (int)room;
    const int first = begins ? 0 : max(s.off - lead, 0), n = s.off + (begins ? 0 : take) - lead - first;
    if (n <= 0) {
      // no more than the tile's lead
    } else if (in_range(a, t)) {
      k.begin(t, s.head);
      k.units(t.u0 + first, n);
      // a part that begins its tile goes to the run's second place, others to its first
      k.end(n == t.units ? -1 : first == 0 ? 2 * w + 1 : 2 * w);
    } else if (threadIdx.x == 0) {
      atomicOr(a.status + t.req, SD_ST_BAD_INPUT);
    }
    if (begins) {
      if (at >= end) break;
      begins = false;
      s = uniform(a.starts[w]);
      continue;
    }
    at += take;
    if (at >= end) break;
    s.off = 0;
    if (++s.index == n_tiles) {
      s.index = 0;
      ++s.head;
    }
    s.tile = uniform(a.tiles[s.index]);
  }
}

// This kernel alone, in a trace, each on one set of inputs.  128 contexts of 1024
// to 16384 tokens, one row each, 32 heads on 8 of 128, bf16: 459 to 468 us for 2.9
// GB, 6.3 TB/s, bound by the memory.  Verify rows (up to 12) over 512 to 8192
// tokens: 276 to 284 us for 1.45 GB, 5.2 TB/s: the beginnings of tiles and the two
// products.  Pieces of prompts (16 requests, up to 512 rows), 0.18 Tflop: 258 to
// 261 us, 0.7 Pflop/s: of a SIMD's cycles the matrix cores work for 36 %, the
// vector units for 43 %, mostly one after the other.
template <int D, int NT, int WT, bool kFp4>
__global__ __launch_bounds__(kAttnThreads, 2) void k_attend(AttnArgs a) {
  using K = Kernel<D, NT, WT, kFp4>;
  __shared__ typename K::Shared sh;
  run_tiles<K>(a, sh);
}

template <bool kFp4>
int launch_attend(hipStream_t stream, int M, int W, const AttnArgs& a) {
  const dim3 grid((unsigned)W), block(kAttnThreads);
#define SDV_ATTN(...)                                                                            \
  do {                                                                                           \
    SDV_TRY_LAUNCH(sdv::launch(k_attend<__VA_ARGS__, kFp4>, grid, block, 0, stream, a));         \
    return SD_OK;                                                                                \
  } while (0)
#define SDV_ATTN_SMALL(D)                                                                        \
  case D:                                                                                        \
    if (M == 16) SDV_ATTN(D, 1, 4);                                                              \
    if (M == 32) SDV_ATTN(D, 1, 2);                                                              \
    if (M == 64) SDV_ATTN(D, 2, 2);                                                              \
    if (M == 128) SDV_ATTN(D, 2, 1);                                                             \
    break;
#define SDV_ATTN_LARGE(D)                                                                        \
  case D:                                                                                        \
    if (M == 32) SDV_ATTN(D, 1, 2);                                                              \
    if (M == 64) SDV_ATTN(D, 1, 1);                                                              \
    break;
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
