// Attention over a cache of 4 bits for a few queries to a tile.
//
// A wave takes 32 tokens of a unit for all of the tile's queries, so no wave
// needs what another has read: each has a ring of its own in LDS, which loads
// fill without passing through registers, several chunks ahead, and there is no
// barrier until the tile's end, where the waves are joined.  Both products are
// fed from the codes:
//  - keys: the lane that holds a row of the matrix instruction takes D / 4
//    neighbouring channels of its token, one read, one or two scales;
//  - values: which channel stands in which row of O^T is free.  Row r of step
//    d is channel ND r + d (ND = D / 16 steps), so a lane's row holds ND
//    neighbouring channels, for all steps together: one read of ND / 2 bytes
//    for each of the lane group's tokens, and words of two channels of a token
//    become words of two tokens of a channel by a byte permutation.
// (Values passed through LDS as bf16 cost 12 cycles of it for each KB stored and
// 10 for each read back: 128 contexts of 1024 to 16384 tokens, one row each, 8
// heads of 128: 177 us.  Codes straight into registers, a chunk ahead: 145 us.
// This form, alone in a trace: 133 us for 0.8 GB, 6.0 TB/s; the vector units,
// which turn codes into bf16 for both products, are busy for 58 % of it.)
#pragma once

#include "attend_kernel.h"

namespace sdv {
namespace attn {

template <int D, int NT>
struct Direct : Queries<D, NT, 2, true, true, 1, 4> {
  static constexpr int M = NT * 16, TT = 128, TW = 32, NS = 2;
  using Base = Queries<D, NT, NS, true, true, 1, 4>;
  using Base::a, Base::tid, Base::lane, Base::wave, Base::l16, Base::g;
  using Base::q0, Base::queries, Base::ctx, Base::row0, Base::h, Base::table;
  using Base::k_head, Base::v_head, Base::ks_head, Base::vs_head;
  using Base::qf, Base::o, Base::m, Base::l, Base::all_hi, Base::all_lo;
  using Base::KS, Base::ND, Base::DG, Base::kRow, Base::block_of, Base::place;
  static constexpr int KW = KS / 4 > 0 ? KS / 4 : 1;   // scales of a lane's keys
  static constexpr int VW = ND / 8 > 0 ? ND / 8 : 1;   // words of its values of a token
  static_assert(D == 64 || D == 128 || D == 256, "neighbouring channels share scales");

  // A chunk of 32 tokens: keys and values as they lie in the cache (a token's
  // pieces of 16 bytes of keys at c ^ swizzle, so that the tokens that one read
  // takes lie in different banks), then the scales of both.
  static constexpr int kSideBytes = TW * kRow, kScaleBytes = TW * DG;
  static constexpr int kChunk = 2 * kSideBytes + 2 * kScaleBytes;
  static constexpr int kLoads = kSideBytes / 1024;                    // of a side
  static constexpr int kScaleLoads = (2 * kScaleBytes + 255) / 256;   // of both
  static constexpr int kRing = D == 256 ? 2 : 4;
  static constexpr int kOps = 2 * kLoads + kScaleLoads;               // loads of a chunk
  static_assert(kOps * (kRing - 1) <= 15, "the count's low bits");

  struct Shared {
    union {
      alignas(1024) uint8_t ring[4][kRing][kChunk];
      f32x4 o[2][NT][ND][64];     // two waves' sums, as their lanes hold them
    };
    float2 ml[2][NT][64];
  };
  Shared& sh;

  SDV_DEV Direct(const AttnArgs& args, Shared& shared) : Base(args), sh(shared) {}
  SDV_DEV void begin(const Tile& t, int head) { Base::begin(t, head, 0, M); }

  // Row r = 4 g + e of the matrix instruction is token 4 e + g of each 16: one
  // read of values then takes four neighbouring tokens.
  static SDV_DEV int token_of_row(int r) { return 4 * (r & 3) + (r >> 2); }
  static SDV_DEV int swz(int t) {
    return D == 64 ? t >> 3 & 1 : D == 128 ? t >> 2 & 3 : (t >> 2 & 1) | (t >> 3 & 1) << 2;
  }
  SDV_DEV int first_of(int u) const { return u * TT + wave * TW; }

  // Requests a chunk; says whether a block is outside the pool.
  SDV_DEV bool load(int u, int slot) const {
    bool bad = false;
    uint64_t at[2];   // the cache holds 16 neighbouring tokens in one block
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int tok = min(first_of(u) + 16 * s, (ctx - 1) / 16 * 16);   // past the end: masked
      at[s] = place(tok, ((const ConstPtr)table)[block_of(tok)], bad);
    }
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds_at(sh.ring[wave][slot]));
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int x = j * 1024 + lane * 16, t = x / kRow, c = x % kRow / 16;
      const uint32_t ko = t % 16 * kRow + (c ^ swz(t % 16)) * 16, vo = t % 16 * kRow + c * 16;
      if constexpr (kLoads == 1) {
        const uint64_t from = (lane < 32 ? at[0] : at[1]) * kRow;
        load_to_lds<true>(k_head + from + ko, to);
        load_to_lds<true>(v_head + from + vo, to + kSideBytes);
      } else {
        const uint64_t from = at[j / (kLoads / 2)] * kRow;
        load_to_lds<true>(k_head + from, ko, to + j * 1024);
        load_to_lds<true>(v_head + from, vo, to + kSideBytes + j * 1024);
      }
    }
#pragma unroll
    for (int j = 0; j < kScaleLoads; ++j) {
      const int x = (j * 64 + lane) * 4, side = x / kScaleBytes, y = x % kScaleBytes;   // bytes
      const uint8_t* from = (side ? vs_head : ks_head) + (y < kScaleBytes / 2 ? at[0] * DG : at[1] * DG) +
                            y % (kScaleBytes / 2);
      if (side < 2) load_word_to_lds(from, to + 2 * kSideBytes + j * 256);
    }
    return bad;
  }

  struct Keys {
    uint32_t codes[KS];
    float scale[KW];
  };
  SDV_DEV void load_keys(const uint8_t* chunk, int s, Keys& k) const {
    const int t = token_of_row(l16);
    const uint8_t* codes = chunk + (16 * s + t) * kRow;
    const uint8_t* scales = chunk + 2 * kSideBytes + (16 * s + t) * DG;
    if constexpr (KS == 2) {
      const u32x2 w = *(const u32x2*)(codes + ((g >> 1) ^ swz(t)) * 16 + (g & 1) * 8);
      k.codes[0] = w[0], k.codes[1] = w[1];
      k.scale[0] = fp4_scale(scales[g >> 1]);
    } else {
#pragma unroll
      for (int x = 0; x < KW; ++x) {
        const u32x4 w = *(const u32x4*)(codes + ((KW * g + x) ^ swz(t)) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) k.codes[4 * x + i] = w[i];
        k.scale[x] = fp4_scale(scales[KW * g + x]);
      }
    }
  }
  struct Values {
    uint32_t v[2][4][VW], scale[2][4];
  };
  SDV_DEV void load_values(const uint8_t* chunk, Values& c) const {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * s + 4 * e + g;
        const uint8_t* from = chunk + kSideBytes + t * kRow + l16 * (ND / 2);
        if constexpr (ND == 4) c.v[s][e][0] = *(const uint16_t*)from;
        else if constexpr (ND == 8) c.v[s][e][0] = *(const uint32_t*)from;
        else {
          const u32x2 w = *(const u32x2*)from;
          c.v[s][e][0] = w[0], c.v[s][e][1] = w[1];
        }
        c.scale[s][e] = chunk[2 * kSideBytes + kScaleBytes + t * DG + l16 * ND / 32];
      }
  }

  static SDV_DEV uint32_t pair(uint32_t codes, float scale, int sel) {
    switch (sel) {
      case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
      case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
      case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
      default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    }
  }

  // Whether some query of the tile does not see all of a chunk's tokens.
  SDV_DEV bool cut_by_mask(int first) const { return first + TW > all_hi || first < all_lo; }

  // bad: the chunk has a block outside the pool.  Says whether values that are
  // not finite stood beside masked weights: add_faults has to follow.
  SDV_DEV bool unit(int u, const uint8_t* chunk, bool bad) {
    const int first = first_of(u);
    Keys k[2];
    load_keys(chunk, 0, k[0]);
    load_keys(chunk, 1, k[1]);
    f32x4 s[NS][NT];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[i][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 w = fp4_to_bf16(k[i].codes[ks], k[i].scale[ks / 4]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          s[i][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b16x8, w), qf[nt][ks], s[i][nt], 0, 0, 0);
      }
    }
    Values c;
    load_values(chunk, c);
    bool fault = false;
    if (bad || cut_by_mask(first)) {
      this->mask(first, s);
      if (__builtin_expect(bad, 0)) this->mask_pool(first, 0, M, s);
      bool odd = false;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= c.scale[i][e] >= kFirstFault;
      fault = __ballot(odd) != 0;
      if (__builtin_expect(fault, 0)) take_out_faults(c);
    }
    this->move_maximum(s);
    u32x2 p[NT][NS];
    this->weights(s, p);
#pragma unroll
    for (int j = 0; j < ND / 2; ++j) {   // rows of channels 2 j and 2 j + 1 of the lane's
      uint32_t w[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = pair(c.v[i][e][j / 4], fp4_scale(c.scale[i][e]), j % 4);
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        const uint32_t halves = odd ? 0x07060302u : 0x05040100u;   // of two tokens
        const u32x4 v = {__builtin_amdgcn_perm(w[0][1], w[0][0], halves), __builtin_amdgcn_perm(w[0][3], w[0][2], halves),
                         __builtin_amdgcn_perm(w[1][1], w[1][0], halves), __builtin_amdgcn_perm(w[1][3], w[1][2], halves)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          o[2 * j + odd][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(b16x8, v),
              __builtin_bit_cast(b16x8, u32x4{p[nt][0][0], p[nt][0][1], p[nt][1][0], p[nt][1][1]}), o[2 * j + odd][nt], 0,
              0, 0);
      }
    }
    return fault;
  }

  // Bit 0 of each of eight codes that its scale takes past the largest bf16: by
  // 2^126 the levels from 4 on, by 2^127 those from 2 on, all (to NaN) by 255.
  static constexpr uint32_t kFirstFault = 253;
  static SDV_DEV uint32_t faults(uint32_t codes, uint32_t byte) {
    const uint32_t x = byte == 255u ? ~0u : byte == 254u ? codes >> 2 : byte == 253u ? codes >> 2 & codes >> 1 : 0u;
    return x & 0x11111111u;
  }

  // Values that are not finite beside masked weights become zeros before the
  // product ...
  static SDV_DEV void take_out_faults(Values& c) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int x = 0; x < VW; ++x) c.v[i][e][x] &= ~(faults(c.v[i][e][x], c.scale[i][e]) * 15u);
        c.scale[i][e] = c.scale[i][e] == 255u ? 0u : c.scale[i][e];
      }
  }
  // ... and are added to the sums of the queries that see them, behind the last
  // unit: they outlast any weight, and the sums' registers are the only ones
  // that this rare path finds in use.  This lane's sums are of channels
  // ND (4 g + e) + d.
  SDV_DEV void add_faults(int u) {
    const int first = first_of(u);
    bool bad = false;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int tok = min(first + 16 * s, ctx - 1);
      place(tok, table[block_of(tok)], bad);
    }
    if (!bad && !cut_by_mask(first)) return;
#pragma unroll 1
    for (int i = 0; i < TW; ++i) {
      const int tok = first + i;
      if (tok >= ctx) break;
      bool out = false;
      const uint64_t at = place(tok, __builtin_amdgcn_readfirstlane(table[block_of(tok)]), out);
      if (out) continue;
      const uint8_t* scales = vs_head + at * DG;
      const char* codes = v_head + at * kRow;
      int mine = 4 * g;
      asm volatile("" : "+v"(mine));   // addresses are formed here, not kept in registers throughout
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t byte = scales[(uint32_t)(ND * (mine + e) / 32)];
#pragma unroll
        for (int d = 0; d < ND; d += 4) {
          const uint32_t w = *(const uint16_t*)(codes + (uint32_t)((mine + e) * (ND / 2) + d / 2));   // four channels
          const uint32_t fault = faults(w, byte);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t bits = byte == 255u ? 0x7FC00000u : 0x7F800000u | (w >> (4 * y + 3) & 1) << 31;
            const float x = fault >> 4 * y & 1 ? __uint_as_float(bits) : 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[d + y][nt][e] += this->sees(tok, nt) ? x : 0.f;
            __builtin_amdgcn_sched_barrier(0);   // rare: few registers, not speed
          }
        }
      }
    }
  }

  // Until at most so many chunks, the newest, are on their way; reads of LDS
  // stay on their side of it, and those before it are done.
  static SDV_DEV void wait_chunks(int left) {
    if (left == 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    else if (left == 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kOps) : "memory");
    else if (left == 2) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kRing > 2 ? 2 * kOps : 0) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kRing > 3 ? 3 * kOps : 0) : "memory");
  }

  // Units [u, u + n).  A wave waits for its own loads alone: it reads what it
  // has requested, and asks for a chunk again when it has read the one that
  // lies in its place.
  SDV_DEV void units(int u, int n) {
    uint32_t bad = 0;             // a bit for each place of the ring
    int fault0 = n, fault1 = 0;   // the units that have faults are in [fault0, fault1)
    Base::wait_all();
    __syncthreads();              // its sums, which lay in the ring, have been read
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i)
      if (i < n) bad |= (uint32_t)load(u + i, i) << i;
    for (int i = 0; i < n; ++i) {
      const int next = i + kRing - 1, slot = i % kRing;
      // Turn by turn with the CU's other workgroup, of which the older one would
      // come first throughout and end a quarter earlier (128 contexts of 1024 to
      // 16384 tokens, one row each, 8 heads of 128: 139 us, 143 without).
      if ((i & 1) == this->turn) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
      if (next < n) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the place has been read
        const uint32_t bit = 1u << next % kRing;
        bad = load(u + next, next % kRing) ? bad | bit : bad & ~bit;
      }
      wait_chunks(min(kRing - 1, n - 1 - i));
      const bool fault = unit(u + i, sh.ring[wave][slot], (bad >> slot & 1) != 0);
      fault0 = fault ? min(fault0, i) : fault0;
      fault1 = fault ? i + 1 : fault1;
    }
#pragma unroll 1
    for (int i = fault0; i < fault1; ++i) add_faults(u + i);
  }

  // Waves 2 and 3 into 0 and 1, then 1 into 0.
  SDV_DEV void join_waves() {
#pragma unroll
    for (int half = 2; half > 0; half >>= 1) {
      __syncthreads();                             // what was here has been read
      if (wave >= half && wave < 2 * half) {
        const int to = wave - half;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int d = 0; d < ND; ++d) sh.o[to][nt][d][lane] = o[d][nt];
          sh.ml[to][nt][lane] = make_float2(m[nt], l[nt]);
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 ml = sh.ml[wave][nt][lane];
          const float top = fmaxf(m[nt], ml.x), ref = top == -__builtin_huge_valf() ? 0.f : top;
          const float f = fast_exp2(m[nt] - ref), x = fast_exp2(ml.x - ref);
          m[nt] = top;
          l[nt] = l[nt] * f + ml.y * x;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            o[d][nt] = o[d][nt] * f + sh.o[wave][nt][d][lane] * x;
            if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // not all of them in registers at a time
          }
        }
      }
    }
  }

  SDV_DEV void end(int slot) {                       // slot < 0: the tile is whole
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt] = sum_over_groups(l[nt]);
    join_waves();
    if (wave > 0) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = nt * 16 + l16, qi = q0 + col;
      if (qi >= queries) continue;
      if (slot < 0) {
        const int i = qi / a.group, head = h * a.group + qi - i * a.group;
        const float inv = l[nt] == 0.f ? 0.f : 1.f / l[nt];
        uint16_t* to = a.out + (int64_t)(row0 + i) * a.ld_out + (int64_t)head * D + 4 * g * ND;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int d = 0; d < ND; d += 4)
            *(uint2*)(to + e * ND + d) = make_uint2(pack_bf16(o[d][nt][e] * inv, o[d + 1][nt][e] * inv),
                                                    pack_bf16(o[d + 2][nt][e] * inv, o[d + 3][nt][e] * inv));
        if (a.lse && g == 0)
          a.lse[(int64_t)(row0 + i) * a.n_q + head] =
              l[nt] == 0.f ? -__builtin_huge_valf() : (m[nt] + __log2f(l[nt])) * 0.69314718055994531f;
      } else {
        float* to = a.part + ((int64_t)slot * M + col) * D + 4 * g * ND;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int d = 0; d < ND; d += 4)
            *(f32x4*)(to + e * ND + d) = f32x4{o[d][nt][e], o[d + 1][nt][e], o[d + 2][nt][e], o[d + 3][nt][e]};
        if (g == 0) a.ml[(int64_t)slot * M + col] = make_float2(m[nt], l[nt]);
      }
    }
  }
};

template <int D, int NT>
__global__ __launch_bounds__(kAttnThreads, 2) void k_attend_direct(AttnArgs a) {
  using K = Direct<D, NT>;
  __shared__ typename K::Shared sh;
  run_tiles<K>(a, sh);
}

}  // namespace attn
}  // namespace sdv
