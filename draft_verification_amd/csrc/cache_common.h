// The paged key/value cache as its writers and readers see it.
#pragma once

#include "sdv_common.h"

namespace sdv {

// Memory of one side (keys or values): [n_blocks][n_kv][block_size][D] in
// bf16, or codes [n_blocks][n_kv][block_size][D / 2] bytes and scales
// [n_blocks][n_kv][block_size][D / 32] bytes.
struct Cache {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int n_kv, bs, n_blocks;
  double per_bs;   // 1 / bs
};

// Token (block, off) of head h, as an index of tokens.
SDV_DEV int64_t cache_token(const Cache& c, int64_t block, int h, int off) {
  return (block * c.n_kv + h) * c.bs + off;
}

// Slot s as a block and an offset in it; false where it is outside the cache.
// The block's number is below 2^31, so the quotient in fp64 is off by less than
// one; it saves a division of 64-bit integers, some hundred instructions.
SDV_DEV bool cache_slot(const Cache& c, int64_t s, int64_t* block, int* off) {
  if (s < 0 || s >= (int64_t)c.n_blocks * c.bs) return false;
  int64_t b = (int64_t)((double)s * c.per_bs);
  int64_t o = s - b * c.bs;
  if (o < 0) --b, o += c.bs;
  if (o >= c.bs) ++b, o -= c.bs;
  *block = b;
  *off = (int)o;
  return true;
}

// The scale byte (exponent + 127) of 32 channels whose largest magnitude has
// these bits: the smallest exponent e with max <= 7 * 2^e, at least -126.
// Every channel is then within half of the spacing of its level (6 is the
// last, and 7 half way to where 8 would be).  255 where one is not finite.
SDV_DEV uint32_t fp4_scale_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return 255u;
  const int e = (int)((bits + 0x1FFFFFu) >> 23) - 2;   // a mantissa over 1.75 carries
  return (uint32_t)(e < 1 ? 1 : e);
}
SDV_DEV float fp4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }   // 255: the conversions give NaN

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two channels rounded to bf16 (nearest even), the first in the low half.
SDV_DEV uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Eight channels of 4 bits, first in the lowest bits, as four words of bf16.
// Exact: a level has one bit behind its first, a scale none.
SDV_DEV uint4 fp4_to_bf16(uint32_t codes, float scale) {
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return o;
}
// ... and back: nearest level, ties to the even code, past the last level 6.
SDV_DEV uint32_t fp4_from_f32(const float (&x)[8], float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[0], x[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2], x[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4], x[5], scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6], x[7], scale, 3);
  return r;
}

}  // namespace sdv
