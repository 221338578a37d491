// sd_qk_rope, sd_cache_append and sd_cache_read: what happens to the heads of
// queries, keys and values between the projection and attention.
//
// A head x of D channels becomes y = x * rsqrt(mean(x^2) + eps) * w, and its
// first rot channels, in pairs (a, b), become (a cos - b sin, b cos + a sin)
// with the angle pos * inv_freq[pair].  Position times frequency is far
// outside fp32 for long contexts (10^6 radians leave 0.06 of resolution), so
// the angle is formed in fp64, in turns, and only its fraction goes to fp32.
// Everything else is fp32 and rounded once.
//
// Every channel is read once and written once: HBM bounds large calls, the
// chain position -> angle -> product small ones.
#include "cache_common.h"
#include "sdv_host.h"

namespace {

using sdv::Cache;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxHead = 256;
constexpr double kTurn = 0.15915494309189533577;   // 1 / (2 pi)

struct HeadArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_out;
  long long ld_q, ld_k, ld_v, ld_qo, ld_ko;   // elements between rows
  const int32_t* pos;
  const int64_t* slot;
  const float* wq;
  const float* wk;
  const float* inv_freq;
  Cache cache;
  float eps, per_D;   // 1 / D
  int n_rows, n_q, n_kv, n_v, D, rot;
  int lanes;   // per head, a power of two
  int iters;   // steps of 64 / lanes heads that a wave takes
  int parts;   // waves per row
};

// Eight channels as a lane holds them: four from `lo` on and four from `hi`.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <bool kStream, typename V>
SDV_DEV V load_vec(const V* p) {
  return kStream ? __builtin_nontemporal_load(p) : *p;
}
template <bool kStream>
SDV_DEV void load_runs(const uint16_t* p, int lo, int hi, float (&x)[8]) {
  const u32x2 a = load_vec<kStream>((const u32x2*)(p + lo)), b = load_vec<kStream>((const u32x2*)(p + hi));
  x[0] = sdv::bf16lo(a[0]), x[1] = sdv::bf16hi(a[0]), x[2] = sdv::bf16lo(a[1]), x[3] = sdv::bf16hi(a[1]);
  x[4] = sdv::bf16lo(b[0]), x[5] = sdv::bf16hi(b[0]), x[6] = sdv::bf16lo(b[1]), x[7] = sdv::bf16hi(b[1]);
}
template <bool kStream>
SDV_DEV void load_runs(const float* p, int lo, int hi, float (&x)[8]) {
  const f32x4 a = load_vec<kStream>((const f32x4*)(p + lo)), b = load_vec<kStream>((const f32x4*)(p + hi));
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
SDV_DEV void store_runs(uint16_t* p, int lo, int hi, const float (&x)[8]) {
  *(uint2*)(p + lo) = make_uint2(sdv::pack_bf16(x[0], x[1]), sdv::pack_bf16(x[2], x[3]));
  *(uint2*)(p + hi) = make_uint2(sdv::pack_bf16(x[4], x[5]), sdv::pack_bf16(x[6], x[7]));
}
SDV_DEV void store_runs(float* p, int lo, int hi, const float (&x)[8]) {
  *(float4*)(p + lo) = make_float4(x[0], x[1], x[2], x[3]);
  *(float4*)(p + hi) = make_float4(x[4], x[5], x[6], x[7]);
}

// A lane gets the value of lane ^ 1, lane ^ 2; of 8, of 16 mirrored.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;
template <int kFrom>
SDV_DEV float other(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kFrom, 0xF, 0xF, true));
}
// Over the `lanes` lanes (1 to 32) of each group, within the vector unit: an
// exchange through LDS takes longer than all else in a step.
SDV_DEV float sum_over_lanes(float v, int lanes) {
  if (lanes > 1) v += other<kXor1>(v);
  if (lanes > 2) v += other<kXor2>(v);
  if (lanes > 4) v += other<kMirror8>(v);
  if (lanes > 8) v += other<kMirror16>(v);
  if (lanes > 16) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  return v;
}

// Where keys and values go.
enum { kToRows = 0, kToBf16 = 1, kToFp4 = 2 };

// A wave takes `iters` steps of one row's heads, 64 / lanes heads at a time,
// D / 8 lanes of a group with eight channels each.  Lane c of a rotated head
// has four pairs: with the halves paired, channels 4c.. and rot/2 + 4c..; with
// neighbours paired, 8c.. ; so its four angles serve all heads of the row.
// Into rows nothing but rows is read, and streaming loads win (16384 rows of 40
// heads of 128: 53 us, 61 us with cached ones); into the cache they make no
// difference (8192 rows of 80 heads into bf16: 68 us both ways).
// Bound by the memory and the vector units where calls are large: those rows
// move at 4.8 TB/s, into bf16 at 4.4.  Into 4 bits the vector units alone bound
// it (8192 rows of 16 heads: 18 us for 37 MB).  A few rows: 3.2 us, the chain
// above.
template <typename T, int kTo, bool kNeighbours>
__global__ __launch_bounds__(kThreads) void k_heads(HeadArgs a) {
  // Channels in their order, for groups of 32: only 4 bits need them.
  __shared__ float order[kTo == kToFp4 ? kThreads * 8 : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const unsigned job = blockIdx.x * kWaves + wave;
  const int row = (int)(job / (unsigned)a.parts), part = (int)(job - (unsigned)row * (unsigned)a.parts);
  if (row >= a.n_rows) return;
  const int pos = a.pos ? a.pos[row] : 0;
  if (pos < 0) return;
  constexpr bool kStream = kTo == kToRows;
  // Into 4 bits, where the arithmetic counts, values go a way of their own:
  // their lanes hold neighbours, and a step of nothing but values has no norm
  // and no exchange.  (Into bf16 the branches cost more: 76 us, 69 without.)
  constexpr bool kApart = kTo == kToFp4;
  const int c = lane & (a.lanes - 1), group = lane / a.lanes, groups = 64 / a.lanes;
  const int heads = a.n_q + a.n_kv + a.n_v;
  const bool in = c * 8 < a.D, turned = c * 8 < a.rot;
  const int lo = turned && !kNeighbours ? 4 * c : 8 * c;
  const int hi = turned && !kNeighbours ? a.rot / 2 + 4 * c : 8 * c + 4;

  int64_t block = -1;
  int off = 0;
  if constexpr (kTo != kToRows) {
    if (!sdv::cache_slot(a.cache, a.slot[row], &block, &off)) block = -1;
  }
  const int first = part * a.iters * groups + group;
  auto at = [&](int h) -> const T* {
    if (h < a.n_q) return (const T*)a.q + row * a.ld_q + (int64_t)h * a.D;
    if (h < a.n_q + a.n_kv) return (const T*)a.k + row * a.ld_k + (int64_t)(h - a.n_q) * a.D;
    return (const T*)a.v + row * a.ld_v + (int64_t)(h - a.n_q - a.n_kv) * a.D;
  };
  const int first_v = a.n_q + a.n_kv;
  auto load = [&](int h, float (&to)[8]) {
    const bool apart = kApart && h >= first_v;
    if (in && h < heads) load_runs<kStream>(at(h), apart ? 8 * c : lo, apart ? 8 * c + 4 : hi, to);
  };
  float x[8] = {}, next[8] = {};
  load(first, next);   // while the angles are formed

  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {};
  if (turned) {
    const float4 f = *(const float4*)(a.inv_freq + 4 * c);
    const float fr[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double t = (double)pos * ((double)fr[i] * kTurn);
      sincospif((float)(2.0 * (t - rint(t))), &sn[i], &cs[i]);
    }
  }
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.f;
  if (in && a.wq) load_runs<false>(a.wq, lo, hi, wq);
  if (in && a.wk) load_runs<false>(a.wk, lo, hi, wk);

  for (int it = 0; it < a.iters; ++it) {
    const int h = first + it * groups;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = next[i];
    const bool live = h < heads;
    if (it + 1 < a.iters) load(h + groups, next);
    const bool is_q = h < a.n_q, is_v = h >= first_v;
    const bool some = !kApart || __ballot(!is_v) != 0;   // heads of the step that are no values
    if (some && (a.wq || a.wk)) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[i] * x[i];
      s = sum_over_lanes(s, a.lanes);
      const float r = rsqrtf(s * a.per_D + a.eps);
      if (!is_v && (is_q ? a.wq : a.wk)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (is_q ? wq[i] : wk[i]);
      }
    }
    if (turned && !is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ia = kNeighbours ? 2 * i : i, ib = kNeighbours ? 2 * i + 1 : 4 + i;
        const float u = x[ia], w = x[ib];
        x[ia] = u * cs[i] - w * sn[i];
        x[ib] = w * cs[i] + u * sn[i];
      }
    }
    if (is_q) {
      if (live && in) store_runs((T*)a.q_out + row * a.ld_qo + (int64_t)h * a.D, lo, hi, x);
      if constexpr (kTo != kToFp4) continue;
    }
    const int hk = is_v ? h - a.n_q - a.n_kv : h - a.n_q;
    if constexpr (kTo == kToRows) {
      if (live && in) store_runs((T*)a.k_out + row * a.ld_ko + (int64_t)hk * a.D, lo, hi, x);
    } else if constexpr (kTo == kToBf16) {
      if (live && in && block >= 0)
        store_runs((uint16_t*)(is_v ? a.cache.v : a.cache.k) + sdv::cache_token(a.cache, block, hk, off) * a.D,
                   lo, hi, x);
    } else {
      // Keys through LDS into the channels' order: lane c then has 8c .. 8c + 7,
      // and four neighbours a group of 32.  A wave's own part: its LDS
      // accesses are done in order, so no barrier is needed.
      if (some && !kNeighbours && a.rot > 0) {
        float* o = order + wave * 512 + group * a.lanes * 8;
        *(float4*)(o + (is_v ? 8 * c : lo)) = make_float4(x[0], x[1], x[2], x[3]);
        *(float4*)(o + (is_v ? 8 * c + 4 : hi)) = make_float4(x[4], x[5], x[6], x[7]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const float4 y = *(const float4*)(o + 8 * c), z = *(const float4*)(o + 8 * c + 4);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();   // the next step's stores stay behind these loads
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w, x[4] = z.x, x[5] = z.y, x[6] = z.z, x[7] = z.w;
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;   // ordered as the magnitudes, NaN last
        top = top > b ? top : b;
      }
      top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, kXor1, 0xF, 0xF, true));
      top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, kXor2, 0xF, 0xF, true));
      const uint32_t byte = sdv::fp4_scale_byte(top);
      const uint32_t codes = byte == 255u ? 0u : sdv::fp4_from_f32(x, sdv::fp4_scale(byte));
      if (live && in && !is_q && block >= 0) {
        const int64_t t = sdv::cache_token(a.cache, block, hk, off);
        ((uint32_t*)(is_v ? a.cache.v : a.cache.k))[t * (a.D / 8) + c] = codes;
        if ((c & 3) == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[t * (a.D / 32) + (c >> 2)] = (uint8_t)byte;
      }
    }
  }
}

struct ReadArgs {
  const int64_t* slot;
  Cache cache;
  void* k_out;
  void* v_out;
  long long ld_k, ld_v;
  int n_rows, D;
  int vecs;   // of eight channels per row, both sides
};

// A workgroup per row, a thread per eight channels of its keys or values: the
// row's slot is taken apart once.  8192 rows of 16 heads of 128 from 4 bits to
// bf16: 12 us for 37 MB, 3.1 TB/s (13 us with a thread's row found from its
// number), bound by loads in a chain: slot, then codes.
template <typename T, bool kFp4>
__global__ __launch_bounds__(kThreads) void k_cache_read(ReadArgs a) {
  const int row = blockIdx.x;
  int64_t block;
  int off;
  if (!sdv::cache_slot(a.cache, a.slot[row], &block, &off)) return;
  for (int i = threadIdx.x; i < a.vecs; i += blockDim.x) {
    const bool is_v = i >= a.vecs / 2;
    const int e = is_v ? i - a.vecs / 2 : i;
    const int h = (int)((unsigned)e / (unsigned)(a.D / 8)), c = e - h * (a.D / 8);
    const int64_t t = sdv::cache_token(a.cache, block, h, off);
    const void* side = is_v ? a.cache.v : a.cache.k;
    uint4 w;
    if constexpr (kFp4) {
      const uint8_t byte = (is_v ? a.cache.v_scale : a.cache.k_scale)[t * (a.D / 32) + (c >> 2)];
      w = sdv::fp4_to_bf16(((const uint32_t*)side)[t * (a.D / 8) + c], sdv::fp4_scale(byte));
    } else {
      w = ((const uint4*)side)[t * (a.D / 8) + c];
    }
    T* out = (is_v ? (T*)a.v_out + row * a.ld_v : (T*)a.k_out + row * a.ld_k) + (int64_t)h * a.D + 8 * c;
    if constexpr (sizeof(T) == 2) {
      *(uint4*)out = w;
    } else {
      *(float4*)out = make_float4(sdv::bf16lo(w.x), sdv::bf16hi(w.x), sdv::bf16lo(w.y), sdv::bf16hi(w.y));
      *(float4*)(out + 4) = make_float4(sdv::bf16lo(w.z), sdv::bf16hi(w.z), sdv::bf16lo(w.w), sdv::bf16hi(w.w));
    }
  }
}

// Waves that fill the chip several times over; past them a wave takes more of
// its row's heads, whose angles it forms once.  With 16384 and 8192 of them,
// 8192 rows of 64 heads and 16 into a bf16 cache take 69 and 76 us, and 16
// heads a row into 4 bits, with their reading back, 44 and 41 us.
constexpr long long kEnoughWaves = 16384, kEnoughWavesFp4 = 8192;

int run_heads(hipStream_t stream, HeadArgs& a, int dtype, int to, bool neighbours) {
  const int heads = a.n_q + a.n_kv + a.n_v;
  a.per_D = 1.0f / a.D;
  a.lanes = 1;
  while (a.lanes * 8 < a.D) a.lanes *= 2;
  if (to == kToFp4 && a.lanes < 4) a.lanes = 4;
  const int steps = (heads + 64 / a.lanes - 1) / (64 / a.lanes);
  const long long waves = to == kToFp4 ? kEnoughWavesFp4 : kEnoughWaves;
  const long long iters = ((long long)a.n_rows * steps + waves - 1) / waves;
  a.iters = (int)(iters < steps ? iters : steps);
  a.parts = (steps + a.iters - 1) / a.iters;
  const long long groups = ((long long)a.n_rows * a.parts + kWaves - 1) / kWaves;
  if (groups * kThreads > 0xFFFFFFFFll) return SD_EUNSUPPORTED;
  const dim3 grid((unsigned)groups);
#define SDV_HEADS(T, TO)                                                                                       \
  do {                                                                                                         \
    if (neighbours) SDV_TRY_LAUNCH(sdv::launch(k_heads<T, TO, true>, grid, dim3(kThreads), 0, stream, a));     \
    else SDV_TRY_LAUNCH(sdv::launch(k_heads<T, TO, false>, grid, dim3(kThreads), 0, stream, a));               \
    return SD_OK;                                                                                              \
  } while (0)
  if (dtype == SD_DTYPE_BF16) {
    if (to == kToRows) SDV_HEADS(uint16_t, kToRows);
    if (to == kToBf16) SDV_HEADS(uint16_t, kToBf16);
    SDV_HEADS(uint16_t, kToFp4);
  }
  if (to == kToRows) SDV_HEADS(float, kToRows);
  if (to == kToBf16) SDV_HEADS(float, kToBf16);
  SDV_HEADS(float, kToFp4);
#undef SDV_HEADS
}

bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }

// Row pieces of n heads: a pointer, a leading dimension that holds them.
bool bad_rows(const void* p, long long ld, int n, int D) {
  return n > 0 && (!p || off16(p) || ld < (long long)n * D || ld % 8 != 0);
}
sdv::Span rows_span(const void* p, int n_rows, int n, int D, long long ld, int es) {
  return sdv::span(p, n_rows, (long long)n * D * es, ld * es);
}

int check_heads(int n_rows, int D, int dtype, int n_q, int n_kv, float eps, const float* wq, const float* wk,
                const float* inv_freq, int rot, int interleaved, const int32_t* pos) {
  if (n_rows < 0 || D < 8 || D % 8 != 0 || n_q < 0 || n_kv < 0) return SD_EINVAL;
  if (dtype != SD_DTYPE_F32 && dtype != SD_DTYPE_BF16) return SD_EINVAL;
  if (rot < 0 || rot > D || rot % 8 != 0 || (interleaved != 0 && interleaved != 1)) return SD_EINVAL;
  if (rot > 0 && (!inv_freq || (n_rows > 0 && !pos) || off16(inv_freq))) return SD_EINVAL;
  if ((wq || wk) && !(eps >= 0.0f && eps < __builtin_huge_valf())) return SD_EINVAL;
  if ((wq && off16(wq)) || (wk && off16(wk))) return SD_EINVAL;
  if (D > kMaxHead || n_q > SD_MAX_HEADS || n_kv > SD_MAX_HEADS) return SD_EUNSUPPORTED;
  return SD_OK;
}

// The four arrays of a cache: how many bytes each holds.
int check_cache(int type, int n_kv, int D, int bs, int n_blocks, const void* k, const void* v, const void* ks,
                const void* vs, sdv::Span (&spans)[4]) {
  if (type != SD_CACHE_BF16 && type != SD_CACHE_FP4) return SD_EINVAL;
  if (n_kv < 1 || bs < 1 || n_blocks < 0) return SD_EINVAL;
  if (type == SD_CACHE_FP4 && D % 32 != 0) return SD_EINVAL;
  if (!k || !v || off16(k) || off16(v)) return SD_EINVAL;
  if (type == SD_CACHE_FP4 && (!ks || !vs || off16(ks) || off16(vs))) return SD_EINVAL;
  if ((long long)n_blocks * bs > (1ll << 40)) return SD_EUNSUPPORTED;
  const long long tokens = (long long)n_blocks * bs * n_kv;
  const long long bytes = type == SD_CACHE_FP4 ? tokens * (D / 2) : tokens * D * 2;
  spans[0] = sdv::span(k, bytes);
  spans[1] = sdv::span(v, bytes);
  spans[2] = sdv::span(type == SD_CACHE_FP4 ? ks : nullptr, tokens * (D / 32));
  spans[3] = sdv::span(type == SD_CACHE_FP4 ? vs : nullptr, tokens * (D / 32));
  return SD_OK;
}

}  // namespace

extern "C" int sd_qk_rope(hipStream_t stream, int n_rows, int D, int dtype, const void* q, int n_q, long long ld_q,
                          const void* k, int n_kv, long long ld_k, const int32_t* pos, const float* q_weight,
                          const float* k_weight, float eps, const float* inv_freq, int rot_dim, int interleaved,
                          void* q_out, long long ld_q_out, void* k_out, long long ld_k_out) {
  const int rc = check_heads(n_rows, D, dtype, n_q, n_kv, eps, q_weight, k_weight, inv_freq, rot_dim, interleaved, pos);
  if (rc != SD_OK) return rc;
  if (n_rows == 0 || n_q + n_kv == 0) return SD_OK;
  if (bad_rows(q, ld_q, n_q, D) || bad_rows(k, ld_k, n_kv, D) || bad_rows(q_out, ld_q_out, n_q, D) ||
      bad_rows(k_out, ld_k_out, n_kv, D))
    return SD_EINVAL;
  const int es = dtype == SD_DTYPE_F32 ? 4 : 2;
  const sdv::Span qi = rows_span(n_q ? q : nullptr, n_rows, n_q, D, ld_q, es),
                  ki = rows_span(n_kv ? k : nullptr, n_rows, n_kv, D, ld_k, es),
                  qo = rows_span(n_q ? q_out : nullptr, n_rows, n_q, D, ld_q_out, es),
                  ko = rows_span(n_kv ? k_out : nullptr, n_rows, n_kv, D, ld_k_out, es);
  const bool same_q = q == q_out && ld_q == ld_q_out, same_k = k == k_out && ld_k == ld_k_out;
  const sdv::Span written[] = {qo, ko};
  const sdv::Span read[] = {sdv::span(pos, 4ll * n_rows), sdv::span(q_weight, 4ll * D), sdv::span(k_weight, 4ll * D),
                            sdv::span(rot_dim ? inv_freq : nullptr, 2ll * rot_dim)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
  if ((!same_q && sdv::meet(qo, qi)) || (!same_k && sdv::meet(ko, ki)) || sdv::meet(qo, ki) || sdv::meet(ko, qi))
    return SD_EINVAL;
  HeadArgs a = {};
  a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
  a.ld_q = ld_q, a.ld_k = ld_k, a.ld_qo = ld_q_out, a.ld_ko = ld_k_out;
  a.pos = pos, a.wq = q_weight, a.wk = k_weight, a.inv_freq = inv_freq, a.eps = eps;
  a.n_rows = n_rows, a.n_q = n_q, a.n_kv = n_kv, a.D = D, a.rot = rot_dim;
  return run_heads(stream, a, dtype, kToRows, interleaved != 0);
}

extern "C" int sd_cache_append(hipStream_t stream, int n_rows, int D, int dtype, const void* q, int n_q,
                               long long ld_q, const void* k, long long ld_k, const void* v, long long ld_v, int n_kv,
                               const int32_t* row_pos, const int64_t* row_slot, const float* q_weight,
                               const float* k_weight, float eps, const float* inv_freq, int rot_dim, int interleaved,
                               void* q_out, long long ld_q_out, int cache_type, int block_size, int n_blocks,
                               void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale) {
  int rc = check_heads(n_rows, D, dtype, n_q, n_kv, eps, q_weight, k_weight, inv_freq, rot_dim, interleaved, row_pos);
  if (rc != SD_OK) return rc;
  if (cache_type != SD_CACHE_BF16 && cache_type != SD_CACHE_FP4) return SD_EINVAL;
  if (n_rows == 0) return SD_OK;
  sdv::Span c[4];
  rc = check_cache(cache_type, n_kv, D, block_size, n_blocks, k_cache, v_cache, k_scale, v_scale, c);
  if (rc != SD_OK) return rc;
  if (!row_slot || bad_rows(q, ld_q, n_q, D) || bad_rows(k, ld_k, n_kv, D) || bad_rows(v, ld_v, n_kv, D) ||
      bad_rows(q_out, ld_q_out, n_q, D))
    return SD_EINVAL;
  const int es = dtype == SD_DTYPE_F32 ? 4 : 2;
  const sdv::Span qi = rows_span(n_q ? q : nullptr, n_rows, n_q, D, ld_q, es),
                  qo = rows_span(n_q ? q_out : nullptr, n_rows, n_q, D, ld_q_out, es);
  const sdv::Span written[] = {qo, c[0], c[1], c[2], c[3]};
  const sdv::Span read[] = {sdv::span(row_pos, 4ll * n_rows), sdv::span(row_slot, 8ll * n_rows),
                            sdv::span(q_weight, 4ll * D), sdv::span(k_weight, 4ll * D),
                            sdv::span(rot_dim ? inv_freq : nullptr, 2ll * rot_dim),
                            rows_span(k, n_rows, n_kv, D, ld_k, es), rows_span(v, n_rows, n_kv, D, ld_v, es)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
  if (!(q == q_out && ld_q == ld_q_out) && sdv::meet(qo, qi)) return SD_EINVAL;
  for (const sdv::Span& s : c)
    if (sdv::meet(s, qi)) return SD_EINVAL;
  HeadArgs a = {};
  a.q = q, a.k = k, a.v = v, a.q_out = q_out;
  a.ld_q = ld_q, a.ld_k = ld_k, a.ld_v = ld_v, a.ld_qo = ld_q_out;
  a.pos = row_pos, a.slot = row_slot, a.wq = q_weight, a.wk = k_weight, a.inv_freq = inv_freq, a.eps = eps;
  a.n_rows = n_rows, a.n_q = n_q, a.n_kv = n_kv, a.n_v = n_kv, a.D = D, a.rot = rot_dim;
  a.cache = Cache{k_cache, v_cache, k_scale, v_scale, n_kv, block_size, n_blocks, 1.0 / block_size};
  return run_heads(stream, a, dtype, cache_type == SD_CACHE_FP4 ? kToFp4 : kToBf16, interleaved != 0);
}

extern "C" int sd_cache_read(hipStream_t stream, int n_rows, int D, const int64_t* row_slot, int cache_type, int n_kv,
                             int block_size, int n_blocks, const void* k_cache, const void* v_cache,
                             const uint8_t* k_scale, const uint8_t* v_scale, int dtype, void* k_out, long long ld_k,
                             void* v_out, long long ld_v) {
  if (n_rows < 0 || D < 8 || D % 8 != 0 || (dtype != SD_DTYPE_F32 && dtype != SD_DTYPE_BF16)) return SD_EINVAL;
  if (cache_type != SD_CACHE_BF16 && cache_type != SD_CACHE_FP4) return SD_EINVAL;
  if (n_rows == 0) return SD_OK;
  if (D > kMaxHead || n_kv > SD_MAX_HEADS) return SD_EUNSUPPORTED;
  sdv::Span c[4];
  const int rc = check_cache(cache_type, n_kv, D, block_size, n_blocks, k_cache, v_cache, k_scale, v_scale, c);
  if (rc != SD_OK) return rc;
  if (!row_slot || bad_rows(k_out, ld_k, n_kv, D) || bad_rows(v_out, ld_v, n_kv, D)) return SD_EINVAL;
  const int es = dtype == SD_DTYPE_F32 ? 4 : 2;
  const sdv::Span written[] = {rows_span(k_out, n_rows, n_kv, D, ld_k, es), rows_span(v_out, n_rows, n_kv, D, ld_v, es)};
  const sdv::Span read[] = {c[0], c[1], c[2], c[3], sdv::span(row_slot, 8ll * n_rows)};
  if (sdv::overlap(written, read)) return SD_EINVAL;
  ReadArgs a = {};
  a.slot = row_slot, a.k_out = k_out, a.v_out = v_out, a.ld_k = ld_k, a.ld_v = ld_v;
  a.cache = Cache{(void*)k_cache, (void*)v_cache, (uint8_t*)k_scale, (uint8_t*)v_scale, n_kv, block_size, n_blocks, 1.0 / block_size};
  a.n_rows = n_rows, a.D = D, a.vecs = 2 * n_kv * (D / 8);
  const int threads = a.vecs < kThreads ? (a.vecs + 63) / 64 * 64 : kThreads;
  if ((long long)n_rows * threads > 0xFFFFFFFFll) return SD_EUNSUPPORTED;
  const dim3 grid((unsigned)n_rows), block((unsigned)threads);
  if (cache_type == SD_CACHE_FP4) {
    if (es == 4) SDV_TRY_LAUNCH(sdv::launch(k_cache_read<float, true>, grid, block, 0, stream, a));
    else SDV_TRY_LAUNCH(sdv::launch(k_cache_read<uint16_t, true>, grid, block, 0, stream, a));
  } else {
    if (es == 4) SDV_TRY_LAUNCH(sdv::launch(k_cache_read<float, false>, grid, block, 0, stream, a));
    else SDV_TRY_LAUNCH(sdv::launch(k_cache_read<uint16_t, false>, grid, block, 0, stream, a));
  }
  return SD_OK;
}
