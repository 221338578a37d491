// Host-side launch helper: hipLaunchKernel returns the launch status directly,
// so a stale error left by unrelated code is never misreported as ours.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <tuple>
#include <utility>

namespace sdv {

// The memory of an argument: `rows` pieces of `width` bytes, `stride` bytes
// apart, from lo to hi.  NULL and empty arguments meet nothing.
struct Span {
  uintptr_t lo, hi;
  long long rows, width, stride;
};
inline Span span(const void* p, long long rows, long long width, long long stride) {
  const uintptr_t lo = (uintptr_t)p;
  if (!p || rows < 1 || width < 1) return Span{lo, lo, 0, 0, 1};
  const __int128 end = (__int128)lo + (__int128)(rows - 1) * stride + width;
  return Span{lo, end > (__int128)UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end, rows, width, stride};
}
inline Span span(const void* p, long long bytes) {
  const uintptr_t lo = (uintptr_t)p, most = UINTPTR_MAX - lo;
  if (!p || bytes < 1) return Span{lo, lo, 0, 0, 1};
  return Span{lo, lo + ((uintptr_t)bytes < most ? (uintptr_t)bytes : most), 1, bytes, bytes};
}
inline bool meet(const Span& a, const Span& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.rows <= 1 || b.rows <= 1 || a.stride != b.stride) return a.rows > 0 && b.rows > 0;
  // rows of one buffer side by side: b's row k, d + k * stride behind a's row
  // 0, for the two k that bring them nearest (a's row i meets b's row i + k)
  const long long d = (long long)(b.lo - a.lo), s = a.stride;
  const long long down = d >= 0 ? d / s : -((-d + s - 1) / s);   // floor
  for (long long k = -down - 1; k <= -down; ++k) {
    const long long off = d + k * s;
    if (k > -a.rows && k < b.rows && off < a.width && off + b.width > 0) return true;
  }
  return false;
}
// Whether a written argument meets another one.
template <size_t W, size_t N>
inline bool overlap(const Span (&written)[W], const Span (&read)[N]) {
  for (size_t i = 0; i < W; ++i) {
    for (size_t k = i + 1; k < W; ++k)
      if (meet(written[i], written[k])) return true;
    for (size_t k = 0; k < N; ++k)
      if (meet(written[i], read[k])) return true;
  }
  return false;
}

template <typename... KArgs, typename Tuple, size_t... I>
static hipError_t launch_impl(void (*k)(KArgs...), dim3 g, dim3 b, size_t shmem, hipStream_t s,
                              Tuple& t, std::index_sequence<I...>) {
  void* argv[sizeof...(KArgs) + 1] = {(void*)&std::get<I>(t)..., nullptr};
  return hipLaunchKernel((const void*)k, g, b, argv, shmem, s);
}

// launch(kernel, grid, block, shmem, stream, args...): arguments are converted
// to the kernel's exact parameter types before their addresses are taken.
template <typename... KArgs, typename... Args>
static hipError_t launch(void (*k)(KArgs...), dim3 g, dim3 b, size_t shmem, hipStream_t s,
                         Args&&... args) {
  static_assert(sizeof...(KArgs) == sizeof...(Args), "kernel argument count");
  std::tuple<KArgs...> t(std::forward<Args>(args)...);
  return launch_impl(k, g, b, shmem, s, t, std::index_sequence_for<KArgs...>{});
}

}  // namespace sdv

#define SDV_TRY_LAUNCH(expr)                   \
  do {                                         \
    if ((expr) != hipSuccess) return SD_ELAUNCH; \
  } while (0)
