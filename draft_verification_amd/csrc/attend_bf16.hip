// The attention kernel over a bf16 cache.
#include "attend_kernel.h"

int sdv::attend_bf16(hipStream_t stream, int M, int W, const AttnArgs& a) {
  return attn::launch_attend<false>(stream, M, W, a);
}
