// The attention kernel over a cache of 4 bits.
#include "attend_kernel.h"

int sdv::attend_fp4(hipStream_t stream, int M, int W, const AttnArgs& a) {
  return attn::launch_attend<true>(stream, M, W, a);
}
