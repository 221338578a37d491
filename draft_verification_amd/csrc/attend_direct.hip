// The attention kernel over a cache of 4 bits for a few queries.
#include "attend_direct.h"

int sdv::attend_direct(hipStream_t stream, int M, int W, const AttnArgs& a) {
  const dim3 grid((unsigned)W), block(kAttnThreads);
#define SDV_DIRECT(DD, NT)                                                                           \
  if (a.shape.D == DD && M == 16 * NT) {                                                             \
    static_assert(attn_direct(DD, 16 * NT, true, 16), "form");                                       \
    SDV_TRY_LAUNCH(launch(attn::k_attend_direct<DD, NT>, grid, block, 0, stream, a));                \
    return SD_OK;                                                                                    \
  }
  SDV_DIRECT(64, 1)
  SDV_DIRECT(64, 2)
  SDV_DIRECT(64, 3)
  SDV_DIRECT(64, 4)
  SDV_DIRECT(128, 1)
  SDV_DIRECT(128, 2)
  SDV_DIRECT(128, 3)
  SDV_DIRECT(256, 1)
#undef SDV_DIRECT
  return SD_EUNSUPPORTED;
}
