// Attention over the paged 4-bit cache, head_dim 64.
#include "kvc_cache_attend.cuh"

namespace kvc {
cudaError_t launch_cache_attend_d64(int g, int dtype, const CacheAttnArgs &a, int sms,
                                    cudaStream_t st) {
  return g == 64 ? cache_attend_g<64, 64>(dtype, a, sms, st)
                 : cache_attend_g<64, 32>(dtype, a, sms, st);
}
}  // namespace kvc
