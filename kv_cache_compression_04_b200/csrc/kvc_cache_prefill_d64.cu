// Attention over the paged 4-bit cache for many query rows, head_dim 64.
#include "kvc_cache_prefill.cuh"

namespace kvc {
cudaError_t launch_cache_prefill_d64(int g, int dtype, const CacheAttnArgs &a, int sms,
                                     cudaStream_t st) {
  if (g == 64) return cache_prefill_t<64, 64>(dtype, a, sms, st);
  return cache_prefill_t<64, 32>(dtype, a, sms, st);
}
}  // namespace kvc
