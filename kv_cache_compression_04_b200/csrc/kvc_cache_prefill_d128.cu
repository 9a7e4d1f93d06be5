// Attention over the paged 4-bit cache for many query rows, head_dim 128.
#include "kvc_cache_prefill.cuh"

namespace kvc {
cudaError_t launch_cache_prefill_d128(int g, int dtype, const CacheAttnArgs &a, int sms,
                                     cudaStream_t st) {
  if (g == 128) return cache_prefill_t<128, 128>(dtype, a, sms, st);
  if (g == 64) return cache_prefill_t<128, 64>(dtype, a, sms, st);
  return cache_prefill_t<128, 32>(dtype, a, sms, st);
}
}  // namespace kvc
