// Many rows of the paged 4-bit cache (write), head_dim 128.
#include "kvc_cache_blocks.cuh"

namespace kvc {
cudaError_t launch_cache_write_blocks_d128(int g, int dtype, const CachePool &c, const RowArgs &r,
                                         uint32_t blocks, int sms, cudaStream_t st) {
  if (g == 128) return launch_blocks<128, 128, true>(dtype, c, r, blocks, sms, st);
  if (g == 64) return launch_blocks<128, 64, true>(dtype, c, r, blocks, sms, st);
  return launch_blocks<128, 32, true>(dtype, c, r, blocks, sms, st);
}
}  // namespace kvc
