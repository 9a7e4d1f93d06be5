// Many rows of the paged 4-bit cache (read), head_dim 64.
#include "kvc_cache_blocks.cuh"

namespace kvc {
cudaError_t launch_cache_read_blocks_d64(int g, int dtype, const CachePool &c, const RowArgs &r,
                                         uint32_t blocks, int sms, cudaStream_t st) {
  if (g == 64) return launch_blocks<64, 64, false>(dtype, c, r, blocks, sms, st);
  return launch_blocks<64, 32, false>(dtype, c, r, blocks, sms, st);
}
}  // namespace kvc
