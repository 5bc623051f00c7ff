// Compiled instances of the decode kernel over E4M3 KV with per-block (page, kv
// head) scales for q = __half (a translation unit of their own so the build
// runs in parallel).
#include "decode_mma.cuh"

namespace fadecode {
bool find_block_scale_kernel_f16_e4m3(int head_dim, int group, DecodeKernel* k) {
  return find_block_scale_kernel_for<__half>(head_dim, group, k);
}
}  // namespace fadecode
