// Compiled instances of the decode kernel over E4M3 KV with per-block (page, kv
// head) scales for q = __nv_bfloat16 (a translation unit of their own so the build
// runs in parallel).
#include "decode_mma.cuh"

namespace fadecode {
bool find_block_scale_kernel_bf16_e4m3(int head_dim, int group, DecodeKernel* k) {
  return find_block_scale_kernel_for<__nv_bfloat16>(head_dim, group, k);
}
bool find_block_scale_multi_token_kernel_bf16_e4m3(int head_dim, int group, int q_len,
                                                   DecodeKernel* k) {
  return find_multi_token_kernel_for<__nv_bfloat16, __nv_fp8_e4m3, kScalePerBlock>(head_dim, group,
                                                                                   q_len, k);
}
}  // namespace fadecode
