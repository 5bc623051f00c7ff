// Compiled instances of the decode kernel over E4M3 KV with per-block scales
// and ragged query rows, for requests of two or three 8-column tiles, q =
// __nv_bfloat16 (a translation unit of their own so the build runs in
// parallel).
#include "decode_mma.cuh"

namespace fadecode {
bool find_block_scale_ragged_q_tiles_kernel_bf16_e4m3(int head_dim, int group, int tiles,
                                                      DecodeKernel* k) {
  return find_ragged_q_tiles_kernel_for<__nv_bfloat16, __nv_fp8_e4m3, kScalePerBlock>(
      head_dim, group, tiles, k);
}
}  // namespace fadecode
