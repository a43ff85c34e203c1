// Paged attention for head_dim 64.
#include "paged_attn_launch.cuh"

cudaError_t sf::pa::launch_hd64(Args& a, int q_dtype, int sms, long max_units, cudaStream_t st) {
  return launch_types<64>(a, q_dtype, sms, max_units, st);
}
