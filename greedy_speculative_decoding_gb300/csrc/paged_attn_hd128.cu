// Paged attention for head_dim 128.
#include "paged_attn_launch.cuh"

cudaError_t sf::pa::launch_hd128(Args& a, int q_dtype, int sms, long max_units, cudaStream_t st) {
  return launch_types<128>(a, q_dtype, sms, max_units, st);
}
