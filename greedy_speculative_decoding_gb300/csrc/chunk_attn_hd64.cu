#include "chunk_attn_launch.cuh"

namespace sf {
namespace pa {

cudaError_t launch_chunk_hd64(Args& a, int dtype, int sms, long max_units, cudaStream_t st) {
  return launch_chunk_types<64>(a, dtype, sms, max_units, st);
}

}  // namespace pa
}  // namespace sf
