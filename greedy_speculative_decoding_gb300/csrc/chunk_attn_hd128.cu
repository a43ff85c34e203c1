#include "chunk_attn_launch.cuh"

namespace sf {
namespace pa {

cudaError_t launch_chunk_hd128(Args& a, int dtype, int sms, long max_units, cudaStream_t st) {
  return launch_chunk_types<128>(a, dtype, sms, max_units, st);
}

}  // namespace pa
}  // namespace sf
