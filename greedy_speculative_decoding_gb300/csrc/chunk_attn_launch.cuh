// Launches of the chunk attention kernel for one head dimension (one
// translation unit each).
#pragma once

#include "chunk_attn.cuh"
#include "paged_attn_launch.cuh"

namespace sf {
namespace pa {

template <int HD, typename TC>
cudaError_t launch_chunk(Args& a, int sms, long max_units, cudaStream_t st) {
  using S = ChunkShape<HD, TC>;
  static std::atomic<uint64_t> ready{0};
  return launch<HD, TC, S::MT>(k_chunk_attn<HD, TC>, S::kThreads, S::kSmem, S::kPiece, ready, a, sms, 1, max_units, st);
}

template <int HD>
cudaError_t launch_chunk_types(Args& a, int dtype, int sms, long max_units, cudaStream_t st) {
  return dtype == SF_DT_BF16 ? launch_chunk<HD, bf16>(a, sms, max_units, st) : launch_chunk<HD, __half>(a, sms, max_units, st);
}

}  // namespace pa
}  // namespace sf
