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
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  const cudaError_t e = launch_main(k_chunk_attn<HD, TC>, S::kThreads, S::kSmem, S::kPiece, ready, a, sms, 1, max_units,
                                    st, cfg, attr);
  if (e != cudaSuccess) return e;
  cfg.gridDim.x *= a.rounds;
  cfg.gridDim.y = (a.mt_max + kChunkJoinQueries - 1) / kChunkJoinQueries;
  cfg.blockDim = dim3(kChunkJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_chunk_join<HD, TC>, a);
}

template <int HD>
cudaError_t launch_chunk_types(Args& a, int dtype, int sms, long max_units, cudaStream_t st) {
  return dtype == SF_DT_BF16 ? launch_chunk<HD, bf16>(a, sms, max_units, st) : launch_chunk<HD, __half>(a, sms, max_units, st);
}

}  // namespace pa
}  // namespace sf
