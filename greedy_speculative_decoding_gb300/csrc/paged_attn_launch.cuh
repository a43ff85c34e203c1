// Launches of the paged attention kernels for one head dimension (one
// translation unit each).
#pragma once

#include <atomic>

#include "paged_attn_tc.cuh"

namespace sf {
namespace pa {

// Launch a main kernel (`ctas` CTAs an SM); leaves the launch's configuration.
inline cudaError_t launch_main(void (*fn)(Args), int threads, int smem, int piece, std::atomic<uint64_t>& ready, Args& a,
                               int sms, int ctas, long max_units, cudaStream_t st, cudaLaunchConfig_t& cfg,
                               cudaLaunchAttribute (&attr)[1]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const long most = (long)sms * ctas, items = (long)a.B * a.nkv * a.ntq_max;
  a.piece = piece;
  max_units += piece * items;
  const int grid = (int)(max_units < most ? max_units : most);
  // Many parts an item, and not so many queries that their CTAs come in waves.
  a.wide = items * 8 <= grid && items * a.mt_max <= 1024;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

// A main kernel and the join.
template <int HD, typename TQ, int MT>
cudaError_t launch(void (*fn)(Args), int threads, int smem, int piece, std::atomic<uint64_t>& ready, Args& a,
                   int sms, int ctas, long max_units, cudaStream_t st) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[1];
  const cudaError_t e = launch_main(fn, threads, smem, piece, ready, a, sms, ctas, max_units, st, cfg, attr);
  if (e != cudaSuccess) return e;
  if (a.by_item) cfg.gridDim.x = (unsigned)((long)a.B * a.nkv * a.ntq_max);
  cfg.gridDim.y = a.wide ? a.mt_max : (a.mt_max + 3) / 4;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_paged_join<HD, TQ, MT>, a);
}

template <int HD, typename TC, bool F32, int WM, int WK>
cudaError_t launch_mma(Args& a, int sms, long max_units, cudaStream_t st) {
  using S = Shape<HD, WM, WK, F32>;
  static_assert(S::kPiece <= kMaxPiece);
  using TQ = typename std::conditional<F32, float, TC>::type;
  static std::atomic<uint64_t> ready{0};   // devices whose shared-memory limit for this kernel is set
  return launch<HD, TQ, S::MT>(k_paged_attn<HD, TC, F32, WM, WK>, S::kThreads, S::kSmem, S::kPiece, ready, a, sms,
                               S::kCtas, max_units, st);
}

template <int HD, typename TC, bool F32>
cudaError_t launch_tc(Args& a, int sms, long max_units, cudaStream_t st) {
  using S = TcShape<HD, TC, F32>;
  static_assert(S::kPiece <= kMaxPiece);
  using TQ = typename std::conditional<F32, float, TC>::type;
  static std::atomic<uint64_t> ready{0};
  return launch<HD, TQ, S::MT>(k_paged_attn_tc<HD, TC, F32>, S::kThreads, S::kSmem, S::kPiece, ready, a, sms,
                               S::kCtas, max_units, st);
}

template <int HD, typename TC, bool F32>
cudaError_t launch_tiles(Args& a, int sms, long max_units, cudaStream_t st) {
  if (a.mt == 16) return launch_mma<HD, TC, F32, 1, 4>(a, sms, max_units, st);
  if constexpr (HD == 64 || !F32) {
    if (a.mt == 32) return launch_mma<HD, TC, F32, 2, 2>(a, sms, max_units, st);
  }
  return launch_tc<HD, TC, F32>(a, sms, max_units, st);
}

template <int HD>
cudaError_t launch_types(Args& a, int q_dtype, int sms, long max_units, cudaStream_t st) {
  switch (q_dtype) {
    case SF_DT_BF16: return launch_tiles<HD, bf16, false>(a, sms, max_units, st);
    case SF_DT_F16: return launch_tiles<HD, __half, false>(a, sms, max_units, st);
    default: return launch_tiles<HD, bf16, true>(a, sms, max_units, st);
  }
}

cudaError_t launch_hd64(Args& a, int q_dtype, int sms, long max_units, cudaStream_t st);
cudaError_t launch_hd128(Args& a, int q_dtype, int sms, long max_units, cudaStream_t st);
cudaError_t launch_chunk_hd64(Args& a, int dtype, int sms, long max_units, cudaStream_t st);
cudaError_t launch_chunk_hd128(Args& a, int dtype, int sms, long max_units, cudaStream_t st);

}  // namespace pa
}  // namespace sf
