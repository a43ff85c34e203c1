// Launch interface of the paged-cache operators (paged_plan.cu, paged_append.cu, paged_attn.cu).
#pragma once

#include <utility>

#include "sf_kernels.h"

namespace sf {

constexpr int kMaxPlanBatch = 8192;   // requests of one page plan (their prefix sums lie in shared memory)
constexpr int kMinPage = 16, kMaxPage = 256;

inline bool page_ok(int page) { return page >= kMinPage && page <= kMaxPage && (page & (page - 1)) == 0; }
inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

struct PlanArgs {
  const int* lens;     // [B]; a request has lens[b] + len_add tokens
  int len_add;
  const int* starts;   // [B + 1] row starts, or null: rows_each rows each
  int rows_each;
  int* tables;         // [B][W]
  const int* held;
  int* free;
  const int* n_free;
  int* slots;
  int* positions;
  int* held_out;
  int* n_free_out;
  int* status;
  int B, W, cap, shift, N;
  // 1: the launch overlaps the end of the kernel before it, the next launch its own (plan, append and attention of one
  // row: 13.3 us a pass in a stream, 16.7 without this and the append's overlap). 0 in the engine, whose projections
  // count on everything but the kernel just before them being done.
  int early;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st);

// The engine's attention over its target's pages: fp32 queries [M][nq * hd],
// `rows` token rows of each of B sequences, the last of them at position
// lens[b] + len_add - 1; the output goes where the output projection reads it.
struct EngineAttn {
  sf_paged_cache cache;
  const float* q;
  bf16* out;                 // fragment order, or the tensor-core operand order (umma)
  int umma;
  const int* tables;
  int table_width;
  const int* lens;
  int len_add, B, rows, nq;
  const unsigned long long* mask;   // [B * rows], or null: causal
  float scale;
  int* err;
  void* workspace;
};
cudaError_t launch_engine_paged_attention(const EngineAttn& e, int num_sms, cudaStream_t st);
// Row masks of a verify pass over candidate guesses of g tokens (see RowSet).
cudaError_t launch_tree_mask(unsigned long long* mask, int B, int rows, int g, cudaStream_t st, bool pdl);

// Whether two of n1 x n2 vectors of hd elements, s1 and s2 apart, share an
// element (a call that writes them would leave whichever came last).
inline bool vectors_overlap(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t hd) {
  __int128 s = s1 < 0 ? -(__int128)s1 : s1, t = s2 < 0 ? -(__int128)s2 : s2;
  if ((n1 > 1 && s < hd) || (n2 > 1 && t < hd)) return true;
  if (n1 <= 1 || n2 <= 1) return false;
  if (s > t) {
    std::swap(s, t);
    std::swap(n1, n2);
  }
  if (t >= (n1 - 1) * s + hd) return false;   // one after the other, as nearly always
  for (int64_t b = 1; b < n2 && b * t < n1 * s; ++b) {
    const __int128 a = b * t / s, r = b * t - a * s;
    if (r < hd || (a + 1 < n1 && s - r < hd)) return true;
  }
  return false;
}

// Checks a cache descriptor; on failure records the message and returns the status.
sf_status check_cache(const sf_paged_cache* c, const char* who);

}  // namespace sf
