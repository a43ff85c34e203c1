// Launch interface of the paged-cache operators (paged_plan.cu, paged_append.cu, paged_attn.cu).
#pragma once

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

// Checks a cache descriptor; on failure records the message and returns the status.
sf_status check_cache(const sf_paged_cache* c, const char* who);

}  // namespace sf
