// Block tables and slot maps from request lengths (sf_page_plan).
//
// The plan is a pair of prefix sums over the requests: of the pages given
// back and of the pages wanted. With them every piece of the result follows
// by itself: page k granted in this pass is entry top - 1 - k of the stack
// that the releases leave, and an entry of that stack is either one of the
// old free list (below n_free, which the pass does not write) or a released
// page, still in its table row. So nothing reads what another thread writes:
// the pages granted, the pages given back and the token rows form one list of
// pieces that the threads take in any order, and several CTAs can each
// compute the sums for themselves (a few int32 per request) and share out the
// list. They meet once, before the counts held on entry are replaced.
#include <algorithm>
#include <atomic>

#include "paged.h"

namespace sf {
namespace {

constexpr int kPlanThreads = 1024;   // of a CTA, at most
constexpr int kPlanCluster = 8;      // CTAs of a pass with many rows
// Rows from which a cluster is worth its launch: one CTA takes about 0.8 ns a
// row, so 8192 rows are the 6 us that all the rest of a call costs.
constexpr int kPlanClusterRows = 8192;

struct PlanArgs {
  const int* lens;
  const int* starts;
  int* tables;
  const int* held;
  int* free;
  const int* n_free;
  int* slots;
  int* positions;
  int* held_out;
  int* n_free_out;
  int* status;
  int B, W, cap, shift, N;
};

// Inclusive sums of x and y over the CTA's threads, and their totals (64 bits:
// the wants of a bad batch can pass 2^31).
__device__ __forceinline__ void scan2(long long& x, long long& y, long long& tx, long long& ty,
                                      longlong2* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) warp_sums[warp] = make_longlong2(x, y);
  __syncthreads();
  longlong2 s = lane < warps ? warp_sums[lane] : make_longlong2(0, 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, s.x, o), b = __shfl_up_sync(0xffffffffu, s.y, o);
    if (lane >= o) {
      s.x += a;
      s.y += b;
    }
  }
  tx = __shfl_sync(0xffffffffu, s.x, 31);
  ty = __shfl_sync(0xffffffffu, s.y, 31);
  const long long px = __shfl_sync(0xffffffffu, s.x, warp > 0 ? warp - 1 : 0);
  const long long py = __shfl_sync(0xffffffffu, s.y, warp > 0 ? warp - 1 : 0);
  if (warp > 0) {
    x += px;
    y += py;
  }
  __syncthreads();   // the sums have been read
}

// Largest b in [lo, hi] with a[b] <= i (a[lo] <= i, a non-decreasing).
__device__ __forceinline__ int last_at_most(const int* a, int lo, int hi, int i) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* s_start = plan_smem;            // [B + 1] row starts
  int* s_back = s_start + a.B + 1;     // [B + 1] exclusive sums of pages given back
  int* s_want = s_back + a.B + 1;      // [B + 1] exclusive sums of pages granted
  int* s_held = s_want + a.B + 1;      // [B] pages held on entry
  int* s_need = s_held + a.B;          // [B] pages held afterwards
  int* s_len = s_need + a.B;           // [B] tokens; -1 when the request's rows get no slots
  __shared__ longlong2 warp_sums[32];
  const int tid = threadIdx.x, NT = blockDim.x;
  const int n_free = min(max(*a.n_free, 0), a.cap);

  // The sums, cut off at one page more than there are (a sum past the stack's
  // height serves nobody).
  const long long most = (long long)a.cap + 1;
  long long back_sum = 0, want_sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + tid;
    int back = 0, want = 0, held = 0, need = 0, len = -1;
    if (b < a.B) {
      const int s = a.starts[b], rows = a.starts[b + 1] - s;
      held = a.held[b];
      len = a.lens[b];
      need = (int)(((long long)len + (1 << a.shift) - 1) >> a.shift);
      const bool bad = len < 0 || need > a.W || rows > len || held < 0 || held > a.W;
      if (bad) {
        len = -2;
        need = held;
      }
      back = max(held - need, 0);
      want = max(need - held, 0);
      s_start[b] = s;
      if (b == a.B - 1) s_start[a.B] = s + rows;
      s_held[b] = held;
      s_need[b] = need;
      s_len[b] = len;
    }
    long long x = back, y = want, tx, ty;
    scan2(x, y, tx, ty, warp_sums);
    if (b < a.B) {
      s_back[b] = (int)min(back_sum + x - back, most);
      s_want[b] = (int)min(want_sum + y - want, most);
    }
    back_sum += tx;
    want_sum += ty;
  }
  if (tid == 0) {
    s_back[a.B] = (int)min(back_sum, most);
    s_want[a.B] = (int)min(want_sum, most);
  }
  const bool many = gridDim.x > 1;     // one cluster
  if (many) cluster_arrive();          // held and n_free have been read
  __syncthreads();
  const int top = (int)min(n_free + back_sum, (long long)a.cap);
  // The grants end at the first request whose want does not fit: every later
  // one that wants pages has a larger sum still.
  for (int b = tid; b < a.B; b += NT) {
    int st = 0;
    if (s_len[b] == -2) st = 2;
    else if (s_need[b] > s_held[b] && s_want[b] + (s_need[b] - s_held[b]) > top) st = 1;
    if (st) {
      s_len[b] = -1;
      s_need[b] = s_held[b];
    }
    if (blockIdx.x == 0) a.status[b] = st;
  }
  __syncthreads();
  // Granted pages: the sum up to the first refusal (sums past it exceed top,
  // except those of requests that want nothing, which repeat it).
  const int granted = s_want[last_at_most(s_want, 0, a.B, top)];
  const int given = top - n_free;

  // Entry i of the stack after the releases.
  auto stack_at = [&](int i) {
    if (i < n_free) return a.free[i];
    const int r = i - n_free;
    const int b = last_at_most(s_back, 0, a.B, r);
    return a.tables[(size_t)b * a.W + s_need[b] + (r - s_back[b])];
  };
  const long pieces = (long)granted + given + a.N;
  for (long k0 = blockIdx.x * (long)NT + tid; k0 < pieces; k0 += (long)gridDim.x * NT) {
    if (k0 < granted) {
      const int k = (int)k0;
      const int b = last_at_most(s_want, 0, a.B, k);
      a.tables[(size_t)b * a.W + s_held[b] + (k - s_want[b])] = stack_at(top - 1 - k);
      continue;
    }
    if (k0 < granted + (long)given) {
      const int i = n_free + (int)(k0 - granted);
      a.free[i] = stack_at(i);
      continue;
    }
    const int i = (int)(k0 - granted - given);
    int slot = -1, pos = 0;
    if (i >= s_start[0] && i < s_start[a.B]) {
      const int b = last_at_most(s_start, 0, a.B, i);
      if (b < a.B && s_len[b] >= 0) pos = s_len[b] - (s_start[b + 1] - i);
      if (b < a.B && pos >= 0 && pos < s_len[b]) {   // (starts that decrease can lead anywhere)
        const int p = pos >> a.shift;
        const int page = p < s_held[b] ? a.tables[(size_t)b * a.W + p]
                                       : stack_at(top - 1 - (s_want[b] + p - s_held[b]));
        slot = (page << a.shift) + (pos & ((1 << a.shift) - 1));
      }
    }
    a.slots[i] = slot;
    a.positions[i] = slot < 0 ? 0 : pos;
  }
  // held_out and n_free_out may be held and n_free: every CTA has read them.
  __syncthreads();
  if (many) cluster_wait();
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.B; b += NT) a.held_out[b] = s_need[b];
    if (tid == 0) *a.n_free_out = top - granted;
  }
}

size_t plan_smem_bytes(int B) { return (size_t)(3 * (B + 1) + 3 * B) * sizeof(int); }

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" sf_status sf_page_plan(const int32_t* d_lens, const int32_t* d_starts, int32_t batch, int32_t page,
                                  int32_t* d_tables, int32_t table_width, const int32_t* d_held, int32_t* d_free,
                                  int32_t capacity, const int32_t* d_n_free, int32_t n_rows, int32_t* d_slots,
                                  int32_t* d_positions, int32_t* d_held_out, int32_t* d_n_free_out, int32_t* d_status,
                                  void* cuda_stream) {
  if (!d_lens || !d_starts || !d_tables || !d_held || !d_free || !d_n_free || !d_held_out || !d_n_free_out || !d_status)
    return set_error(SF_ERR_ARG, "sf_page_plan: null pointer");
  if (batch < 1 || batch > kMaxPlanBatch)
    return set_error(SF_ERR_ARG, "sf_page_plan: batch %d outside 1..%d", batch, kMaxPlanBatch);
  if (!page_ok(page)) return set_error(SF_ERR_ARG, "sf_page_plan: page must be 16, 32, 64, 128 or 256");
  if (table_width < 1 || table_width > (1 << 30) / page || capacity < 1 || capacity > INT32_MAX / page)
    return set_error(SF_ERR_ARG, "sf_page_plan: need 1 <= table_width <= 2^30 / page, 1 <= capacity, capacity * page < 2^31");
  if (n_rows < 0 || (n_rows > 0 && (!d_slots || !d_positions)))
    return set_error(SF_ERR_ARG, "sf_page_plan: n_rows negative, or rows without slots and positions");
  const PlanArgs a{d_lens,      d_starts,   d_tables,     d_held,   d_free, d_n_free,    d_slots,  d_positions,
                   d_held_out, d_n_free_out, d_status, batch,  table_width, capacity, log2_of(page), n_rows};
  static std::atomic<uint64_t> ready{0};   // devices whose shared-memory limit for the kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(k_page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)plan_smem_bytes(kMaxPlanBatch));
    if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) {
    const int ctas = n_rows >= kPlanClusterRows ? kPlanCluster : 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(std::min(kPlanThreads, std::max(128, (std::max(batch, n_rows) + 31) / 32 * 32)));
    cfg.dynamicSmemBytes = plan_smem_bytes(batch);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k_page_plan, a);
  }
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_plan: %s", cudaGetErrorString(e));
  return SF_OK;
}
