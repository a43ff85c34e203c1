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

// Tokens and first row of a request (starts null: rows_each rows each).
__device__ __forceinline__ int plan_len(const PlanArgs& a, int b) { return a.lens[b] + a.len_add; }
__device__ __forceinline__ int plan_start(const PlanArgs& a, int b) { return a.starts ? a.starts[b] : b * a.rows_each; }

constexpr int kPlanThreads = 1024;   // of a CTA, at most
constexpr int kPlanCluster = 8;      // CTAs of a pass with many pieces
// From 64 requests or 1024 rows the pieces (a finished request gives back all
// its pages) outweigh the cluster's launch: 512 requests with one row each,
// 6400 pages given back, take 9.6 us in one CTA and 5.5 us in eight; 8
// requests with 72 rows 3.5 us in one, 4.2 us in eight.
constexpr int kPlanClusterRequests = 64, kPlanClusterRows = 1024;
// Rows from which they get a kernel of their own over the whole GPU: 16000 rows
// take 5.5 us in the plan's cluster and 6.8 us so, 32000 rows 7.8 and 7.0 us,
// 512000 rows 66 and 8.4 us.
constexpr int kPlanManyRows = 32768;
constexpr int kRowThreads = 256, kRowCtas = 608;

// Sums that stop at `most` (at most 2^28, so that two of them fit an int).
__device__ __forceinline__ int add_to(int a, int b, int most) { return min(a + b, most); }

// Exclusive sums of x and y over the CTA's threads, and their totals.
__device__ __forceinline__ void scan2(int& x, int& y, int& tx, int& ty, int most, int2* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = add_to(v, u, most);
    }
    return v;
  };
  x = scan(x);
  y = scan(y);
  if (lane == 31) warp_sums[warp] = make_int2(x, y);
  __syncthreads();
  const int2 s = lane < warps ? warp_sums[lane] : make_int2(0, 0);
  const int sx = scan(s.x), sy = scan(s.y);
  tx = __shfl_sync(0xffffffffu, sx, 31);
  ty = __shfl_sync(0xffffffffu, sy, 31);
  const int px = __shfl_sync(0xffffffffu, sx, max(warp - 1, 0)), py = __shfl_sync(0xffffffffu, sy, max(warp - 1, 0));
  const int ux = __shfl_up_sync(0xffffffffu, x, 1), uy = __shfl_up_sync(0xffffffffu, y, 1);
  x = add_to(warp > 0 ? px : 0, lane > 0 ? ux : 0, most);
  y = add_to(warp > 0 ? py : 0, lane > 0 ? uy : 0, most);
  __syncthreads();   // the sums have been read
}

// Largest b in [0, n] with a[b] <= i (a[0] <= i, a non-decreasing); p2: a
// power of two above n / 2.
__device__ __forceinline__ int last_at_most(const int* a, int n, int p2, int i) {
  int b = 0;
  for (int s = p2; s > 0; s >>= 1) {
    const int t = b + s;
    const bool take = t <= n && a[min(t, n)] <= i;
    b = take ? t : b;
  }
  return b;
}

__global__ void __launch_bounds__(kPlanThreads) k_page_plan(const PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* s_start = plan_smem;            // [B + 1] row starts
  int* s_back = s_start + a.B + 1;     // [B + 1] exclusive sums of pages given back
  int* s_want = s_back + a.B + 1;      // [B + 1] exclusive sums of pages granted
  int* s_held = s_want + a.B + 1;      // [B] pages held on entry
  int* s_need = s_held + a.B;          // [B] pages held afterwards
  int* s_len = s_need + a.B;           // [B] tokens; -1 when the request's rows get no slots
  __shared__ int2 warp_sums[32];
  __shared__ int s_granted;
  const int tid = threadIdx.x, NT = blockDim.x;
  pdl_wait();
  if (a.early) pdl_launch_next();
  const int n_free = min(max(*a.n_free, 0), a.cap);

  // The sums, cut off at one page more than there are (a sum past the stack's
  // height serves nobody).
  const int most = a.cap + 1;
  int back_sum = 0, want_sum = 0;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + tid;
    int back = 0, want = 0, held = 0, need = 0, len = -1;
    if (b < a.B) {
      const int s = plan_start(a, b), rows = plan_start(a, b + 1) - s;
      held = a.held[b];
      len = plan_len(a, b);
      need = (int)(((long long)len + (1 << a.shift) - 1) >> a.shift);
      const bool bad = len < 0 || need > a.W || rows > len || held < 0 || held > a.W;
      if (bad) {
        len = -2;
        need = held;
      }
      back = min(max(held - need, 0), most);
      want = min(max(need - held, 0), most);
      s_start[b] = s;
      if (b == a.B - 1) s_start[a.B] = s + rows;
      s_held[b] = held;
      s_need[b] = need;
      s_len[b] = len;
    }
    int tx, ty;
    scan2(back, want, tx, ty, most, warp_sums);
    if (b < a.B) {
      s_back[b] = add_to(back_sum, back, most);
      s_want[b] = add_to(want_sum, want, most);
    }
    back_sum = add_to(back_sum, tx, most);
    want_sum = add_to(want_sum, ty, most);
  }
  if (tid == 0) {
    s_back[a.B] = back_sum;
    s_want[a.B] = want_sum;
    s_granted = 0;
  }
  const bool many = gridDim.x > 1;     // one cluster
  if (many) cluster_arrive();          // held and n_free have been read
  __syncthreads();
  const int top = min(n_free + back_sum, a.cap);
  // The grants end at the first request whose want does not fit: every later
  // one that wants pages has a larger sum still.
  for (int b = tid; b < a.B; b += NT) {
    int st = 0;
    const int want = min(s_need[b] - s_held[b], most), upto = s_want[b] + want;
    if (s_len[b] == -2) st = 2;
    else if (want > 0 && upto > top) st = 1;
    else if (want > 0) atomicMax(&s_granted, upto);
    if (st) {
      s_len[b] = -1;
      s_need[b] = s_held[b];
    }
    if (blockIdx.x == 0) a.status[b] = st;
  }
  __syncthreads();
  const int granted = s_granted, given = top - n_free;
  const int p2 = a.B > 1 ? 1 << (31 - __clz(a.B)) : 1;

  // Entry i of the stack after the releases.
  auto stack_at = [&](int i) {
    if (i < n_free) return a.free[i];
    const int r = i - n_free;
    const int b = last_at_most(s_back, a.B, p2, r);
    return a.tables[(size_t)b * a.W + s_need[b] + (r - s_back[b])];
  };
  const long pieces = (long)granted + given + a.N;
  for (long k0 = blockIdx.x * (long)NT + tid; k0 < pieces; k0 += (long)gridDim.x * NT) {
    if (k0 < granted) {
      const int k = (int)k0;
      const int b = last_at_most(s_want, a.B, p2, k);
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
    const int b = i >= s_start[0] ? min(last_at_most(s_start, a.B, p2, i), a.B - 1) : 0;
    const int x = s_len[b] - (s_start[b + 1] - i);
    if (i >= s_start[b] && i < s_start[b + 1] && x >= 0 && x < s_len[b]) {   // (starts that decrease can lead anywhere)
      const int p = x >> a.shift, held = s_held[b];
      const int page = p < held ? a.tables[(size_t)b * a.W + p] : stack_at(top - 1 - (s_want[b] + p - held));
      slot = (page << a.shift) + (x & ((1 << a.shift) - 1));
      pos = slot < 0 ? 0 : x;
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  // held_out and n_free_out may be held and n_free: every CTA has read them.
  __syncthreads();
  if (many) cluster_wait();
  if (blockIdx.x == 0) {
    for (int b = tid; b < a.B; b += NT) a.held_out[b] = s_need[b];
    if (tid == 0) *a.n_free_out = top - granted;
  }
}

// Slots and positions of many rows, once the plan kernel has left the tables
// and statuses: threads take four consecutive rows at a time (of one request
// and one or two pages, mostly), CTAs a stretch of rows each.
__global__ void __launch_bounds__(kRowThreads) k_plan_rows(const PlanArgs a) {
  extern __shared__ int s_start[];   // [B + 1]
  for (int b = threadIdx.x; b <= a.B; b += kRowThreads) s_start[b] = plan_start(a, b);
  const int p2 = a.B > 1 ? 1 << (31 - __clz(a.B)) : 1;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  const long quads = ((long)a.N + 3) / 4;
  const long q0 = blockIdx.x * quads / gridDim.x, q1 = (blockIdx.x + 1) * quads / gridDim.x;
  pdl_wait();
  __syncthreads();
  for (long q = q0 + threadIdx.x; q < q1; q += kRowThreads) {
    const int i0 = 4 * (int)q;
    // The request that holds the row, kept while the next rows are its own.
    int b = i0 >= s_start[0] ? min(last_at_most(s_start, a.B, p2, i0), a.B - 1) : 0;
    int first = s_start[b], end = s_start[b + 1], len = a.status[b] ? -1 : plan_len(a, b), known = -1, page = 0;
    int slot[4], pos[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      slot[e] = -1;
      pos[e] = 0;
      while (i >= end && b + 1 < a.B) {
        ++b;
        first = end;
        end = s_start[b + 1];
        len = a.status[b] ? -1 : plan_len(a, b);
        known = -1;
      }
      const int x = len - (end - i);
      if (i < first || i >= end || x < 0 || x >= len) continue;   // (starts that decrease can lead anywhere)
      if (x >> a.shift != known) {
        known = x >> a.shift;
        page = a.tables[(size_t)b * a.W + known];
      }
      slot[e] = (page << a.shift) + (x & ((1 << a.shift) - 1));
      pos[e] = slot[e] < 0 ? 0 : x;
    }
    if (vec && a.N - i0 >= 4) {   // (i0 + 4 may be 2^31)
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < a.N - i0) {
          a.slots[i0 + e] = slot[e];
          a.positions[i0 + e] = pos[e];
        }
    }
  }
}

size_t plan_smem_bytes(int B) { return (size_t)(3 * (B + 1) + 3 * B) * sizeof(int); }

}  // namespace

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices whose shared-memory limit for the kernel is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(k_page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)plan_smem_bytes(kMaxPlanBatch));
    if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) {
    const bool apart = a.N >= kPlanManyRows;
    const int ctas = a.B >= kPlanClusterRequests || a.N >= kPlanClusterRows ? kPlanCluster : 1;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(ctas > 1 ? kPlanThreads : std::max(128, (std::max(a.B, a.N) + 31) / 32 * 32));
    cfg.dynamicSmemBytes = plan_smem_bytes(a.B);
    cfg.stream = st;
    cfg.attrs = a.early ? attr : attr + 1;
    cfg.numAttrs = a.early + (ctas > 1);
    PlanArgs plan = a;
    if (apart) plan.N = 0;
    e = cudaLaunchKernelEx(&cfg, k_page_plan, plan);
    if (e == cudaSuccess && apart) {
      cfg.gridDim = dim3(kRowCtas);
      cfg.blockDim = dim3(kRowThreads);
      cfg.dynamicSmemBytes = (size_t)(a.B + 1) * sizeof(int);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, k_plan_rows, a);
    }
  }
  return e;
}

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
  PlanArgs a{};
  a.lens = d_lens, a.starts = d_starts, a.tables = d_tables, a.held = d_held, a.free = d_free, a.n_free = d_n_free;
  a.slots = d_slots, a.positions = d_positions, a.held_out = d_held_out, a.n_free_out = d_n_free_out;
  a.status = d_status;
  a.early = 1;
  a.B = batch, a.W = table_width, a.cap = capacity, a.shift = log2_of(page), a.N = n_rows;
  const cudaError_t e = launch_page_plan(a, static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_plan: %s", cudaGetErrorString(e));
  return SF_OK;
}
