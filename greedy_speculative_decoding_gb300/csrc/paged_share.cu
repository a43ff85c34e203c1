// Pages that several requests hold: requests cut or ended (sf_page_free),
// forked (sf_page_fork), and the held pages moved to the lowest numbers
// (sf_page_compact). shares[p] counts page p's holders beyond the first.
//
// Each is one cluster of CTAs, or one small CTA. What must be known of every
// request of the list (its entries' place among all entries, whether an earlier
// one names the same request) every CTA finds for itself in shared memory; the
// entries are then dealt out, a stretch to each CTA and two to eight in a row to
// each thread, so that their loads are on their way together. Counts change by atomic
// additions of whole numbers, whose order does not matter, and where order
// matters (which of the releases of one page puts it onto the stack) the first
// in the list wins. What bounds all three is the chain of barriers and of loads
// that depend on one another.
#include <algorithm>
#include <atomic>
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "paged.h"

namespace sf {
namespace {

constexpr int kThreads = 1024, kCluster = 8;   // of many entries; few: one CTA of kFewThreads
constexpr int kFewThreads = 256;
constexpr int kMaxPages = 1 << 20;   // of a compaction (its bit map lies in shared memory)

// Exclusive sum of x over the CTA's threads and its total.
__device__ __forceinline__ int scan_cta(int x, int& total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int s = lane < (int)blockDim.x / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  __syncthreads();   // the sums have been read
  return (warp > 0 ? before : 0) + incl - x;
}

// Largest i in [0, n] with a[i] <= k (a[0] = 0, non-decreasing).
__device__ __forceinline__ int place_of(const int* a, int n, int k) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= k) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int ceil_pages(int tokens, int shift) {
  return (int)(((long long)tokens + (1 << shift) - 1) >> shift);
}

// Marks for every request the first of the list that names it.
__device__ __forceinline__ void first_of(const int* list, int n, int B, int* s_first) {
  for (int b = threadIdx.x; b < B; b += blockDim.x) s_first[b] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int r = list[i];
    if (r >= 0 && r < B) atomicMin(&s_first[r], i);
  }
  __syncthreads();
}

// Calls f with the entries that a thread takes one after the other. In a cluster
// four, or eight where that leaves one round of the threads: more a thread are
// more loads under way together, but fewer threads at work (a release and a fork
// of 18997 entries: 2, which is two rounds, 27.7 us, 4 21.9, 8 28.8). One CTA: two,
// as there is little to do and the code has to be fetched.
template <bool FEW, typename F>
__device__ __forceinline__ void with_run(int n, int threads, F f) {
  if constexpr (FEW) {
    f(std::integral_constant<int, 2>());
  } else {
    if (n <= 4 * threads) f(std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 8>());
  }
}

struct FreeArgs {
  const int *requests, *keep;
  int n;
  int* tables;
  int* held;
  int* shares;
  int* free;
  int* n_free;
  int* status;
  int B, W, P, cap, shift;
};

template <bool FEW>   // one CTA of kFewThreads
__global__ void __launch_bounds__(FEW ? kFewThreads : kThreads, 1) k_page_free(const FreeArgs a) {
  extern __shared__ int share_smem[];
  int* s_first = share_smem;        // [B] the first of the list that names a request
  int* s_at = s_first + a.B;        // [n + 1] entries released before
  int* s_row = s_at + a.n + 1;      // [n] the request, or -1
  int* s_from = s_row + a.n;        // [n] its first entry released
  __shared__ int warp_sums[32], s_mine;
  const int tid = threadIdx.x, NT = blockDim.x, ctas = gridDim.x, rank = blockIdx.x;
  pdl_wait();
  pdl_launch_next();
  first_of(a.requests, a.n, a.B, s_first);
  const int n_free = min(max(*a.n_free, 0), a.cap);
  int total = 0;
  for (int i0 = 0; i0 < a.n; i0 += NT) {
    const int i = i0 + tid;
    int count = 0, r = -1, from = 0;
    if (i < a.n) {
      const int b = a.requests[i], keep = a.keep ? a.keep[i] : 0;
      bool bad = b < 0 || b >= a.B || s_first[b] != i || keep < 0;
      if (!bad) {
        const int held = a.held[b];
        from = ceil_pages(keep, a.shift);
        bad = held < 0 || held > a.W || from > held;
        if (!bad && keep & ((1 << a.shift) - 1)) {   // new tokens would go into the page where the cut ends
          const int p = a.tables[(size_t)b * a.W + from - 1];
          bad = p >= 0 && p < a.P && a.shares[p] > 0;
        }
        if (!bad) {
          r = b;
          count = held - from;
        }
      }
      s_row[i] = r;
      s_from[i] = from;
    }
    int t;
    const int before = scan_cta(count, t, warp_sums);
    if (i < a.n) s_at[i] = total + before;
    total += t;
  }
  if (tid == 0) s_at[a.n] = total;
  cluster_sync();   // held, n_free and shares have been read
  int all = 0;   // pages that go onto the stack
  with_run<FEW>(total, ctas * NT, [&](auto run) {
    constexpr int kRun = decltype(run)::value;
    // A stretch of the releases for each CTA, in rounds of kRun for each thread:
    // their pages, or -1 (one round, nearly always: they are looked up once).
    const int k0 = (int)((long long)total * rank / ctas), k1 = (int)((long long)total * (rank + 1) / ctas);
    const int round = NT * kRun, rounds = (k1 - k0 + round - 1) / round;
    int page[kRun];
    auto look_up = [&](int rd) {
      const int first = k0 + rd * round + tid * kRun;
      int i = first < k1 ? place_of(s_at, a.n - 1, first) : 0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const int k = first + e;
        page[e] = -1;
        if (k < k1) {
          while (k >= s_at[i + 1]) ++i;
          const int p = a.tables[(size_t)s_row[i] * a.W + s_from[i] + (k - s_at[i])];
          page[e] = p >= 0 && p < a.P ? p : -1;
        }
      }
    };
    if (rounds == 1) look_up(0);
    // Count the releases. A page that has as many as holders is left at -1.
    for (int rd = 0; rd < rounds; ++rd) {
      if (rounds > 1) look_up(rd);
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (page[e] >= 0) atomicSub(&a.shares[page[e]], 1);
    }
    cluster_sync();
    // Its first release claims it (claims lie below all counts: total < 2^30).
    for (int rd = 0; rd < rounds; ++rd) {
      if (rounds > 1) look_up(rd);
      const int first = k0 + rd * round + tid * kRun;
      int count[kRun];
#pragma unroll
      for (int e = 0; e < kRun; ++e) count[e] = page[e] >= 0 ? __ldcg(&a.shares[page[e]]) : 0;
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (count[e] < 0) atomicMin(&a.shares[page[e]], INT_MIN + first + e);
    }
    cluster_sync();
    // Claimed pages go onto the stack in the list's order: first how many they
    // are in each CTA's stretch, then where they go.
    auto claimed = [&](int rd) {   // bit e: release e of the thread's has its page
      const int first = k0 + rd * round + tid * kRun;
      int count[kRun], bits = 0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) count[e] = page[e] >= 0 ? __ldcg(&a.shares[page[e]]) : 0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) bits |= (page[e] >= 0 && count[e] == INT_MIN + first + e) << e;
      return bits;
    };
    int mine = 0, bits = 0;
    for (int rd = 0; rd < rounds; ++rd) {
      if (rounds > 1) look_up(rd);
      bits = claimed(rd);
      mine += __popc(bits);
    }
    int of_cta;
    scan_cta(mine, of_cta, warp_sums);
    if (tid == 0) s_mine = of_cta;
    cluster_sync();
    int at = n_free;
    for (int c = 0; c < ctas; ++c) {
      int x;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(dsmem_addr(smem_u32(&s_mine), c)) : "memory");
      at += c < rank ? x : 0;
      all += x;
    }
    for (int rd = 0; rd < rounds; ++rd) {
      if (rounds > 1) {
        look_up(rd);
        bits = claimed(rd);
      }
      int t;
      int pos = at + scan_cta(__popc(bits), t, warp_sums);
      at += t;
#pragma unroll
      for (int e = 0; e < kRun; ++e)
        if (bits >> e & 1) {
          if (pos < a.cap) a.free[pos] = page[e];
          a.shares[page[e]] = 0;
          ++pos;
        }
    }
  });
  if (rank == 0) {
    for (int i = tid; i < a.n; i += NT) {
      const int r = s_row[i];
      if (r >= 0) a.held[r] = s_from[i];
      a.status[i] = r >= 0 ? 0 : 2;
    }
    if (tid == 0) *a.n_free = min(n_free + all, a.cap);
  }
  cluster_sync();   // (the others' counts have been read)
}

struct ForkArgs {
  const int *src, *dst, *lens;
  int n;
  int* tables;
  int* held;
  int* shares;
  const int* free;
  int* n_free;
  int *source, *target, *slots, *status;
  int B, W, P, cap, shift;
};

template <bool FEW>   // one CTA of kFewThreads
__global__ void __launch_bounds__(FEW ? kFewThreads : kThreads, 1) k_page_fork(const ForkArgs a) {
  extern __shared__ int share_smem[];
  int* s_first = share_smem;        // [B]
  int* s_at = s_first + a.B;        // [n + 1] shared entries before
  int* s_src = s_at + a.n + 1;      // [n] source, or -1 when the fork is not made
  int* s_dst = s_src + a.n;         // [n]
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, NT = blockDim.x, ctas = gridDim.x, rank = blockIdx.x;
  pdl_wait();
  pdl_launch_next();
  first_of(a.dst, a.n, a.B, s_first);
  const int top = min(max(*a.n_free, 0), a.cap);
  int total = 0, wants = 0;
  for (int i0 = 0; i0 < a.n; i0 += NT) {
    const int i = i0 + tid;
    int s = -1, d = -1, len = 0, status = 2, want = 0;
    if (i < a.n) {
      s = a.src[i];
      d = a.dst[i];
      if (s >= 0 && s < a.B && d >= 0 && d < a.B && s != d && s_first[d] == i) {
        len = a.lens[s];
        const int held = a.held[s];
        if (len >= 0 && held <= a.W && ceil_pages(len, a.shift) <= held && a.held[d] == 0) {
          status = 0;
          want = (len & ((1 << a.shift) - 1)) > 0;
        }
      }
    }
    int t;
    const int before = wants + scan_cta(want, t, warp_sums);
    wants += t;
    if (want && before >= top) status = 1;
    const int full = status == 0 ? len >> a.shift : 0;
    const int at = total + scan_cta(full, t, warp_sums);
    total += t;
    if (i < a.n) {
      s_at[i] = at;
      s_src[i] = status == 0 ? s : -1;
      s_dst[i] = d;
      if (rank == 0) {
        int from = -1, to = -1;
        if (status == 0 && want) {
          from = a.tables[(size_t)s * a.W + full];
          to = a.free[top - 1 - before];
          a.tables[(size_t)d * a.W + full] = to;
        }
        a.source[i] = from;
        a.target[i] = to;
        a.slots[i] = to >= 0 ? len & ((1 << a.shift) - 1) : 0;
        a.status[i] = status;
      }
    }
  }
  if (tid == 0) s_at[a.n] = total;
  cluster_sync();   // held and n_free have been read
  with_run<FEW>(total, ctas * NT, [&](auto run) {
    constexpr int kRun = decltype(run)::value;
    for (int first = (rank * NT + tid) * kRun; first < total; first += ctas * NT * kRun) {
      int page[kRun];
      const int i0 = place_of(s_at, a.n - 1, first);
      int i = i0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const int k = first + e;
        if (k < total) {
          while (k >= s_at[i + 1]) ++i;
          page[e] = a.tables[(size_t)s_src[i] * a.W + (k - s_at[i])];
        }
      }
      i = i0;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        const int k = first + e;
        if (k < total) {
          while (k >= s_at[i + 1]) ++i;
          a.tables[(size_t)s_dst[i] * a.W + (k - s_at[i])] = page[e];
          if (page[e] >= 0 && page[e] < a.P) atomicAdd(&a.shares[page[e]], 1);
        }
      }
    }
  });
  if (rank == 0) {
    for (int i = tid; i < a.n; i += NT)
      if (s_src[i] >= 0) a.held[s_dst[i]] = ceil_pages(a.lens[s_src[i]], a.shift);
    if (tid == 0) *a.n_free = top - min(wants, top);
  }
}

struct CompactArgs {
  const int* tables;
  const int* held;
  const int* shares;
  int *tables_out, *shares_out, *free, *n_free, *source, *target, *count;
  int B, W, P, moves;
};

// Set bits before each block of 8 words, and words.
struct Used {
  const uint32_t* word;
  const int* block;   // [blocks + 1]
  int blocks;
  __device__ __forceinline__ bool at(int p) const { return word[p >> 5] >> (p & 31) & 1; }
  // Held pages below p.
  __device__ __forceinline__ int before(int p) const {
    int c = block[p >> 8];
    for (int w = p >> 8 << 3; w < p >> 5; ++w) c += __popc(word[w]);
    return (p & 31) ? c + __popc(word[p >> 5] & ((1u << (p & 31)) - 1)) : c;
  }
  // The page that r pages which nobody holds lie below.
  __device__ __forceinline__ int unheld(int r) const {
    int lo = 0, hi = blocks - 1;   // the block: unheld pages before it are at most r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (256 * mid - block[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    r -= 256 * lo - block[lo];
    int w = 8 * lo;
    while (w < 8 * blocks - 1 && r >= 32 - __popc(word[w])) r -= 32 - __popc(word[w++]);
    uint32_t x = ~word[w];
    for (; r > 0 && x; --r) x &= x - 1;
    return 32 * w + __ffs(x) - 1;
  }
};

__global__ void __launch_bounds__(kThreads) k_page_compact(const CompactArgs a) {
  extern __shared__ int share_smem[];
  const int blocks = (a.P + 255) / 256, words = 8 * blocks;
  uint32_t* s_word = reinterpret_cast<uint32_t*>(share_smem);   // [words] a bit for every page that is held
  int* s_block = share_smem + words;                            // [blocks + 1]
  int* s_at = s_block + blocks + 1;                             // [B + 1] entries before
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, NT = blockDim.x, ctas = gridDim.x, rank = blockIdx.x;
  pdl_wait();
  pdl_launch_next();
  for (int w = tid; w < words; w += NT) s_word[w] = 0;
  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + tid;
    int t;
    const int at = total + scan_cta(b < a.B ? min(max(a.held[b], 0), a.W) : 0, t, warp_sums);
    if (b < a.B) s_at[b] = at;
    total += t;
  }
  if (tid == 0) s_at[a.B] = total;
  __syncthreads();
  // Every CTA marks the pages of its share of the entries; then each joins all
  // marks of its share of the words.
  for (int k = rank * NT + tid; k < total; k += ctas * NT) {
    const int b = place_of(s_at, a.B - 1, k);
    const int p = a.tables[(size_t)b * a.W + (k - s_at[b])];
    if (p >= 0 && p < a.P) atomicOr(&s_word[p >> 5], 1u << (p & 31));
  }
  cluster_sync();
  for (int w = rank * NT + tid; w < words; w += ctas * NT) {
    uint32_t x = 0;
    for (int c = 0; c < ctas; ++c) {
      uint32_t y;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(y) : "r"(dsmem_addr(smem_u32(&s_word[w]), c)) : "memory");
      x |= y;
    }
    for (int c = 0; c < ctas; ++c)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(smem_u32(&s_word[w]), c)), "r"(x) : "memory");
  }
  cluster_sync();   // (and all have read the tables)
  int held = 0;
  for (int q0 = 0; q0 < blocks; q0 += NT) {
    const int q = q0 + tid;
    int c = 0;
    if (q < blocks)
      for (int i = 0; i < 8; ++i) c += __popc(s_word[8 * q + i]);
    int t;
    const int at = held + scan_cta(c, t, warp_sums);
    if (q < blocks) s_block[q] = at;
    held += t;
  }
  if (tid == 0) s_block[blocks] = held;
  __syncthreads();
  const Used used{s_word, s_block, blocks};
  const int low = held < a.P ? used.before(held) : held;   // held pages that stay
  auto to = [&](int p) { return p < held ? p : used.unheld(used.before(p) - low); };
  const int first = rank * NT + tid, step = ctas * NT;
  for (int k = first; k < a.B * a.W; k += step) {
    const int b = k / a.W, p = a.tables[k];
    const bool live = k - b * a.W < s_at[b + 1] - s_at[b] && p >= 0 && p < a.P;
    const int t = live ? to(p) : p;
    if (t != p || a.tables_out != a.tables) a.tables_out[k] = t;
  }
  for (int p = first; p < a.P; p += step) {
    const bool h = used.at(p);
    if (p < held) {
      if (h && a.shares_out != a.shares) a.shares_out[p] = a.shares[p];
      continue;
    }
    if (h) {
      const int i = used.before(p) - low, t = used.unheld(i);
      a.shares_out[t] = a.shares[p];
      a.source[i] = p;
      a.target[i] = t;
    }
    a.shares_out[p] = 0;
  }
  for (int i = held - low + first; i < a.moves; i += step) a.source[i] = a.target[i] = -1;
  for (int i = first; i < a.P - held; i += step) a.free[i] = a.P - 1 - i;
  if (rank == 0 && tid == 0) {
    *a.n_free = a.P - held;
    *a.count = held - low;
  }
}

// Launches a cluster of CTAs, or one small CTA for at most kFew entries and
// requests, as the tables could hold them (us, one CTA and a cluster: a release
// that finds nothing 4.4 and 6.2, a compaction of 97 pages 5.3 and 6.1; a release
// and a fork in tables of 336 entries 12.2 and 15.3, 672 12.1 and 14.9, 1408 23.9
// and 16.4).
constexpr long kFew = 1024;
template <typename Args>
cudaError_t launch_share(void (*fn)(Args), const Args& a, bool few, size_t smem, std::atomic<uint64_t>& ready,
                         cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1))) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = few ? 1 : kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(few ? 1 : kCluster);
  cfg.blockDim = dim3(few ? kFewThreads : kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

struct Array {
  const int32_t* at;
  int64_t n;
  bool written;
};
sf_status check_apart(const char* who, std::initializer_list<Array> arrays) {
  Range r[16];
  int n = 0;
  for (const Array& x : arrays) r[n++] = Range{x.at, (uint64_t)x.n * sizeof(int32_t), x.written};
  return ranges_apart(r, n) ? SF_OK : set_error(SF_ERR_ARG, "%s: an array that the call writes overlaps another", who);
}

// What the three calls refuse alike.
sf_status check_tables(const char* who, int32_t batch, int32_t table_width, int32_t n_pages) {
  if (batch < 1 || batch > kMaxPlanBatch)
    return set_error(SF_ERR_ARG, "%s: batch %d outside 1..%d", who, batch, kMaxPlanBatch);
  if (table_width < 1 || (int64_t)batch * table_width >= 1 << 30)
    return set_error(SF_ERR_ARG, "%s: need 1 <= table_width and batch * table_width < 2^30", who);
  if (n_pages < 1) return set_error(SF_ERR_ARG, "%s: need n_pages >= 1", who);
  return SF_OK;
}
sf_status check_list(const char* who, int32_t n, int32_t page, int32_t table_width, int32_t capacity) {
  if (n < 0 || n > kMaxPlanBatch) return set_error(SF_ERR_ARG, "%s: %d requests, outside 0..%d", who, n, kMaxPlanBatch);
  if (!page_ok(page)) return set_error(SF_ERR_ARG, "%s: page must be 16, 32, 64, 128 or 256", who);
  if (table_width > (1 << 30) / page || (int64_t)n * table_width >= 1 << 30 || capacity < 1)
    return set_error(SF_ERR_ARG, "%s: need table_width <= 2^30 / page, n * table_width < 2^30 and capacity >= 1", who);
  return SF_OK;
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" sf_status sf_page_free(const int32_t* d_requests, const int32_t* d_keep, int32_t n, int32_t batch, int32_t page,
                                  int32_t* d_tables, int32_t table_width, int32_t* d_held, int32_t* d_shares,
                                  int32_t n_pages, int32_t* d_free, int32_t capacity, int32_t* d_n_free,
                                  int32_t* d_status, void* cuda_stream) {
  sf_status s = check_tables("sf_page_free", batch, table_width, n_pages);
  if (s == SF_OK) s = check_list("sf_page_free", n, page, table_width, capacity);
  if (s != SF_OK) return s;
  if (n == 0) return SF_OK;
  if (!d_requests || !d_tables || !d_held || !d_shares || !d_free || !d_n_free || !d_status)
    return set_error(SF_ERR_ARG, "sf_page_free: null pointer");
  s = check_apart("sf_page_free", {{d_requests, n, false}, {d_keep, n, false}, {d_tables, (int64_t)batch * table_width, false},
                                   {d_held, batch, true}, {d_shares, n_pages, true}, {d_free, capacity, true},
                                   {d_n_free, 1, true}, {d_status, n, true}});
  if (s != SF_OK) return s;
  static std::atomic<uint64_t> ready[2];
  const bool few = (long)n * table_width + batch <= kFew;
  const FreeArgs a{d_requests, d_keep, n, d_tables, d_held, d_shares, d_free, d_n_free, d_status, batch, table_width,
                   n_pages, capacity, log2_of(page)};
  const cudaError_t e = launch_share(few ? k_page_free<true> : k_page_free<false>, a, few,
                                     ((size_t)batch + 3 * n + 1) * sizeof(int), ready[few],
                                     static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_free: %s", cudaGetErrorString(e));
  return SF_OK;
}

extern "C" sf_status sf_page_fork(const int32_t* d_src, const int32_t* d_dst, int32_t n, const int32_t* d_lens,
                                  int32_t batch, int32_t page, int32_t* d_tables, int32_t table_width, int32_t* d_held,
                                  int32_t* d_shares, int32_t n_pages, const int32_t* d_free, int32_t capacity,
                                  int32_t* d_n_free, int32_t* d_source, int32_t* d_target, int32_t* d_slots,
                                  int32_t* d_status, void* cuda_stream) {
  sf_status s = check_tables("sf_page_fork", batch, table_width, n_pages);
  if (s == SF_OK) s = check_list("sf_page_fork", n, page, table_width, capacity);
  if (s != SF_OK) return s;
  if (n == 0) return SF_OK;
  if (!d_src || !d_dst || !d_lens || !d_tables || !d_held || !d_shares || !d_free || !d_n_free || !d_source || !d_target ||
      !d_slots || !d_status)
    return set_error(SF_ERR_ARG, "sf_page_fork: null pointer");
  s = check_apart("sf_page_fork", {{d_src, n, false}, {d_dst, n, false}, {d_lens, batch, false},
                                   {d_tables, (int64_t)batch * table_width, true}, {d_held, batch, true},
                                   {d_shares, n_pages, true}, {d_free, capacity, false}, {d_n_free, 1, true},
                                   {d_source, n, true}, {d_target, n, true}, {d_slots, n, true}, {d_status, n, true}});
  if (s != SF_OK) return s;
  static std::atomic<uint64_t> ready[2];
  const bool few = (long)n * table_width + batch <= kFew;
  const ForkArgs a{d_src, d_dst, d_lens, n, d_tables, d_held, d_shares, d_free, d_n_free, d_source, d_target, d_slots,
                   d_status, batch, table_width, n_pages, capacity, log2_of(page)};
  const cudaError_t e = launch_share(few ? k_page_fork<true> : k_page_fork<false>, a, few,
                                     ((size_t)batch + 3 * n + 1) * sizeof(int), ready[few],
                                     static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_fork: %s", cudaGetErrorString(e));
  return SF_OK;
}

extern "C" sf_status sf_page_compact(const int32_t* d_tables, int32_t batch, int32_t table_width, const int32_t* d_held,
                                     const int32_t* d_shares, int32_t n_pages, int32_t* d_tables_out,
                                     int32_t* d_shares_out, int32_t* d_free, int32_t capacity, int32_t* d_n_free,
                                     int32_t* d_source, int32_t* d_target, int32_t moves, int32_t* d_count,
                                     void* cuda_stream) {
  sf_status s = check_tables("sf_page_compact", batch, table_width, n_pages);
  if (s != SF_OK) return s;
  if (n_pages > kMaxPages) return set_error(SF_ERR_UNSUPPORTED, "sf_page_compact: n_pages %d above %d", n_pages, kMaxPages);
  if (capacity < n_pages || moves < n_pages / 2)
    return set_error(SF_ERR_ARG, "sf_page_compact: the stack needs room for all pages, source and target for half of them");
  if (!d_tables || !d_held || !d_shares || !d_tables_out || !d_shares_out || !d_free || !d_n_free || !d_count ||
      (moves > 0 && (!d_source || !d_target)))
    return set_error(SF_ERR_ARG, "sf_page_compact: null pointer");
  const int64_t entries = (int64_t)batch * table_width;
  s = check_apart("sf_page_compact", {{d_tables == d_tables_out ? nullptr : d_tables, entries, false},
                                      {d_shares == d_shares_out ? nullptr : d_shares, n_pages, false},
                                      {d_held, batch, false}, {d_tables_out, entries, true}, {d_shares_out, n_pages, true},
                                      {d_free, capacity, true}, {d_n_free, 1, true}, {d_source, moves, true},
                                      {d_target, moves, true}, {d_count, 1, true}});
  if (s != SF_OK) return s;
  static std::atomic<uint64_t> ready{0};
  const CompactArgs a{d_tables, d_held, d_shares, d_tables_out, d_shares_out, d_free, d_n_free, d_source, d_target,
                      d_count, batch, table_width, n_pages, moves};
  const size_t blocks = ((size_t)n_pages + 255) / 256;
  const cudaError_t e = launch_share(k_page_compact, a, (long)batch * table_width + n_pages <= kFew, (9 * blocks + 1 + batch + 1) * sizeof(int), ready,
                                     static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_compact: %s", cudaGetErrorString(e));
  return SF_OK;
}
