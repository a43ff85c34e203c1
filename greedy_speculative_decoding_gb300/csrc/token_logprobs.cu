// Log probabilities of given tokens from rows of logits, with entropy, rank
// and the top alternatives (sf_token_logprobs).
//
// One pass over a row x: with the maximum m, s = sum e^(x_v - m) and
// t = sum e^(x_v - m) (x_v - m),
//   log p_v = (x_v - m) - log s,   entropy = log s - t / s.
// Every thread keeps m, s and t of its own elements (a new maximum m' turns s
// into f s and t into f (t + (m - m') s), f = e^(m - m')), and counts those in
// front of the given token. Everything in fp32, joined in a fixed order.
//
// The k top alternatives need no sort of the row. A group of four threads
// knows the largest of its elements; the k largest of these maxima are k
// elements, so nothing below the k-th of them can be among the top k, and
// nothing of the other groups either. Only the elements of those k groups are
// looked at again (from L2), and the few that reach the bound are put in order.
//
// Order: larger logits first, equal ones by token; a NaN counts as -infinity.
//
// A row is read once; it is one CTA's, or with few rows a cluster's, each CTA a
// stretch of it, joined through distributed shared memory. A thread copies its
// vectors to places of its own in shared memory (cp.async), two times four on
// their way while it works on four, so that memory does not wait for the
// arithmetic (us: loaded into registers behind it, 1021 rows of 152064 bf16
// logits 74, now 65; 400 fp32 rows 47.5, now 40; once four on their way 73 and 49,
// three or four times two 71 and 42). 1021 rows of bf16 run at 4.8 TB/s, 400 of
// fp32 at 6.0; 72 fp32 rows take 10.8 and with 20 alternatives 19, one row 6.5 and
// with five 9.7: few rows are a chain of loads, reductions, the second look and
// the cluster's barriers; many are bound by memory in fp32, and in 16 bits by the
// six instructions of an element and by the last wave's empty places. CTAs of 256
// threads, four on an SM, so that some stream while others choose (with loads
// into registers, 1021 rows 74 and 72 rows 13.6: of 512 threads 89 and 19.1, of
// 128 76 and 30).
#include <algorithm>
#include <type_traits>

#include "paged.h"

namespace sf {
namespace {

constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;          // (of 4: one row 8.9 us for 6.8; of 16: 5.8 for 6.3, but with five 9.5 for 9.4, 16 rows 12.4 for 10.8)
constexpr int kBuffer = 1024;           // elements that reach the bound; more (rows made for it) are handled apart
constexpr int kAhead = 4;               // vectors that a thread works on together
constexpr int kStages = 2;              // as often as many on their way
constexpr float kLog2E = 1.44269504088896f;

struct ScoreArgs {
  const void* x;
  long row;
  const int* tokens;
  long first;             // the launch's first row
  int ctas, vocab, top;   // (CTAs of a row)
  // 1: another launch does the rest of the rows. 2: that launch. It starts when
  // every CTA of the first has waited for what comes before both, so that is
  // done, and it touches nothing that the first one writes; before its own end it
  // waits for the first one's, as what follows looks at the second alone. (620
  // rows of 152064 bf16 logits 38 us; with the wait in front of its reads 43, in one
  // launch of a CTA a row 43, of clusters 76.)
  int chain;
  float *logprob, *entropy;
  int *rank, *top_ids;
  float* top_logprobs;
};

__device__ __forceinline__ float exp2_fast(float x) {   // relative error 2^-22; 0 below the normal range
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ float to_float(T v) { return static_cast<float>(v); }

// Pairs of fp32 numbers at once.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(__float_as_uint(x)), "r"(__float_as_uint(y)));
  return d;
}
__device__ __forceinline__ float2 unpair(uint64_t d) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(d));
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sixteen bytes of a row.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  using T2 = typename std::conditional<std::is_same<T, bf16>::value, __nv_bfloat162, __half2>::type;
  uint4 w;
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u = word(i * (int)sizeof(T) / 4);
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    else if constexpr (std::is_same<T, bf16>::value) return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
    else return i & 1 ? __high2float(*reinterpret_cast<const __half2*>(&u)) : __low2float(*reinterpret_cast<const __half2*>(&u));
  }
  // A number whose exponential is 0 under every reference from half of it on.
  static constexpr float kLow = std::is_same<T, __half>::value ? -65504.f : -1.0e30f;
  // The elements, those below kLow raised to it (of -infinity, an exponential 0
  // times the exponent would be NaN); a NaN stays. 16 bits: in pairs.
  __device__ __forceinline__ Vec raised() const {
    Vec r;
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[i] = word(i);
      if constexpr (sizeof(T) == 4) {
        u[i] = __float_as_uint(max_nan(__uint_as_float(u[i]), kLow));
      } else {
        T2 low;
        if constexpr (std::is_same<T, bf16>::value) low = __float2bfloat162_rn(kLow);
        else low = __float2half2_rn(kLow);
        const T2 y = __hmax2_nan(*reinterpret_cast<const T2*>(&u[i]), low);
        u[i] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    r.w = make_uint4(u[0], u[1], u[2], u[3]);
    return r;
  }
  // The larger of its elements and mx (a NaN counts as -infinity); 16 bits: in pairs.
  static __device__ __forceinline__ float max_of(const Vec (&v)[kAhead]) {
    if constexpr (sizeof(T) == 4) {
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int u = 0; u < kAhead; u += 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = fmaxf(fmaxf(m[i], v[u].get(i)), v[u + 1].get(i));
      return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    } else {
      T2 m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = v[0].word(i);
        m[i] = *reinterpret_cast<const T2*>(&x);
      }
#pragma unroll
      for (int u = 1; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = v[u].word(i);
          m[i] = __hmax2(m[i], *reinterpret_cast<const T2*>(&x));
        }
      const T2 r = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
      return fmaxf(fmaxf(__low2float(r), __high2float(r)), -INFINITY);   // (two NaN: -infinity)
    }
  }
  // How many of the elements are above `bound` (OR_EQUAL: or equal to it), a number of the type or an infinity.
  template <bool OR_EQUAL>
  static __device__ __forceinline__ int above(const Vec (&v)[kAhead], float bound) {
    int n = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) n += OR_EQUAL ? v[u].get(i) >= bound : v[u].get(i) > bound;
    } else {
      T2 b, sum;
      if constexpr (std::is_same<T, bf16>::value) b = __float2bfloat162_rn(bound), sum = __float2bfloat162_rn(0.f);
      else b = __float2half2_rn(bound), sum = __float2half2_rn(0.f);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = v[u].word(i);
          const T2 y = *reinterpret_cast<const T2*>(&x);
          sum = __hadd2(sum, OR_EQUAL ? __hge2(y, b) : __hgt2(y, b));   // (ones and zeros; exact)
        }
      n = (int)(__low2float(sum) + __high2float(sum));
    }
    return n;
  }
};

// Running maximum, sum of exponentials and of exponentials times exponent.
struct Sums {
  float m, s, t;
  // Moves the reference up to `to` (at least m).
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      if (m != -INFINITY) {   // (else s and t are 0, or NaN)
        const float d = fmaxf(m - to, -1.0e20f), f = exp2_fast(d * kLog2E);   // (f = 0 times an infinity is NaN)
        t = f * fmaf(s, d, t);
        s *= f;
      }
      m = to;
    }
  }
  __device__ __forceinline__ void add(float x) {   // m is at least x
    if (m == -INFINITY) {                          // (then it adds nothing; a NaN stays)
      if (x != x) s = x;
      return;
    }
    const float d = max_nan(x - m, -1.0e30f), e = exp2_fast(d * kLog2E);   // (e = 0 times -infinity is NaN)
    s += e;
    t = fmaf(e, d, t);
  }
  __device__ __forceinline__ void join(Sums o) {
    const float to = fmaxf(m, o.m);
    raise(to);
    o.raise(to);
    s += o.s;
    t += o.t;
  }
  __device__ __forceinline__ Sums shuffled(int o) const {
    return {__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, t, o)};
  }
};

// (logit, token) as a number: larger logits first, then lower tokens. Never 0.
__device__ __forceinline__ unsigned long long order_key(float x, int v) {
  return argmax_key((x == x ? x : -INFINITY) + 0.f, v);   // (-0 is 0)
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <int N>
__device__ __forceinline__ void copy_wait() {   // until all but the last N groups of cp_async16 have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a CTA of a cluster leaves for the first one.
struct Share {
  Sums sums;
  int rank;
  unsigned long long top[kMaxTop];
};

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_token_logprobs(const __grid_constant__ ScoreArgs a) {
  using V = Vec<T>;
  constexpr int kGroups = kThreads / 4;   // groups of four threads, for the top alternatives
  __shared__ uint4 s_ring[kStages][kAhead][kThreads];   // (each thread its own places)
  __shared__ Sums s_sums[kThreads / 32];
  __shared__ int s_rank[kThreads / 32];
  __shared__ __align__(16) float s_max[kGroups];
  __shared__ int s_first[kGroups], s_tied[kGroups];   // (ties at the bound: first token of a group that is equal to it)
  __shared__ int s_groups[kMaxTop];      // the groups whose elements are looked at again
  __shared__ unsigned long long s_bound, s_buffer[kBuffer], s_best[kThreads / 32], s_final[kMaxTop];
  __shared__ int s_count, s_picked, s_ties;
  __shared__ Share s_share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = tid >> 2;
  const int ctas = a.ctas, part = ctas > 1 ? (int)cluster_rank() : 0;
  if (a.chain < 2) pdl_wait();
  if (a.chain == 1) pdl_launch_next();
  const long row = a.first + (ctas > 1 ? blockIdx.x / ctas : blockIdx.x);
  const int token = a.tokens[row];
  const T* x = static_cast<const T*>(a.x) + row * a.row;
  // The row as a few elements up to a 16-byte boundary, vectors, a few elements:
  // of the vectors each CTA has a stretch, the first one the rest as well.
  const int head = min(a.vocab, (int)((-reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)));
  const int nv = (a.vocab - head) / V::N, body = head + nv * V::N;
  const int v0 = (int)((long)nv * part / ctas), v1 = (int)((long)nv * (part + 1) / ctas);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);

  // The element of the head or the tail that a thread has: a token, or -1.
  auto odd_of = [&](int t) {
    return part > 0 ? -1 : t < head ? t : t >= 16 && t - 16 < a.vocab - body ? body + t - 16 : -1;
  };
  // Vectors i, i + kThreads, ... of this thread on their way; behind the stretch: -infinity.
  const uint32_t none_bits = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, bf16>::value ? 0xff80ff80u : 0xfc00fc00u;
  auto fetch = [&](int s, int i) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + u * kThreads < v1) cp_async16(&s_ring[s][u][tid], xv + i + u * kThreads);
      else s_ring[s][u][tid] = make_uint4(none_bits, none_bits, none_bits, none_bits);
    }
    cp_async_commit();
  };
  int i = v0 + tid, stage = 0;
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(s, i + s * kAhead * kThreads);   // (before the token is known)
  if (token < 0 || token >= a.vocab) {         // (the whole cluster)
    cp_async_wait_all();
    if (a.chain == 2) pdl_wait();
    return;
  }
  const int odd = odd_of(tid);
  const float odd_x = odd >= 0 ? to_float(x[odd]) : -INFINITY;
  const float given_x = to_float(x[token]);
  const float given = given_x == given_x ? given_x : -INFINITY;
  // In front of the given token: larger logits, equal ones of lower tokens (with
  // -infinity or NaN given, every lower token, counted at the end).
  const bool all_before = given == -INFINITY;
  const int given_v = token >= head && token < body ? (token - head) / V::N : -1;   // its vector
  int rank = 0;
  auto count_one = [&](float f, int v) { rank += all_before ? v > token && f > given : v < token ? f >= given : f > given; };

  Sums z = {-INFINITY, 0.f, 0.f};
  if (odd >= 0) {
    z.raise(odd_x);
    z.add(odd_x);
    count_one(odd_x, odd);
  }
#pragma unroll 1
  for (; i < v1; i += kAhead * kThreads) {
    copy_wait<kStages - 1>();
    V v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u].w = s_ring[stage][u][tid];
    z.raise(V::max_of(v));
    if (z.m < V::kLow / 2) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < V::N; ++e) z.add(v[u].get(e));
    } else {
      const uint64_t m2 = pair(-z.m, -z.m), c2 = pair(kLog2E, kLog2E);
      uint64_t s2[2] = {pair(z.s, 0.f), 0}, t2[2] = {pair(z.t, 0.f), 0};
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const V x = v[u].raised();
#pragma unroll
        for (int e = 0; e < V::N; e += 2) {
          const uint64_t d2 = add2(pair(x.get(e), x.get(e + 1)), m2);
          const float2 y = unpair(mul2(d2, c2));
          const uint64_t e2 = pair(exp2_fast(y.x), exp2_fast(y.y));
          s2[e / 2 & 1] = add2(s2[e / 2 & 1], e2);
          t2[e / 2 & 1] = fma2(e2, d2, t2[e / 2 & 1]);
        }
      }
      const float2 s = unpair(add2(s2[0], s2[1])), t = unpair(add2(t2[0], t2[1]));
      z.s = s.x + s.y;
      z.t = t.x + t.y;
    }
    if (i + (kAhead - 1) * kThreads < given_v || (given_v < 0 && token >= body)) {   // all of them before it
      if (!all_before) rank += V::template above<true>(v, given);
    } else if (i > given_v) {
      rank += V::template above<false>(v, given);
    } else {
#pragma unroll 1
      for (int u = 0; u < kAhead; ++u) {
        const V y = {s_ring[stage][u][tid]};
#pragma unroll
        for (int e = 0; e < V::N; ++e) count_one(y.get(e), head + (i + u * kThreads) * V::N + e);
      }
    }
    fetch(stage, i + kStages * kAhead * kThreads);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  if (all_before && tid == 0 && part == 0) rank += token;

  // ---- join the threads' sums
  float gm = z.m;
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
  if ((tid & 3) == 0) s_max[group] = gm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z.join(z.shuffled(o));
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
  }
  if (lane == 0) {
    s_sums[warp] = z;
    s_rank[warp] = rank;
  }
  if (tid == 0) s_count = s_picked = s_ties = 0;
  if (tid < kMaxTop) s_share.top[tid] = 0;
  __syncthreads();
  if (warp == 0) {
    z = lane < kThreads / 32 ? s_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
    rank = lane < kThreads / 32 ? s_rank[lane] : 0;
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) {
      z.join(z.shuffled(o));
      rank += __shfl_xor_sync(0xffffffffu, rank, o);
    }
    if (lane == 0) {
      s_share.sums = z;
      s_share.rank = rank;
    }
  }

  // ---- the groups with the k largest maxima
  const int k = a.top;
  if (k > 0) {
    const float mine = s_max[group];
    int larger = 0, equal = 0;
#pragma unroll
    for (int g = 0; g < kGroups / 16; ++g) {   // (a thread of the group a quarter of them)
      const float4 o = reinterpret_cast<const float4*>(s_max)[(tid & 3) * (kGroups / 16) + g];
      larger += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
      equal += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      larger += __shfl_xor_sync(0xffffffffu, larger, o);
      equal += __shfl_xor_sync(0xffffffffu, equal, o);
    }
    const bool first = (tid & 3) == 0;         // (a group's first thread decides)
    if (first && larger < k && larger + equal >= k) {   // the k-th largest
      s_bound = (unsigned long long)float_key(mine + 0.f) << 32;
      s_ties = larger + equal > k;
    }
    __syncthreads();
    const float at = key_value(s_bound);
    // The elements of n groups, by the threads of the CTA together (n <= kGroups).
    const int per = (v1 - v0 + kThreads - 1) / kThreads * 4;   // places for a group's vectors
    auto each = [&](const int* groups, int n, auto f) {
      if (tid < 4 * n) {
        const int g = groups[tid >> 2], w = odd_of(4 * g + (tid & 3));
        if (w >= 0) f(to_float(x[w]), w, g);
      }
#pragma unroll 1
      for (int j = tid; j < n * per; j += kThreads) {
        const int p = j / per, r = j - p * per, g = groups[p], w = v0 + (r >> 2) * kThreads + 4 * g + (r & 3);
        if (w < v1) {
          const V y = {xv[w]};   // (not through the read-only path: the kernel may start before the logits' writer has ended)
#pragma unroll
          for (int e = 0; e < V::N; ++e) f(y.get(e), head + w * V::N + e, g);
        }
      }
    };
    if (s_ties) {   // more maxima equal to the bound than there is room for: the lowest tokens first
      if (first) s_first[group] = INT32_MAX;
      if (first && mine == at) s_tied[atomicAdd(&s_count, 1)] = group;
      __syncthreads();
      each(s_tied, s_count, [&](float v, int t, int g) {
        if ((v == v ? v : -INFINITY) == at) atomicMin(&s_first[g], t);
      });
      __syncthreads();
      if (tid == 0) s_count = 0;
      if (first && mine == at) {
        int before_me = larger;
        for (int g = 0; g < kGroups; ++g) before_me += s_max[g] == at && s_first[g] < s_first[group];
        if (before_me < k && s_first[group] != INT32_MAX) s_groups[atomicAdd(&s_picked, 1)] = group;   // (not one without elements)
        if (before_me == k - 1 && s_first[group] != INT32_MAX) s_bound = order_key(at, s_first[group]);
      } else if (first && larger < k) {
        s_groups[atomicAdd(&s_picked, 1)] = group;
      }
    } else if (first && mine >= at) {
      s_groups[atomicAdd(&s_picked, 1)] = group;
    }
    __syncthreads();

    // ---- their elements from the bound on, put in order
    const unsigned long long bound = s_bound;
    each(s_groups, s_picked, [&](float v, int t, int) {
      const unsigned long long key = order_key(v, t);
      if (key >= bound) {
        const int c = atomicAdd(&s_count, 1);
        if (c < kBuffer) s_buffer[c] = key;
      }
    });
    __syncthreads();
    const int count = s_count;
    if (count <= kBuffer) {
      for (int c = tid; c < count; c += kThreads) {
        const unsigned long long key = s_buffer[c];
        int r = 0;
        for (int j = 0; j < count; ++j) r += s_buffer[j] > key;
        if (r < k) s_share.top[r] = key;
      }
    } else {   // one after the other
      unsigned long long last = ~0ull;
      for (int r = 0; r < k; ++r) {
        unsigned long long best = 0;
        each(s_groups, s_picked, [&](float v, int t, int) {
          const unsigned long long key = order_key(v, t);
          if (key < last && key > best) best = key;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long u = __shfl_xor_sync(0xffffffffu, best, o);
          best = u > best ? u : best;
        }
        if (lane == 0) s_best[warp] = best;
        __syncthreads();
        best = s_best[0];
        for (int w = 1; w < kThreads / 32; ++w) best = s_best[w] > best ? s_best[w] : best;
        if (tid == 0) s_share.top[r] = best;
        last = best;
        __syncthreads();
      }
    }
  }

  // ---- the cluster's shares, joined by its first CTA
  const unsigned long long* top = s_share.top;
  if (ctas > 1) {
    cluster_sync();
    if (part == 0) {
      if (k > 0) {
        for (int c = tid; c < ctas * k; c += kThreads) {
          unsigned long long key;
          asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(key) : "r"(dsmem_addr(smem_u32(&s_share.top[c % k]), c / k)) : "memory");
          s_buffer[c] = key;
        }
        __syncthreads();
        for (int c = tid; c < ctas * k; c += kThreads) {
          const unsigned long long key = s_buffer[c];
          if (key == 0) continue;              // (a stretch of fewer than k elements)
          int r = 0;                           // the larger ones, list by list (each in order)
          for (int q = 0; q < ctas; ++q) {
            int lo = 0;
#pragma unroll
            for (int step = kMaxTop / 2; step > 0; step >>= 1)
              if (lo + step <= k && s_buffer[q * k + lo + step - 1] > key) lo += step;
            if (lo < k && s_buffer[q * k + lo] > key) ++lo;
            r += lo;
          }
          if (r < k) s_final[r] = key;
        }
        top = s_final;
      }
      if (tid < ctas) {
        const uint32_t at = dsmem_addr(smem_u32(&s_share), tid);
        s_sums[tid] = {ld_dsmem(at), ld_dsmem(at + 4), ld_dsmem(at + 8)};
        s_rank[tid] = __float_as_int(ld_dsmem(at + 12));
      }
      __syncthreads();
      if (tid == 0) {
        z = s_sums[0];
        rank = s_rank[0];
        for (int c = 1; c < ctas; ++c) {
          z.join(s_sums[c]);
          rank += s_rank[c];
        }
        s_share.sums = z;
        s_share.rank = rank;
      }
    }
    cluster_sync();   // (the shares have been read)
    if (part > 0) {
      if (a.chain == 2) pdl_wait();
      return;
    }
  } else {
    __syncthreads();
  }
  // log p = (x - m) - log s; a row of -infinity alone has none above -infinity.
  const Sums all = s_share.sums;
  const bool none = all.m == -INFINITY && all.s == 0.f;
  const float logs = logf(all.s);
  auto logp = [&](float v) { return none ? -INFINITY : (v - all.m) - logs; };
  if (tid == 0) {
    if (a.logprob) a.logprob[row] = logp(given_x);
    if (a.entropy) a.entropy[row] = none ? 0.f : logs - all.t / all.s;
    if (a.rank) a.rank[row] = s_share.rank;
  }
  if (tid < k) {
    const unsigned long long key = top[tid];
    if (a.top_ids) a.top_ids[row * k + tid] = key_index(key);
    if (a.top_logprobs) a.top_logprobs[row * k + tid] = logp(key_value(key));
  }
  if (a.chain == 2) pdl_wait();
}

constexpr int kCtaThreads = 256;

// CTAs of a row for n rows of less than a wave. By what was measured, in us: a CTA
// alone takes 0.1 (16 bits: 0.05) for a thousand elements, half as much again with
// alternatives; a cluster 1.2 and 0.007 for every CTA in all, of which a third stays
// where memory, at 7 TB/s, is what bounds the call. us with 1 / 2 / 4 / 8 CTAs a row,
// [] the choice, fp32: 152064 elements, 1 row 16.9 / 11.3 / 8.2 / [6.4], 72 17.7 / 11.9 /
// [10.8] / 11.8, with twenty first 35.7 / 22.6 / 18.0 / [19.0], 152 17.9 / [15.9] / 20.5 /
// 23.3; 32768, 1 row 6.2 / 5.6 / 5.0 / [4.8], 72 [6.5] / 6.0 / 6.3 / 7.5; 8192, 72 [4.2] /
// 4.7 / 5.7 / 7.5; bf16: 152064, 1 row 12.6 / 9.3 / 7.2 / [6.3], 72 13.4 / 9.9 / [9.4] /
// 11.1; 65536, 72 [7.9] / 6.8 / 7.2 / 8.2 (the furthest from the best of 132 measured).
int ctas_of(long n, int vocab, int dtype, bool top) {
  const bool f32 = dtype == SF_DT_F32;
  const double alone = vocab * (f32 ? 1e-4 : 5e-5) * (top ? 1.5 : 1.0), memory = (double)n * vocab * (f32 ? 4 : 2) / 7e6;
  int best = 1;
  double least = 1e30;
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    const double more = c > 1 ? 0.007 * (double)n * c : 0.0;
    const double cost = std::max(alone / c + (c > 1 ? 1.2 : 0.0) + more, memory + 0.3 * more);
    if (cost < least) least = cost, best = c;
  }
  return best;
}

// Rows first .. first + n - 1.
cudaError_t launch_rows(ScoreArgs a, int dtype, long first, long n, int ctas, cudaStream_t st) {
  a.first = first;
  a.ctas = ctas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n * ctas));
  cfg.blockDim = dim3(kCtaThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return dtype == SF_DT_F32    ? cudaLaunchKernelEx(&cfg, k_token_logprobs<float, kCtaThreads>, a)
         : dtype == SF_DT_BF16 ? cudaLaunchKernelEx(&cfg, k_token_logprobs<bf16, kCtaThreads>, a)
                               : cudaLaunchKernelEx(&cfg, k_token_logprobs<__half, kCtaThreads>, a);
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" sf_status sf_token_logprobs(const void* d_logits, int32_t dtype, int64_t row_stride, int32_t n, int32_t vocab,
                                       const int32_t* d_tokens, int32_t top, float* d_logprob, float* d_entropy,
                                       int32_t* d_rank, int32_t* d_top_ids, float* d_top_logprobs, void* cuda_stream) {
  if (n < 0 || vocab < 1 || vocab > INT32_MAX - 64)
    return set_error(SF_ERR_ARG, "sf_token_logprobs: need n >= 0 and 1 <= vocab <= 2^31 - 65");
  if (dtype < SF_DT_F32 || dtype > SF_DT_F16)
    return set_error(SF_ERR_UNSUPPORTED, "sf_token_logprobs: logits must be fp32, bf16 or fp16");
  if (top < 0 || top > kMaxTop || top > vocab)
    return set_error(SF_ERR_ARG, "sf_token_logprobs: need 0 <= top <= %d, and no more than vocab", kMaxTop);
  if (n == 0) return SF_OK;
  const int size = dtype == SF_DT_F32 ? 4 : 2;
  if (!d_logits || !d_tokens || reinterpret_cast<uintptr_t>(d_logits) % size)
    return set_error(SF_ERR_ARG, "sf_token_logprobs: null logits or tokens, or logits not aligned to their type");
  if (row_stride < 0 || row_stride > (int64_t(1) << 38))
    return set_error(SF_ERR_ARG, "sf_token_logprobs: the row stride must be in 0..2^38");
  const uint64_t each = (uint64_t)n * 4, tops = each * top;
  const Range arrays[] = {{d_logits, ((uint64_t)(n - 1) * row_stride + vocab) * size, false}, {d_tokens, each, false},
                          {d_logprob, each, true}, {d_entropy, each, true}, {d_rank, each, true},
                          {d_top_ids, tops, true}, {d_top_logprobs, tops, true}};
  if (!ranges_apart(arrays, 7))
    return set_error(SF_ERR_ARG, "sf_token_logprobs: an array that the call writes overlaps another");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_token_logprobs: %s", cudaGetErrorString(e));
  ScoreArgs a{d_logits, row_stride, d_tokens, 0, 1, vocab, top, 0, d_logprob, d_entropy, d_rank, d_top_ids, d_top_logprobs};
  // Whole waves of rows, a CTA each, then the rest spread over the GPU.
  const long slots = (long)sms * (1024 / kCtaThreads), rest = n > slots ? n % slots : n;
  const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int ctas = rest ? ctas_of(rest, vocab, dtype, top > 0) : 1;
  if (rest < n && ctas > 1) {
    a.chain = 1;
    e = launch_rows(a, dtype, 0, n - rest, 1, st);
    a.chain = 2;
    if (e == cudaSuccess) e = launch_rows(a, dtype, n - rest, rest, ctas, st);
  } else {
    e = launch_rows(a, dtype, 0, n, ctas, st);
  }
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_token_logprobs: %s", cudaGetErrorString(e));
  return SF_OK;
}
