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
// Bound by memory: a row is read once.
#include "paged.h"

namespace sf {
namespace {

constexpr int kThreads = 512;
constexpr int kGroups = kThreads / 4;   // groups of four threads, for the top alternatives
constexpr int kMaxTop = 32;
constexpr int kBuffer = 2048;           // elements that reach the bound; more (rows made for it) are handled apart
constexpr float kLog2E = 1.44269504088896f;

struct ScoreArgs {
  const void* x;
  long row;
  const int* tokens;
  int n, vocab, top;
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

// Sixteen bytes of a row as floats.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 w;
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u = (i * (int)sizeof(T)) / 4 == 0 ? w.x : (i * (int)sizeof(T)) / 4 == 1 ? w.y
                     : (i * (int)sizeof(T)) / 4 == 2 ? w.z : w.w;
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    else if constexpr (std::is_same<T, bf16>::value) return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
    else return i & 1 ? __high2float(*reinterpret_cast<const __half2*>(&u)) : __low2float(*reinterpret_cast<const __half2*>(&u));
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
  __device__ __forceinline__ void add(float x) {   // m is at least x, and finite
    const float d = x - m, e = exp2_fast(d * kLog2E);
    s += e;
    t = fmaf(e, fmaxf(d, -1.0e30f), t);            // (e = 0 times -infinity is NaN)
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

template <typename T>
__global__ void __launch_bounds__(kThreads) k_token_logprobs(const __grid_constant__ ScoreArgs a) {
  using V = Vec<T>;
  __shared__ Sums s_sums[kThreads / 32];
  __shared__ int s_rank[kThreads / 32];
  __shared__ float s_max[kGroups];
  __shared__ int s_first[kGroups];       // (ties at the bound: first token of the group that is equal to it)
  __shared__ int s_groups[kMaxTop];      // the groups whose elements are looked at again
  __shared__ unsigned long long s_bound, s_top[kMaxTop], s_buffer[kBuffer], s_best[kThreads / 32];
  __shared__ int s_count, s_picked, s_ties;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = tid >> 2;
  pdl_wait();
  const long row = blockIdx.x;
  const int token = a.tokens[row];
  if (token < 0 || token >= a.vocab) return;
  const T* x = static_cast<const T*>(a.x) + row * a.row;
  // The row as a few elements up to a 16-byte boundary, vectors, a few elements.
  const int head = min(a.vocab, (int)((-reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T)));
  const int nv = (a.vocab - head) / V::N, body = head + nv * V::N;
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);

  // The element or so of the head and the tail that this thread has: a token, or -1.
  const int odd = tid < head ? tid : tid >= 16 && tid - 16 < a.vocab - body ? body + tid - 16 : -1;
  const float odd_x = odd >= 0 ? to_float(x[odd]) : -INFINITY;

  // In front of the given token: larger logits, equal ones of lower tokens. For
  // those, equal means above the next lower number. With a given -infinity (or
  // NaN) every lower token is in front.
  float given = to_float(x[token]);
  if (!(given == given)) given = -INFINITY;
  const bool all_before = given == -INFINITY;
  const float above = given;
  const float before = all_before ? INFINITY : given == 0.f ? -1.0e-45f
                     : __uint_as_float(__float_as_uint(given) + (given > 0.f ? -1 : 1));
  int rank = tid == 0 && all_before ? token : 0;

  Sums z = {-INFINITY, 0.f, 0.f};
  auto odd_nan = [&](float v) { if (v != v) z.s = v; };
  if (odd >= 0) {
    z.raise(odd_x);
    if (z.m == -INFINITY) odd_nan(odd_x);
    else z.add(odd_x);
    rank += odd_x > (odd < token ? before : above);
  }
#pragma unroll 1
  for (int i = tid; i < nv; i += kThreads) {
    const V v = {__ldg(xv + i)};
    float mx = v.get(0);
#pragma unroll
    for (int e = 1; e < V::N; ++e) mx = fmaxf(mx, v.get(e));
    z.raise(mx);
    if (z.m == -INFINITY) {
#pragma unroll
      for (int e = 0; e < V::N; ++e) odd_nan(v.get(e));
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) z.add(v.get(e));
    }
    const int v0 = head + i * V::N;
#pragma unroll
    for (int e = 0; e < V::N; ++e) rank += v.get(e) > (v0 + e < token ? before : above);
  }

  // ---- join the threads' sums
  Sums all = z;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all.join(all.shuffled(o));
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
  }
  if (lane == 0) {
    s_sums[warp] = all;
    s_rank[warp] = rank;
  }
  float gm = z.m;
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 1));
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
  if ((tid & 3) == 0) s_max[group] = gm;
  if (tid == 0) s_count = s_picked = s_ties = 0;
  __syncthreads();
  all = s_sums[0];
  rank = s_rank[0];
  for (int w = 1; w < kThreads / 32; ++w) {
    all.join(s_sums[w]);
    rank += s_rank[w];
  }
  // log p = (x - m) - log s; a row of -infinity alone has none above -infinity.
  const float logs = logf(all.s);
  auto logp = [&](float v) { return all.m == -INFINITY && all.s == 0.f ? -INFINITY : (v - all.m) - logs; };
  if (tid == 0) {
    if (a.logprob) a.logprob[row] = logp(to_float(x[token]));
    if (a.entropy) a.entropy[row] = all.m == -INFINITY && all.s == 0.f ? 0.f : logs - all.t / all.s;
    if (a.rank) a.rank[row] = rank;
  }
  if (a.top == 0) return;

  // ---- the groups with the k largest maxima
  const int k = a.top;
  int larger = 0, equal = 0;
  if (tid < kGroups) {
    const float mine = s_max[tid];
    for (int g = 0; g < kGroups; ++g) {
      larger += s_max[g] > mine;
      equal += s_max[g] == mine;
    }
    if (larger < k && larger + equal >= k) {   // the k-th largest
      s_bound = (unsigned long long)float_key(mine + 0.f) << 32;
      s_ties = larger + equal > k ? equal : 0;
    }
  }
  __syncthreads();
  const float at = key_value(s_bound);
  // The elements of n groups, by the threads of the CTA together.
  const int per = 4 + (nv + kThreads - 1) / kThreads * 4;   // a group's odd elements and vectors, places for them at least
  auto each = [&](const int* groups, int n, auto f) {
    for (int i = tid; i < n * per; i += kThreads) {
      const int p = i / per, r = i - p * per, g = groups ? groups[p] : p;
      if (r < 4) {
        const int t = 4 * g + r;
        const int v = t < head ? t : t >= 16 && t - 16 < a.vocab - body ? body + t - 16 : -1;
        if (v >= 0) f(to_float(x[v]), v, g);
      } else {
        const int j = (r - 4) / 4 * kThreads + 4 * g + (r & 3);
        if (j < nv) {
          const V v = {__ldg(xv + j)};
#pragma unroll
          for (int e = 0; e < V::N; ++e) f(v.get(e), head + j * V::N + e, g);
        }
      }
    }
  };
  if (s_ties) {   // more maxima equal to the bound than there is room for: the lowest tokens first
    if (tid < kGroups) s_first[tid] = INT32_MAX;
    __syncthreads();
    each(nullptr, kGroups, [&](float v, int t, int g) {
      if (s_max[g] == at && (v == v ? v : -INFINITY) == at) atomicMin(&s_first[g], t);
    });
    __syncthreads();
    if (tid < kGroups && s_max[tid] == at) {
      int before_me = larger;
      for (int g = 0; g < kGroups; ++g) before_me += s_max[g] == at && s_first[g] < s_first[tid];
      if (before_me < k && s_first[tid] != INT32_MAX) s_groups[atomicAdd(&s_picked, 1)] = tid;   // (not one without elements)
      if (before_me == k - 1 && s_first[tid] != INT32_MAX) s_bound = order_key(at, s_first[tid]);
    } else if (tid < kGroups && larger < k) {
      s_groups[atomicAdd(&s_picked, 1)] = tid;
    }
  } else if (tid < kGroups && s_max[tid] >= at) {
    s_groups[atomicAdd(&s_picked, 1)] = tid;
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
  if (tid < k) s_top[tid] = 0;
  __syncthreads();
  const int count = s_count;
  if (count <= kBuffer) {
    for (int c = tid; c < count; c += kThreads) {
      const unsigned long long mine = s_buffer[c];
      int r = 0;
      for (int i = 0; i < count; ++i) r += s_buffer[i] > mine;
      if (r < k) s_top[r] = mine;
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
      if (tid == 0) s_top[r] = best;
      last = best;
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid < k) {
    const unsigned long long key = s_top[tid];
    if (a.top_ids) a.top_ids[row * k + tid] = key_index(key);
    if (a.top_logprobs) a.top_logprobs[row * k + tid] = logp(key_value(key));
  }
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
  ScoreArgs a{d_logits, row_stride, d_tokens, n, vocab, top, d_logprob, d_entropy, d_rank, d_top_ids, d_top_logprobs};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(cuda_stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = dtype == SF_DT_F32    ? cudaLaunchKernelEx(&cfg, k_token_logprobs<float>, a)
                        : dtype == SF_DT_BF16 ? cudaLaunchKernelEx(&cfg, k_token_logprobs<bf16>, a)
                                              : cudaLaunchKernelEx(&cfg, k_token_logprobs<__half>, a);
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_token_logprobs: %s", cudaGetErrorString(e));
  return SF_OK;
}
