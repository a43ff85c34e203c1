// Attention of the requests' newest rows over a paged key-value cache
// (sf_paged_attention).
//
// One warp per (token row, query head): 32 slots at a time, a lane scores one
// slot; the softmax runs online (running maximum, sum and output), in fp32.
#include <cmath>

#include "paged.h"

namespace sf {
namespace {

struct PagedAttnArgs {
  const void *q, *kc, *vc;
  void* out;
  long q_row, q_head, o_row, o_head;
  long k_page, k_head, k_slot, v_page, v_head, v_slot;
  float* lse;
  const int *tables, *lens, *starts;
  const unsigned long long* mask;
  int B, N, W, nq, group, shift, n_pages, max_rows;
  float scale;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(bf16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(__half* p, float x) { *p = __float2half_rn(x); }

template <int HD, typename TQ, typename TC>
__global__ void __launch_bounds__(128) k_paged_attn_rows(const __grid_constant__ PagedAttnArgs a) {
  __shared__ float sq[4][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long w = blockIdx.x * 4l + warp;
  const int b = (int)(w / ((long)a.max_rows * a.nq)), rem = (int)(w - (long)b * a.max_rows * a.nq);
  const int j = rem / a.nq, h = rem - j * a.nq;
  if (b >= a.B) return;
  int s0, rows;
  if (a.starts) {
    s0 = a.starts[b];
    rows = a.starts[b + 1] - s0;
  } else {
    rows = a.N / a.B;
    s0 = b * rows;
  }
  if (j >= rows || s0 < 0 || s0 + j >= a.N) return;
  const int row = s0 + j, kvh = h / a.group;
  const int len = (int)min((long)max(a.lens[b], 0), (long)a.W << a.shift);
  const int p0 = len - rows;   // the pass's first slot
  const unsigned long long bits = a.mask ? a.mask[row] : 0;
  const TQ* q = static_cast<const TQ*>(a.q) + row * a.q_row + h * a.q_head;
  for (int d = lane; d < HD; d += 32) sq[warp][d] = to_f(q[d]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[HD / 32];
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) o[i] = 0.f;
  for (int t = 0; t < len; t += 32) {
    const int s = t + lane, i = s - p0;
    const bool see = s < len && (i < 0 || (a.mask ? i < 64 && ((bits >> i) & 1) : i <= j));
    int page = -1;
    float x = -INFINITY;
    if (see) {
      page = a.tables[(long)b * a.W + (s >> a.shift)];
      float dot = 0.f;
      if (page >= 0 && page < a.n_pages) {
        const TC* k = static_cast<const TC*>(a.kc) + page * a.k_page + kvh * a.k_head +
                      (s & ((1 << a.shift) - 1)) * a.k_slot;
        for (int d = 0; d < HD; ++d) dot = fmaf(sq[warp][d], to_f(k[d]), dot);
      } else {
        page = -1;
      }
      x = dot * a.scale;
    }
    const float m_new = fmaxf(m, warp_max(x));
    const float ref = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = expf(m - ref), p = see ? expf(x - ref) : 0.f;
    l = l * alpha + warp_sum(p);
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) o[e] *= alpha;
    for (int c = 0; c < 32; ++c) {
      const float pc = __shfl_sync(0xffffffffu, p, c);
      const int pg = __shfl_sync(0xffffffffu, page, c);
      if (pg < 0) continue;
      const TC* v = static_cast<const TC*>(a.vc) + pg * a.v_page + kvh * a.v_head +
                    ((t + c) & ((1 << a.shift) - 1)) * a.v_slot;
#pragma unroll
      for (int e = 0; e < HD / 32; ++e) o[e] = fmaf(pc, to_f(v[lane + 32 * e]), o[e]);
    }
    m = m_new;
  }
  TQ* out = static_cast<TQ*>(a.out) + row * a.o_row + h * a.o_head;
#pragma unroll
  for (int e = 0; e < HD / 32; ++e) from_f(out + lane + 32 * e, l == 0.f ? 0.f : o[e] / l);
  if (a.lse && lane == 0) a.lse[(long)row * a.nq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int HD>
cudaError_t launch_rows(const PagedAttnArgs& a, int qt, int ct, cudaStream_t st) {
  const long warps = (long)a.B * a.max_rows * a.nq;
  const int grid = (int)((warps + 3) / 4);
  if (qt == SF_DT_BF16) k_paged_attn_rows<HD, bf16, bf16><<<grid, 128, 0, st>>>(a);
  else if (qt == SF_DT_F16) k_paged_attn_rows<HD, __half, __half><<<grid, 128, 0, st>>>(a);
  else k_paged_attn_rows<HD, float, bf16><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" size_t sf_paged_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                     int32_t max_rows) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads > 65535 || (head_dim != 64 && head_dim != 128) ||
      max_rows < 1 || max_rows > SF_MAX_ROWS)
    return 0;
  return 256;
}

extern "C" sf_status sf_paged_attention(const sf_paged_cache* cache, const sf_rows* q, const sf_rows* out, int32_t n,
                                        const int32_t* d_tables, int32_t table_width, const int32_t* d_lens,
                                        const int32_t* d_starts, int32_t batch, int32_t max_rows,
                                        const uint64_t* d_mask, float scale, float* d_lse, void* d_workspace,
                                        void* cuda_stream) {
  const sf_status cs = check_cache(cache, "sf_paged_attention");
  if (cs != SF_OK) return cs;
  if (!q || !out || n < 0 || batch < 0) return set_error(SF_ERR_ARG, "sf_paged_attention: no q or out, or n or batch negative");
  if (n == 0 || batch == 0) return SF_OK;
  if (!d_tables || !d_lens || !d_workspace) return set_error(SF_ERR_ARG, "sf_paged_attention: null tables, lens or workspace");
  if (reinterpret_cast<uintptr_t>(d_workspace) & 255)
    return set_error(SF_ERR_ARG, "sf_paged_attention: the workspace must be 256-byte aligned");
  if (q->dtype != out->dtype || (q->dtype != cache->dtype && !(q->dtype == SF_DT_F32 && cache->dtype == SF_DT_BF16)))
    return set_error(SF_ERR_UNSUPPORTED, "sf_paged_attention: q and out must have the cache's type, or be fp32 over a bf16 cache");
  if (q->n_heads < 1 || q->n_heads > 65535 || q->n_heads % cache->n_kv_heads || out->n_heads != q->n_heads)
    return set_error(SF_ERR_ARG, "sf_paged_attention: heads must be a multiple of the cache's, the same in q and out");
  if (max_rows < 1 || max_rows > (d_mask ? 64 : SF_MAX_ROWS))
    return set_error(SF_ERR_ARG, "sf_paged_attention: need 1 <= max_rows <= %d (64 with a mask)", SF_MAX_ROWS);
  if (!d_starts && (n % batch || n / batch > max_rows))
    return set_error(SF_ERR_ARG, "sf_paged_attention: without starts, n must be batch times at most max_rows rows");
  if (table_width < 1 || table_width > (1 << 30) / cache->page)
    return set_error(SF_ERR_ARG, "sf_paged_attention: need 1 <= table_width <= 2^30 / page");
  const int al = q->dtype == SF_DT_F32 ? 4 : 8;
  for (const sf_rows* r : {q, out})
    if (!r->data || (reinterpret_cast<uintptr_t>(r->data) & 15) || (n > 1 && r->row % al) ||
        (r->n_heads > 1 && r->head % al))
      return set_error(SF_ERR_ARG, "sf_paged_attention: q and out must be 16-byte aligned with strides of multiples of 16 bytes");
  if (!std::isfinite(scale)) return set_error(SF_ERR_ARG, "sf_paged_attention: scale must be finite");
  PagedAttnArgs a{};
  a.q = q->data, a.q_row = q->row, a.q_head = q->head;
  a.out = out->data, a.o_row = out->row, a.o_head = out->head;
  a.kc = cache->k, a.k_page = cache->k_page, a.k_head = cache->k_head, a.k_slot = cache->k_slot;
  a.vc = cache->v, a.v_page = cache->v_page, a.v_head = cache->v_head, a.v_slot = cache->v_slot;
  a.lse = d_lse;
  a.tables = d_tables, a.lens = d_lens, a.starts = d_starts;
  a.mask = reinterpret_cast<const unsigned long long*>(d_mask);
  a.B = batch, a.N = n, a.W = table_width, a.nq = q->n_heads, a.group = q->n_heads / cache->n_kv_heads;
  a.shift = log2_of(cache->page), a.n_pages = cache->n_pages, a.max_rows = max_rows;
  a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = cache->head_dim == 128 ? launch_rows<128>(a, q->dtype, cache->dtype, st)
                                               : launch_rows<64>(a, q->dtype, cache->dtype, st);
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_paged_attention: %s", cudaGetErrorString(e));
  return SF_OK;
}
