// RoPE and cache append of a pass's token rows (sf_kv_append), the RoPE table.
//
// Bound by memory: every projected element is read once and written once. A
// thread takes the same eight elements of the lower half, and the eight they
// are paired with, of kHeads heads of a row: their rotation is loaded once,
// and all the heads' loads are in flight together (16-byte accesses).
#include <cmath>

#include "paged.h"

namespace sf {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kHeads = 2;   // heads of a thread

struct AppendArgs {
  const void *q, *k, *v;
  long q_row, q_head, k_row, k_head, v_row, v_head;
  void* q_out;
  long o_row, o_head;
  void *kc, *vc;
  long kc_page, kc_head, kc_slot, vc_page, vc_head, vc_slot;
  const int* slots;
  const int* positions;
  const float4* rope;   // (cos, sin) pairs, two to a float4; null: no rotation
  int n, nq, nkv, hd, shift, n_slots, n_pos;
};

__device__ __forceinline__ void load8(float (&x)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(float (&x)[8], const bf16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(float (&x)[8], const __half* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(__float2bfloat16_rn(x[2 * i]), __float2bfloat16_rn(x[2 * i + 1]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// TI: type of the rows; TC: of the cache; TO: of q_out.
template <typename TI, typename TC, typename TO>
__global__ void __launch_bounds__(kAppendThreads) k_append(const __grid_constant__ AppendArgs a) {
  const int half = a.hd >> 1;
  const int per_head = half >> 3;                           // pieces of a head
  const int heads = a.nq + 2 * a.nkv;
  const int groups = (heads + kHeads - 1) / kHeads;
  const int per_row = groups * per_head;                    // threads of a row
  const long u = blockIdx.x * (long)kAppendThreads + threadIdx.x;
  const int i = (int)(u / per_row), r = (int)(u - (long)i * per_row);
  if (i >= a.n) return;
  const int h0 = r / per_head * kHeads, d = (r - r / per_head * per_head) * 8;
  const int slot = a.slots[i];
  const int pos = a.rope ? a.positions[i] : 0;
  float x[kHeads][8], y[kHeads][8];
#pragma unroll
  for (int e = 0; e < kHeads; ++e) {
    const int h = h0 + e;
    if (h >= heads) break;
    const TI* src = h < a.nq ? static_cast<const TI*>(a.q) + i * a.q_row + h * a.q_head
                    : h < a.nq + a.nkv ? static_cast<const TI*>(a.k) + i * a.k_row + (h - a.nq) * a.k_head
                                       : static_cast<const TI*>(a.v) + i * a.v_row + (h - a.nq - a.nkv) * a.v_head;
    load8(x[e], src + d);
    load8(y[e], src + d + half);
  }
  if (slot < 0 || slot >= a.n_slots || (a.rope && (pos < 0 || pos >= a.n_pos))) return;
  float4 cs[4];
  if (a.rope) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = a.rope[((size_t)pos * half + d) / 2 + e];
  }
  const long page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
#pragma unroll
  for (int e = 0; e < kHeads; ++e) {
    const int h = h0 + e;
    if (h >= heads) break;
    if (a.rope && h < a.nq + a.nkv) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float x0 = x[e][2 * p], y0 = y[e][2 * p], x1 = x[e][2 * p + 1], y1 = y[e][2 * p + 1];
        x[e][2 * p] = x0 * cs[p].x - y0 * cs[p].y;
        y[e][2 * p] = y0 * cs[p].x + x0 * cs[p].y;
        x[e][2 * p + 1] = x1 * cs[p].z - y1 * cs[p].w;
        y[e][2 * p + 1] = y1 * cs[p].z + x1 * cs[p].w;
      }
    }
    if (h < a.nq) {
      TO* dst = static_cast<TO*>(a.q_out) + i * a.o_row + h * a.o_head + d;
      store8(dst, x[e]);
      store8(dst + half, y[e]);
    } else {
      const bool k = h < a.nq + a.nkv;
      TC* dst = k ? static_cast<TC*>(a.kc) + page * a.kc_page + (h - a.nq) * a.kc_head + off * a.kc_slot
                  : static_cast<TC*>(a.vc) + page * a.vc_page + (h - a.nq - a.nkv) * a.vc_head + off * a.vc_slot;
      store8(dst + d, x[e]);
      store8(dst + d + half, y[e]);
    }
  }
}

template <typename TI, typename TC>
cudaError_t launch_append(const AppendArgs& a, bool q_as_cache, int grid, cudaStream_t st) {
  if (q_as_cache) k_append<TI, TC, TC><<<grid, kAppendThreads, 0, st>>>(a);
  else k_append<TI, TC, TI><<<grid, kAppendThreads, 0, st>>>(a);
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Why a row tensor is refused, or null.
const char* rows_bad(const sf_rows* r, int n_heads, int n) {
  if (!r->data || !aligned16(r->data)) return "data null or not 16-byte aligned";
  if (r->n_heads != n_heads) return "number of heads";
  const int al = r->dtype == SF_DT_F32 ? 4 : 8;
  if ((n > 1 && r->row % al) || (n_heads > 1 && r->head % al)) return "strides must be multiples of 16 bytes";
  return nullptr;
}

}  // namespace

sf_status check_cache(const sf_paged_cache* c, const char* who) {
  if (!c) return set_error(SF_ERR_ARG, "%s: null cache", who);
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
    return set_error(SF_ERR_ARG, "%s: cache pointers null or not 16-byte aligned", who);
  if (c->dtype != SF_DT_BF16 && c->dtype != SF_DT_F16)
    return set_error(SF_ERR_UNSUPPORTED, "%s: the cache is bf16 or fp16", who);
  if (c->head_dim != 64 && c->head_dim != 128)
    return set_error(SF_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", who);
  if (!page_ok(c->page)) return set_error(SF_ERR_ARG, "%s: page must be 16, 32, 64, 128 or 256", who);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 65535 || c->n_pages < 1 || c->n_pages > INT32_MAX / c->page)
    return set_error(SF_ERR_ARG, "%s: need n_kv_heads >= 1, n_pages >= 1, n_pages * page < 2^31", who);
  const int64_t st[2][3] = {{c->k_page, c->k_head, c->k_slot}, {c->v_page, c->v_head, c->v_slot}};
  for (const auto& s : st) {
    for (int64_t x : s)
      if (x < 8 || x % 8 || x > (int64_t(1) << 38))
        return set_error(SF_ERR_ARG, "%s: cache strides must be positive multiples of 8 below 2^38", who);
    if ((c->n_kv_heads > 1 && s[0] < s[1]) || s[0] < s[2])
      return set_error(SF_ERR_ARG, "%s: the page stride must be the cache's largest", who);
  }
  return SF_OK;
}

}  // namespace sf

using namespace sf;

extern "C" sf_status sf_rope_table(float* d_table, int32_t n_pos, int32_t head_dim, float theta, void* cuda_stream) {
  if (!d_table || !aligned16(d_table)) return set_error(SF_ERR_ARG, "sf_rope_table: table null or not 16-byte aligned");
  if (head_dim < 2 || head_dim % 2 || head_dim > 1024 || n_pos < 1 || n_pos > (1 << 30) / (head_dim / 2))
    return set_error(SF_ERR_ARG, "sf_rope_table: need head_dim even, 2..1024, and 1 <= n_pos, n_pos * head_dim / 2 <= 2^30");
  if (!(theta > 0.f) || !std::isfinite(theta)) return set_error(SF_ERR_ARG, "sf_rope_table: theta must be positive and finite");
  const cudaError_t e = launch_rope_table(reinterpret_cast<float2*>(d_table), n_pos, head_dim, theta,
                                          static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_rope_table: %s", cudaGetErrorString(e));
  return SF_OK;
}

extern "C" sf_status sf_kv_append(const sf_paged_cache* cache, int32_t n, const sf_rows* k, const sf_rows* v,
                                  const int32_t* d_slots, const sf_rows* q, const sf_rows* q_out,
                                  const int32_t* d_positions, const float* d_rope, int32_t n_pos, void* cuda_stream) {
  const sf_status cs = check_cache(cache, "sf_kv_append");
  if (cs != SF_OK) return cs;
  if (n < 0 || !k || !v || (q == nullptr) != (q_out == nullptr))
    return set_error(SF_ERR_ARG, "sf_kv_append: n negative, no k or v, or only one of q and q_out");
  if (n == 0) return SF_OK;
  if (!d_slots || (d_rope && (!d_positions || n_pos < 1 || !aligned16(d_rope))))
    return set_error(SF_ERR_ARG, "sf_kv_append: no slots, or a RoPE table without positions, empty or not 16-byte aligned");
  if (k->dtype < SF_DT_F32 || k->dtype > SF_DT_F16 || v->dtype != k->dtype || (q && q->dtype != k->dtype))
    return set_error(SF_ERR_UNSUPPORTED, "sf_kv_append: q, k and v must have one type, fp32, bf16 or fp16");
  if (k->dtype != SF_DT_F32 && k->dtype != cache->dtype)
    return set_error(SF_ERR_UNSUPPORTED, "sf_kv_append: 16-bit rows must have the cache's type");
  const char* why = rows_bad(k, cache->n_kv_heads, n);
  if (!why) why = rows_bad(v, cache->n_kv_heads, n);
  if (!why && q) {
    if (q->n_heads < 1 || q->n_heads > 65535) why = "number of heads";
    else if (q_out->dtype != q->dtype && q_out->dtype != cache->dtype) why = "q_out must have q's or the cache's type";
    else why = rows_bad(q, q->n_heads, n);
    if (!why) why = rows_bad(q_out, q->n_heads, n);
  }
  if (why) return set_error(SF_ERR_ARG, "sf_kv_append: %s", why);
  AppendArgs a{};
  a.k = k->data, a.k_row = k->row, a.k_head = k->head;
  a.v = v->data, a.v_row = v->row, a.v_head = v->head;
  bool q_as_cache = true;
  if (q) {
    a.q = q->data, a.q_row = q->row, a.q_head = q->head;
    a.q_out = q_out->data, a.o_row = q_out->row, a.o_head = q_out->head;
    a.nq = q->n_heads;
    q_as_cache = q_out->dtype == cache->dtype;
  }
  a.kc = cache->k, a.kc_page = cache->k_page, a.kc_head = cache->k_head, a.kc_slot = cache->k_slot;
  a.vc = cache->v, a.vc_page = cache->v_page, a.vc_head = cache->v_head, a.vc_slot = cache->v_slot;
  a.slots = d_slots;
  a.positions = d_positions;
  a.rope = reinterpret_cast<const float4*>(d_rope);
  a.n = n;
  a.nkv = cache->n_kv_heads;
  a.hd = cache->head_dim;
  a.shift = log2_of(cache->page);
  a.n_slots = cache->n_pages * cache->page;
  a.n_pos = n_pos;
  const long units = (long)n * ((a.nq + 2 * a.nkv + kHeads - 1) / kHeads) * (a.hd / 16);
  const long grid_l = (units + kAppendThreads - 1) / kAppendThreads;
  if (grid_l > INT32_MAX) return set_error(SF_ERR_UNSUPPORTED, "sf_kv_append: too many rows for one call");
  const int grid = (int)grid_l;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e;
  if (k->dtype == SF_DT_BF16) e = launch_append<bf16, bf16>(a, true, grid, st);
  else if (k->dtype == SF_DT_F16) e = launch_append<__half, __half>(a, true, grid, st);
  else if (cache->dtype == SF_DT_BF16) e = launch_append<float, bf16>(a, q_as_cache, grid, st);
  else e = launch_append<float, __half>(a, q_as_cache, grid, st);
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_kv_append: %s", cudaGetErrorString(e));
  return SF_OK;
}
