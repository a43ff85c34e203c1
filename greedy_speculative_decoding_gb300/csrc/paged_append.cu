// RoPE and cache append of a pass's token rows (sf_kv_append), the RoPE table.
//
// Bound by memory: every projected element is read once and written once. A
// thread takes eight elements of the lower half of one head and the eight
// they are paired with (16-byte accesses): few registers, so that as many
// loads as possible are in flight. 16411 bf16 rows of 36 heads of 128: 53.7 us
// (5.8 TB/s) with all threads of an SM in CTAs of 128 and everything streamed
// (56.3 with plain stores, 55.2 with plain loads; with the attention of the
// last row behind it 75.1, and 76.1 with plain stores; at 4000 rows 25.7 and
// 27.6); with plain stores 58 us in CTAs of 256, 69 of 1024, 70 with five CTAs
// of 256; two heads a thread, the rotation loaded once, was slower (78 us).
#include <cmath>
#include <type_traits>

#include "paged.h"

namespace sf {
namespace {

constexpr int kAppendThreads = 128;

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

// Eight consecutive elements as they lie in memory, and in pairs of floats.
template <typename T>
struct Raw {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(T* p) const { __stcs(reinterpret_cast<uint4*>(p), w); }
  __device__ __forceinline__ uint32_t& word(int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
  __device__ __forceinline__ float2 get(int i) {
    if constexpr (std::is_same<T, bf16>::value)
      return make_float2(__uint_as_float(word(i) << 16), __uint_as_float(word(i) & 0xffff0000u));
    else
      return __half22float2(*reinterpret_cast<const __half2*>(&word(i)));
  }
  __device__ __forceinline__ void set(int i, float x, float y) {
    if constexpr (std::is_same<T, bf16>::value) {
      word(i) = pack_bf16x2(__float2bfloat16_rn(x), __float2bfloat16_rn(y));
    } else {
      const __half2 h = __floats2half2_rn(x, y);
      word(i) = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};
template <>
struct Raw<float> {
  float4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = __ldcs(reinterpret_cast<const float4*>(p));
    w[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    __stcs(reinterpret_cast<float4*>(p), w[0]);
    __stcs(reinterpret_cast<float4*>(p) + 1, w[1]);
  }
  __device__ __forceinline__ float2 get(int i) {
    return i & 1 ? make_float2(w[i >> 1].z, w[i >> 1].w) : make_float2(w[i >> 1].x, w[i >> 1].y);
  }
  __device__ __forceinline__ void set(int i, float x, float y) {
    if (i & 1) w[i >> 1].z = x, w[i >> 1].w = y;
    else w[i >> 1].x = x, w[i >> 1].y = y;
  }
};

// TI: type of the rows; TC: of the cache; TO: of q_out.
template <typename TI, typename TC, typename TO>
__global__ void __launch_bounds__(kAppendThreads, sizeof(TI) == 2 ? 16 : 10)
    k_append(const __grid_constant__ AppendArgs a) {
  pdl_wait();   // (the next kernel is not let in early: waiting beside 16411 rows it slowed them by 1.5 us)
  const int half = a.hd >> 1;
  const unsigned per_head = half >> 3;                              // threads of a head
  const unsigned per_row = (a.nq + 2 * a.nkv) * per_head;           // threads of a row
  const unsigned u = blockIdx.x * kAppendThreads + threadIdx.x;
  const unsigned i = u / per_row;
  if (i >= (unsigned)a.n) return;
  const unsigned r = u - i * per_row;
  const int h = r / per_head, d = (r - h * per_head) * 8;
  const int kind = h < a.nq ? 0 : h < a.nq + a.nkv ? 1 : 2;         // q, k, v
  const TI* src = kind == 0   ? static_cast<const TI*>(a.q) + i * a.q_row + h * a.q_head
                  : kind == 1 ? static_cast<const TI*>(a.k) + i * a.k_row + (h - a.nq) * a.k_head
                              : static_cast<const TI*>(a.v) + i * a.v_row + (h - a.nq - a.nkv) * a.v_head;
  Raw<TI> x, y;
  x.load(src + d);
  y.load(src + d + half);
  const int slot = a.slots[i];
  const int pos = a.rope ? a.positions[i] : 0;
  if (slot < 0 || slot >= a.n_slots || (a.rope && (pos < 0 || pos >= a.n_pos))) return;
  const bool turn = a.rope && kind < 2;
  auto finish = [&](auto* dst) {
    using TO_ = typename std::remove_pointer<decltype(dst)>::type;
    Raw<TO_> ox, oy;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float2 f = x.get(p), g = y.get(p);
      if (turn) {
        const float4 c = a.rope[((size_t)pos * half + d) / 2 + p];   // cos, sin of two pairs
        const float2 f0 = f;
        f = make_float2(f.x * c.x - g.x * c.y, f.y * c.z - g.y * c.w);
        g = make_float2(g.x * c.x + f0.x * c.y, g.y * c.z + f0.y * c.w);
      }
      ox.set(p, f.x, f.y);
      oy.set(p, g.x, g.y);
    }
    ox.store(dst + d);
    oy.store(dst + d + half);
  };
  if (kind == 0) {
    finish(static_cast<TO*>(a.q_out) + i * a.o_row + h * a.o_head);
  } else {
    const long page = slot >> a.shift, off = slot & ((1 << a.shift) - 1);
    finish(kind == 1 ? static_cast<TC*>(a.kc) + page * a.kc_page + (h - a.nq) * a.kc_head + off * a.kc_slot
                     : static_cast<TC*>(a.vc) + page * a.vc_page + (h - a.nq - a.nkv) * a.vc_head + off * a.vc_slot);
  }
}

template <typename TI, typename TC>
cudaError_t launch_append(const AppendArgs& a, bool q_as_cache, int grid, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return q_as_cache ? cudaLaunchKernelEx(&cfg, k_append<TI, TC, TC>, a) : cudaLaunchKernelEx(&cfg, k_append<TI, TC, TI>, a);
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
    if (!why && vectors_overlap(n, q_out->row, q->n_heads, q_out->head, cache->head_dim)) why = "rows of q_out overlap";
  }
  if (why) return set_error(SF_ERR_ARG, "sf_kv_append: %s", why);
  // What is written must not lie on itself: pages one after the other, within
  // them no two slots on one another.
  const int64_t nkv = cache->n_kv_heads, page = cache->page, hd = cache->head_dim;
  const int64_t kv[2][3] = {{cache->k_page, cache->k_head, cache->k_slot}, {cache->v_page, cache->v_head, cache->v_slot}};
  for (const auto& s : kv)
    if (vectors_overlap(nkv, s[1], page, s[2], hd) ||
        (cache->n_pages > 1 && s[0] < (nkv > 1 ? (nkv - 1) * s[1] : 0) + (page - 1) * s[2] + hd))
      return set_error(SF_ERR_ARG, "sf_kv_append: slots of the cache overlap");
  if (cache->k == cache->v) return set_error(SF_ERR_ARG, "sf_kv_append: k and v of the cache are one");
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
  const long units = (long)n * (a.nq + 2 * a.nkv) * (a.hd / 16);
  const long grid_l = (units + kAppendThreads - 1) / kAppendThreads;
  if (grid_l > INT32_MAX / kAppendThreads) return set_error(SF_ERR_UNSUPPORTED, "sf_kv_append: too many rows for one call");
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
