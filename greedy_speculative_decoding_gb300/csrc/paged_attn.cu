// Attention over a paged key-value cache: the C entry (the kernels are in
// paged_attn.cuh).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "paged_attn_launch.cuh"

namespace sf {
namespace pa {

constexpr int kMaxCtas = 320;   // CTAs of a launch, at most (two on each of 152 SMs)
constexpr int kMaxDesc = 1024;  // item descriptors

struct Layout {
  size_t ml, part, total;
};
static Layout layout(int n_heads, int n_kv_heads, int head_dim, int max_rows) {   // (whatever the tile)
  const int queries = max_rows * (n_heads / n_kv_heads);
  const size_t mt = std::min(queries, 128);
  Layout l;
  l.ml = kMaxDesc * sizeof(int4);
  l.part = l.ml + 2 * kMaxCtas * mt * sizeof(float2);
  l.total = l.part + 2 * kMaxCtas * mt * head_dim * sizeof(float);
  return l;
}

// Tensor map of the keys or values, {head_dim, slots, heads, pages}: the
// two middle dimensions by ascending stride (*nhd: the heads come first).
static cudaError_t cache_map(CUtensorMap* map, int* nhd, const sf_paged_cache& c, const void* base, int64_t s_page,
                             int64_t s_head, int64_t s_slot) {
  typedef CUresult (*encode_fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<encode_fn> known{nullptr};
  encode_fn encode = known.load(std::memory_order_relaxed);
  if (!encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorSymbolNotFound;
    encode = reinterpret_cast<encode_fn>(fn);
    known.store(encode, std::memory_order_relaxed);
  }
  // Dimensions of one element never move: their strides only have to be legal.
  if (c.n_kv_heads == 1) s_head = std::max<int64_t>(s_slot, c.head_dim) * c.page;
  if (c.n_pages == 1) s_page = std::max(s_head * c.n_kv_heads, s_slot * c.page);
  *nhd = c.n_kv_heads > 1 && s_head < s_slot;
  const cuuint32_t bp = std::min(c.page, kTile);
  cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page, (cuuint64_t)c.n_kv_heads, (cuuint64_t)c.n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)s_slot * 2, (cuuint64_t)s_head * 2, (cuuint64_t)s_page * 2};
  cuuint32_t box[4] = {64, bp, 1, 1};
  if (*nhd) {
    std::swap(dims[1], dims[2]);
    std::swap(strides[0], strides[1]);
    std::swap(box[1], box[2]);
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, c.dtype == SF_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Units of an item at most (its request fills its table), the query tile, and
// the items of the whole call.
struct Sizes {
  long units, items;
  int mt, ntq;
};
static Sizes sizes(const sf_paged_cache& c, int n_heads, int max_rows, int q_dtype, int batch, int table_width, int sms) {
  Sizes z;
  const int queries = max_rows * (n_heads / c.n_kv_heads);
  z.units = std::max(1l, ((long)table_width * c.page + kTile - 1) / kTile);
  auto items = [&](int mt) { return (long)batch * c.n_kv_heads * ((queries + mt - 1) / mt); };
  auto total = [&](int mt) { return items(mt) * z.units; };   // if every request filled its table
  // Larger tiles read the cache less often (again from L2), smaller ones spread
  // few units over more of the GPU and start sooner. Measured, in us, for
  // requests x tokens x KV heads and queries in tables that the requests fill,
  // in tiles of 16 / 32 / 128:
  //   16-bit, head dimension 128: 1 x 4000 x 4, 45: 10.3 / 10.1 / 11.7; 8 x
  //     1000 x 8, 45: 20.9 / 21.7 / 17.2; 20: 16.8 / 14.7 / 15.9
  //   16-bit, 64: 16 x 5..4099 x 2, 91: 21.5 / 17.0 / 17.7; 8 x 4096..8192 x 8,
  //     45: 41.8 / 36.0 / 28.4; 20: 30.9 / 23.6 / 26.9
  //   fp32, 128 (not in tiles of 32): 1 x 8000 x 4, 45: 17.1 / 18.0; 8 x 1000 x
  //     8, 45: 28.4 / 26.3; 20: 21.9 / 23.6; 8 x 4096..8192 x 8, 20: 66.5 / 58.3
  //   fp32, 64: 8 x 1000 x 8, 45: 18.2 / 19.5 / 20.4; 91: 28.3 / 26.4 / 22.3;
  //     20: 14.3 / 14.1 / 19.8; 8 x 4096..8192 x 8, 20: 42.3 / 36.3 / 50.5
  // Wider tables move the choice towards the larger tiles, whatever the lengths
  // (which the host does not know): 1 x 2057 x 4, 63 fp32 queries 10.9 in a table
  // of 2112 tokens, 15.6 in one of 32768; bf16 9.3 and 11.2; 16 x 5..4099 x 2, 91
  // fp16 queries 16.5 and 19.1.
  if (queries <= 16) z.mt = 16;
  else if (q_dtype != SF_DT_F32) z.mt = queries > 32 && total(128) >= (c.head_dim == 64 ? 4096 : 2 * sms) ? 128 : 32;
  else if (queries > 32) z.mt = total(16) >= 4000 ? 128 : 16;
  else z.mt = total(16) < 8192 ? 16 : c.head_dim == 64 ? 32 : 128;
  z.ntq = (queries + z.mt - 1) / z.mt;
  z.items = items(z.mt);
  return z;
}
// The kernel counts a request's units in 32 bits.
static bool units_fit(const sf_paged_cache& c, int n_heads, int max_rows, int q_dtype, int batch, int table_width,
                      int sms) {
  const Sizes z = sizes(c, n_heads, max_rows, q_dtype, batch, table_width, sms);
  return c.n_kv_heads * (long)z.ntq * (z.units + kMaxPiece) <= INT32_MAX;
}

// Enqueue a checked call: `a` holds rows, tables and lengths.
static cudaError_t enqueue(Args& a, const sf_paged_cache& c, int q_dtype, float scale, void* workspace, int sms,
                           cudaStream_t st) {
  cudaError_t e = cache_map(&a.km, &a.k_nhd, c, c.k, c.k_page, c.k_head, c.k_slot);
  if (e == cudaSuccess) e = cache_map(&a.vm, &a.v_nhd, c, c.v, c.v_page, c.v_head, c.v_slot);
  if (e != cudaSuccess) return e;
  a.nkv = c.n_kv_heads;
  a.group = a.nq / a.nkv;
  a.shift = log2_of(c.page);
  // (never 0: the mask's -infinity times 0 would be NaN)
  a.scale2 = std::max(std::fabs(scale) * 1.44269504088896f, FLT_TRUE_MIN);
  a.flip = scale >= 0.f ? 0u : q_dtype == SF_DT_F32 ? 0x80000000u : 0x80008000u;
  const Sizes z = sizes(c, a.nq, a.max_rows, q_dtype, a.B, a.W, sms);
  a.mt = z.mt;
  a.mt_max = std::min(a.max_rows * a.group, a.mt);
  a.ntq_max = z.ntq;
  a.by_item = z.items <= kMaxDesc;
  const Layout lay = layout(a.nq, a.nkv, c.head_dim, a.max_rows);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.desc = reinterpret_cast<int4*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + lay.ml);
  a.part = reinterpret_cast<float*>(ws + lay.part);
  const long max_units = z.items * z.units;
  a.by_warp = a.B <= 32 && max_units + kMaxPiece * z.items <= INT32_MAX;
  sms = std::min(sms, kMaxCtas / 2);
  return c.head_dim == 128 ? launch_hd128(a, q_dtype, sms, max_units, st) : launch_hd64(a, q_dtype, sms, max_units, st);
}

__global__ void k_tree_mask(unsigned long long* mask, int n, int rows, int g) {
  pdl_wait();
  pdl_launch_next();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int j = i % rows;
  unsigned long long m = 1;   // row 0; of candidate (j - 1) / g, the rows up to this one
  for (int r = j - (j > 0 ? (j - 1) % g : 0); r <= j; ++r) m |= 1ull << r;
  mask[i] = m;
}

}  // namespace pa

cudaError_t launch_engine_paged_attention(const EngineAttn& e, int num_sms, cudaStream_t st) {
  pa::Args a{};
  a.q = e.q;
  a.q_row = (long)e.nq * e.cache.head_dim;
  a.q_head = e.cache.head_dim;
  a.frag = e.out;
  a.frag_umma = e.umma;
  a.err = e.err;
  a.tables = e.tables;
  a.W = e.table_width;
  a.lens = e.lens;
  a.len_add = e.len_add;
  a.mask = e.mask;
  a.B = e.B;
  a.N = e.B * e.rows;
  a.nq = e.nq;
  a.max_rows = a.rows_each = e.rows;
  return pa::enqueue(a, e.cache, SF_DT_F32, e.scale, e.workspace, num_sms, st);
}

cudaError_t launch_tree_mask(unsigned long long* mask, int B, int rows, int g, cudaStream_t st, bool pdl) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((B * rows + 127) / 128);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, pa::k_tree_mask, mask, B * rows, rows, g);
}

}  // namespace sf

using namespace sf;

extern "C" size_t sf_paged_attention_workspace_bytes(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim,
                                                     int32_t max_rows) {
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads > 65535 || (head_dim != 64 && head_dim != 128) ||
      max_rows < 1 || max_rows > SF_MAX_ROWS)
    return 0;
  return pa::layout(n_heads, n_kv_heads, head_dim, max_rows).total;
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
  if (vectors_overlap(n, out->row, out->n_heads, out->head, cache->head_dim))
    return set_error(SF_ERR_ARG, "sf_paged_attention: rows of out overlap");
  if (!std::isfinite(scale)) return set_error(SF_ERR_ARG, "sf_paged_attention: scale must be finite");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  pa::Args a{};
  a.q = q->data, a.q_row = q->row, a.q_head = q->head;
  a.out = out->data, a.o_row = out->row, a.o_head = out->head;
  a.lse = d_lse;
  a.tables = d_tables, a.lens = d_lens, a.starts = d_starts;
  a.mask = reinterpret_cast<const unsigned long long*>(d_mask);
  a.B = batch, a.N = n, a.W = table_width, a.nq = q->n_heads, a.max_rows = max_rows, a.rows_each = n / batch;
  if (!pa::units_fit(*cache, q->n_heads, max_rows, q->dtype, batch, table_width, sms))
    return set_error(SF_ERR_UNSUPPORTED, "sf_paged_attention: table_width * page too large for this many heads and rows");
  if (e == cudaSuccess) e = pa::enqueue(a, *cache, q->dtype, scale, d_workspace, sms, static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_paged_attention: %s", cudaGetErrorString(e));
  return SF_OK;
}
