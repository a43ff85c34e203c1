// Whole pages, or their first slots, copied in every layer of a cache
// (sf_page_copy). Bound by memory: a unit is the keys or the values of one page
// in one layer, taken by a CTA; a thread has four 16-byte loads in flight.
#include <algorithm>

#include "paged.h"

namespace sf {
namespace {

constexpr int kCopyThreads = 256, kCopyCtas = 8;   // threads of a CTA, CTAs of an SM

struct CopyArgs {
  uint16_t *k, *v;
  long k_layer, k_page, k_head, k_slot, v_layer, v_page, v_head, v_slot;
  const int *source, *target, *slots, *count;
  int n, layers, nkv, n_pages, page, hd_shift;   // hd_shift: log2 of a slot's 16-byte pieces
};

__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) k_page_copy(const __grid_constant__ CopyArgs a) {
  pdl_wait();
  const int n = a.count ? min(max(*a.count, 0), a.n) : a.n;
  const long per = 2l * a.layers, units = n * per;
  const int mask = (1 << a.hd_shift) - 1;
  for (long u = blockIdx.x; u < units; u += gridDim.x) {
    const long i = u / per;
    const int r = (int)(u - i * per), kv = r & 1, layer = r >> 1;
    const int s = a.source[i], t = a.target[i];
    const int slots = a.slots ? min(max(a.slots[i], 0), a.page) : a.page;
    if (s < 0 || s >= a.n_pages || t < 0 || t >= a.n_pages || slots == 0) continue;
    uint16_t* base = kv ? a.v + layer * a.v_layer : a.k + layer * a.k_layer;
    const uint16_t* from = base + s * (kv ? a.v_page : a.k_page);
    uint16_t* to = base + t * (kv ? a.v_page : a.k_page);
    const long slot = kv ? a.v_slot : a.k_slot, head = kv ? a.v_head : a.k_head;
    const unsigned each = slots << a.hd_shift, pieces = each * a.nkv;   // of 16 bytes, of a head and of all (below 2^28)
    for (unsigned e0 = threadIdx.x; e0 < pieces; e0 += 4 * kCopyThreads) {
      uint4 w[4];
      long at[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned e = e0 + x * kCopyThreads, h = e / each, p = e - h * each;
        at[x] = h * head + (p >> a.hd_shift) * slot + (p & mask) * 8;
        if (e < pieces) w[x] = __ldcs(reinterpret_cast<const uint4*>(from + at[x]));
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (e0 + x * kCopyThreads < pieces) __stcs(reinterpret_cast<uint4*>(to + at[x]), w[x]);
    }
  }
}

// Whether layers of pages lie on one another, a page `extent` elements long:
// layers one after the other, or the layers of a page side by side in it.
bool layers_apart(int64_t layers, int64_t s_layer, int64_t pages, int64_t s_page, int64_t extent) {
  if (layers == 1) return true;
  return s_layer >= (pages - 1) * s_page + extent ||
         (s_layer >= extent && (pages == 1 || (layers - 1) * s_layer + extent <= s_page));
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" sf_status sf_page_copy(const sf_paged_cache* cache, int32_t layers, int64_t k_layer, int64_t v_layer,
                                  const int32_t* d_source, const int32_t* d_target, const int32_t* d_slots, int32_t n,
                                  const int32_t* d_count, void* cuda_stream) {
  const sf_status cs = check_cache(cache, "sf_page_copy");
  if (cs != SF_OK) return cs;
  if (n < 0 || layers < 1 || (int64_t)layers * cache->n_kv_heads > 1 << 24)
    return set_error(SF_ERR_ARG, "sf_page_copy: n negative, layers below 1, or layers * n_kv_heads above 2^24");
  if (n == 0) return SF_OK;
  if (!d_source || !d_target) return set_error(SF_ERR_ARG, "sf_page_copy: null source or target");
  const int64_t st[2][4] = {{k_layer, cache->k_page, cache->k_head, cache->k_slot},
                            {v_layer, cache->v_page, cache->v_head, cache->v_slot}};
  for (const auto& s : st) {
    if (layers > 1 && (s[0] < 8 || s[0] % 8 || s[0] > (int64_t(1) << 38)))
      return set_error(SF_ERR_ARG, "sf_page_copy: layer strides must be positive multiples of 8 below 2^38");
    const int64_t extent = (cache->n_kv_heads - 1) * s[2] + (cache->page - 1) * s[3] + cache->head_dim;
    if (vectors_overlap(cache->n_kv_heads, s[2], cache->page, s[3], cache->head_dim) ||
        (cache->n_pages > 1 && s[1] < extent) || !layers_apart(layers, s[0], cache->n_pages, s[1], extent))
      return set_error(SF_ERR_ARG, "sf_page_copy: slots, pages or layers of the cache overlap");
  }
  if (cache->k == cache->v) return set_error(SF_ERR_ARG, "sf_page_copy: k and v of the cache are one");
  CopyArgs a{};
  a.k = static_cast<uint16_t*>(cache->k), a.v = static_cast<uint16_t*>(cache->v);
  a.k_layer = layers > 1 ? k_layer : 0, a.k_page = cache->k_page, a.k_head = cache->k_head, a.k_slot = cache->k_slot;
  a.v_layer = layers > 1 ? v_layer : 0, a.v_page = cache->v_page, a.v_head = cache->v_head, a.v_slot = cache->v_slot;
  a.source = d_source, a.target = d_target, a.slots = d_slots, a.count = d_count;
  a.n = n, a.layers = layers, a.nkv = cache->n_kv_heads, a.n_pages = cache->n_pages, a.page = cache->page;
  a.hd_shift = log2_of(cache->head_dim / 8);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long>((long)sms * kCopyCtas, 2l * n * layers));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_page_copy, a);
  }
  if (e != cudaSuccess) return set_error(SF_ERR_CUDA, "sf_page_copy: %s", cudaGetErrorString(e));
  return SF_OK;
}
