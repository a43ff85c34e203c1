// Attention of the requests' newest rows over a paged key-value cache.
//
// For a token row and query head, out = sum_s p_s v_s / sum_s p_s with
// p_s = 2^(x_s - max x), x_s = (q . k_s) * scale * log2(e), over the slots s
// that the row sees. The cache is read once: the maximum, the sum and the
// output run along with the slots (in fp32; a new maximum rescales them). For
// fp16 the p_s are a power of two larger (Num::kUp), and so are both sums.
//
// Work. An item is (request, KV head, tile of MT queries): the queries are
// the request's rows times the query heads that read this KV head. An item
// has one unit per 64 slots of the request, and before them a few that stand
// for the beginning of an item (queries to load, a result to leave). The units
// of all items, in order, are dealt out evenly to the CTAs, so lengths that
// differ by orders of magnitude load the GPU evenly and a single long request
// is spread over all of it. A CTA that holds an item from end to end writes the result; of
// an item that several CTAs share each leaves its part (output, maximum, sum)
// in the workspace, and the join kernel adds the parts in slot order.
//
// A CTA: one producer warp follows the block table and brings 64 slots of
// keys and values at a time into a ring in shared memory (TMA boxes of 64
// dimensions by min(page, 64) slots, 128-byte swizzle); WM x WK consumer
// warps compute on them with mma.sync: warp (wm, wk) takes 16 queries and
// 64 / WK of the slots, with a running maximum, sum and output of its own,
// joined over wk at the end of the item: 1 x 4 warps for tiles of 16 queries
// (one new token: the query heads of one KV head), 2 x 2 for tiles of 32.
// Tiles of 128 queries are paged_attn_tc.cuh's.
#pragma once

#include <type_traits>

#include "paged.h"
#include "umma.cuh"

namespace sf {
namespace pa {

constexpr int kTile = 64;                 // slots of a unit
constexpr int kMaxPiece = 8;              // units that an item's beginning counts for, at most
constexpr uint32_t kWaitPolls = 750000;   // bound of every wait: one to three seconds, at 1.33 to 4 us a poll (measured)

struct Args {
  CUtensorMap km, vm;      // cache as {head_dim, slot or head, head or slot, page}
  int k_nhd, v_nhd;        // 1: the tensor map's second dimension is the head
  const void* q;
  void* out;
  long q_row, q_head, o_row, o_head;
  float* lse;
  const int *tables, *lens, *starts;
  const unsigned long long* mask;
  int B, N, W, nq, nkv, group, shift, max_rows, rows_each, len_add;
  float scale2;            // |scale| * log2(e)
  uint32_t flip;           // sign bits that turn q into -q where scale is negative, or 0
  int mt;                  // queries of a tile (MT)
  int mt_max;              // queries of an item at most (min(MT, max_rows * group))
  int ntq_max;             // items of a (request, KV head) at most
  int piece;               // units that an item's beginning counts for
  int rounds;              // of a chunk's units, at most
  int fold;                // fp32 queries, tiles of 128: units after which O moves to the sums (a power of two)
  int by_warp;             // few requests: every warp finds the CTA's units by itself
  int wide;                // few items: a CTA joins one query, else four
  int by_item;             // descriptors by item (else by the CTA that starts it)
  int4* desc;              // {first CTA, CTAs, request, KV head * ntq + query tile}
  float* part;             // [CTA][2][mt_max][HD]: output parts (0: of an item begun before, 1: begun here)
  float2* part_ml;         // [CTA][2][mt_max]: (maximum, sum)
  bf16* frag;              // fp32 queries: the output in a projection's operand order instead of rows (act_store)
  int frag_umma;
  int* err;                // status word, or null
  uint32_t polls;          // bound of a chunk's waits (kWaitPolls, unless a test makes some run out)
};

constexpr int kRounds = 3;   // that a chunk's units may be dealt out in

// A request as the kernel sees it: whatever lens and starts hold, rows lie in
// [0, N) and slots within the table.
struct Request {
  int s0, rows, len, p0, nt, ntq;   // first row, rows computed, slots, the pass's first slot, units, query tiles
};

template <int MT>
__device__ __forceinline__ Request request(const Args& a, int b) {
  Request r;
  int rows;
  if (a.starts) {
    r.s0 = a.starts[b];
    rows = a.starts[b + 1] - r.s0;
  } else {
    r.s0 = b * a.rows_each;
    rows = a.rows_each;
  }
  r.len = (int)min((long)max(a.lens[b] + a.len_add, 0), (long)a.W << a.shift);
  r.p0 = r.len - rows;
  r.rows = (r.s0 < 0 || r.s0 >= a.N) ? 0 : max(0, min(min(rows, a.max_rows), a.N - r.s0));
  r.nt = r.rows > 0 ? max(1, (r.len + kTile - 1) / kTile) : 0;
  r.ntq = (r.rows * a.group + MT - 1) / MT;
  return r;
}

// T units over G CTAs: T / G each, and the first T % G one more.
struct Deal {
  long each, more;
  __device__ __forceinline__ Deal(long T, long G) : each(div(T, G)), more(T - each * G) {}
  static __device__ __forceinline__ long div(long x, long y) {   // (a 64-bit division is a long call)
    return (x | y) >> 32 ? x / y : (long)((unsigned)x / (unsigned)y);
  }
  __device__ __forceinline__ long first(long c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int cta_of(long u) const {
    const long big = more * (each + 1);
    return (int)(u < big ? div(u, each + 1) : more + div(u - big, each));
  }
};

// Wait on an mbarrier phase; false after seconds without it (the copies and
// products waited for take microseconds). Counted in polls: a kernel that is
// switched out while it waits, whatever the clock says, has not waited.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) {
  return mbar_wait(bar, parity, kWaitPolls);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_wait(bar, parity, 1)) return true;
  return wait_long(bar, parity);   // (out of line: a call costs nothing then)
}

template <typename T>
struct Num;
template <>
struct Num<bf16> {
  static constexpr uint32_t kExp = 0x7f80u;   // exponent bits: all set in infinities and NaN
  static constexpr int kUp = 0;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Num<__half> {
  static constexpr uint32_t kExp = 0x7c00u;
  // Probabilities are at most 2^kUp, so that fp16 holds those down to 2^-29 of
  // the largest with all their bits and the rest to 2^-40 of it. (At most 1,
  // they lost bits from 2^-14 on and everything from 2^-25: behind one slot far
  // above the others the others' values were gone while the sum counted them.)
  static constexpr int kUp = 15;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __low2float(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __high2float(*reinterpret_cast<const __half2*>(&w)); }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ float exp2_approx(float x) {   // relative error 2^-22; 0 below the normal range
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
template <int HD, int WM, int WK, bool F32>
struct Shape {
  static constexpr int MT = 16 * WM;                 // queries of an item
  static constexpr int kWarps = WM * WK;             // consumer warps
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kHalf = HD / 64;              // 64-dimension boxes of a key
  static constexpr int kBox = kTile * 128;           // bytes of one box column: 64 slots x 64 dimensions
  static constexpr int kStage = 2 * kHalf * kBox;    // keys and values of a unit
  static constexpr int QP = HD + 8;                  // pitch of fp32 queries in shared memory (others: registers)
  // Parts (output, and behind it maximum and sum) in shared memory: pitch (4
  // more would cost 32 fp32 queries a stage of the ring).
  static constexpr int OP = HD + (F32 && WM == 2 ? 4 : 8);
  static constexpr int kQBytes = F32 ? 3 * MT * QP * 2 : 0;
  static constexpr int kOBytes = WK * MT * OP * 4;
  static constexpr int kExtra = kQBytes + kOBytes;
  static constexpr int kMaxStages = 6;
  // Two CTAs on an SM when at least two stages fit in half its shared memory
  // and the registers do: the 16-bit kernel with two query tiles at head
  // dimension 128 would spill (8 sequences of 4096 to 8192 tokens, 8 KV heads,
  // 20 queries: 38.6 us with one CTA, 45.3 with two).
  static constexpr int kFit2 = (kHalfSmBytes - 1024 - kExtra) / kStage;
  static constexpr int kCtas = kFit2 >= 2 && !(HD == 128 && WK == 2) ? 2 : 1;
  static constexpr int kFit1 = (220 * 1024 - 1024 - kExtra) / kStage;
  static constexpr int kFit = kCtas == 2 ? kFit2 : kFit1;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kSmem = 1024 + kStages * kStage + kExtra;
  // Units that an item's beginning counts for: a CTA that begins one in the
  // midst of its units otherwise ends that much later. 32 sequences of 0 to
  // 8191 tokens, 7 queries: 47.4 us, 48.4 with none (2 to 5 are alike, 49.1
  // with 14); 120 of up to 1000 tokens 29.3 and 36.5; fp32, one of 2057 tokens,
  // 63 queries 11.1 and 14.1; 16 of 5 to 4099 tokens, 91 queries 13.1 and 15.8.
  static constexpr int kPiece = 4;
  // Units after which a warp's output and sum move to the part in shared
  // memory. The tensor cores cut off what they add, always towards zero, and
  // rounded sums of many like terms err one way as well: over 2^20 slots in one
  // CTA outputs were 0.08% too small in tiles of 16 and 0.25% in tiles of 32,
  // sums of equal probabilities 1e-4 off.
  static constexpr int kFold = 128;
};

// Where a CTA's units begin.
struct Start {
  long T;       // units in all (items' beginnings included)
  long base;    // units before request b
  int b;
  Request r;    // request b
};

// Every warp by itself, for at most 32 requests and 2^31 units: the first
// copies need not wait for the other warps.
template <int MT>
__device__ __forceinline__ Start locate_warp(const Args& a) {
  const int lane = threadIdx.x & 31;
  Request r{};
  if (lane < a.B) r = request<MT>(a, lane);
  const int n = a.nkv * r.ntq * (r.nt + a.piece);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const int T = __shfl_sync(0xffffffffu, incl, 31);
  Start s{};
  s.T = T;
  const long G = min((long)gridDim.x, s.T);
  if ((long)blockIdx.x >= G) return s;
  const int u0 = (int)Deal(T, G).first(blockIdx.x);
  s.b = __ffs(__ballot_sync(0xffffffffu, incl > u0)) - 1;
  s.base = __shfl_sync(0xffffffffu, incl - n, s.b);
  s.r.s0 = __shfl_sync(0xffffffffu, r.s0, s.b);
  s.r.rows = __shfl_sync(0xffffffffu, r.rows, s.b);
  s.r.len = __shfl_sync(0xffffffffu, r.len, s.b);
  s.r.p0 = __shfl_sync(0xffffffffu, r.p0, s.b);
  s.r.nt = __shfl_sync(0xffffffffu, r.nt, s.b);
  s.r.ntq = __shfl_sync(0xffffffffu, r.ntq, s.b);
  return s;
}

// All threads of the CTA together, for any number of requests.
template <int MT, int NT>
__device__ __forceinline__ Start locate_cta(const Args& a, long* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = NT / 32;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request<MT>(a, b);
    mine += (long)a.nkv * r.ntq * (r.nt + a.piece);
  }
  long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  Start s;
  long before = 0;
  s.T = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += sh[w];
    s.T += sh[w];
  }
  const long G = min((long)gridDim.x, s.T);
  const long u0 = (long)blockIdx.x < G ? Deal(s.T, G).first(blockIdx.x) : -1;
  const long lo = before + incl - mine;
  if (u0 >= lo && u0 < lo + mine) {
    long base = lo;
    for (int b = b0; b < b1; ++b) {
      const Request r = request<MT>(a, b);
      const long n = (long)a.nkv * r.ntq * (r.nt + a.piece);
      if (u0 < base + n) {
        sh[NW] = base;
        sh[NW + 1] = b;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  s.base = u0 < 0 ? 0 : sh[NW];
  s.b = u0 < 0 ? 0 : (int)sh[NW + 1];
  s.r = request<MT>(a, s.b);
  return s;
}

// Walks the pieces of items that a CTA's units [u, u1) make up.
template <int MT>
struct Walk {
  long u;          // units before the next piece
  int left, rem;   // units of the CTA from there on; units of request b before it
  int b;
  Request r;
  int item, kvh, qt, t0, t1;   // the current piece: item within the request, units of slots t0 .. t1 - 1
  bool open = false;           // its item begins here and goes on in the next CTA
  __device__ __forceinline__ Walk(const Start& s, long first, long last)
      : u(first), left((int)(last - first)), rem((int)(first - s.base)), b(s.b), r(s.r) {}
  // The next piece; false at the end.
  __device__ __forceinline__ bool next(const Args& a) {
    while (left > 0) {
      const int len = r.nt + a.piece;
      if (rem >= a.nkv * r.ntq * len) {
        rem = 0;
        r = request<MT>(a, ++b);
        continue;
      }
      const int it = rem / len, first = rem - it * len, take = min(len - first, left);
      u += take;
      rem += take;
      left -= take;
      if (first + take <= a.piece) continue;   // (no slots: the item's pieces are the next CTAs')
      item = it;
      t0 = max(0, first - a.piece);
      t1 = first + take - a.piece;
      kvh = item / r.ntq;
      qt = item - kvh * r.ntq;
      open = t0 == 0 && t1 < r.nt;
      return true;
    }
    return false;
  }
};

template <typename TQ>
__device__ __forceinline__ void store2(TQ* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = Num<TQ>::pack(x, y);
}
template <>
__device__ __forceinline__ void store2<float>(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}

// The producer warp: the pieces' units, 64 slots of keys and values each, into
// the ring.
template <int STAGES, int HALF, int BOX, int STAGE, int MT>
__device__ __forceinline__ void produce(const Args& a, Walk<MT>& w, unsigned char* ring, uint64_t* full,
                                        uint64_t* empty, bool& ok) {
  const int lane = threadIdx.x & 31;
  const int bp = min(1 << a.shift, kTile);        // slots of a box
  const int np = kTile / bp;                      // boxes of a column
  const int boxes = np * HALF * 2;
  const int i = lane % np, h = (lane / np) % HALF, is_v = lane / (np * HALF);
  const uint32_t dst0 = smem_u32(ring) + (is_v * HALF + h) * BOX + i * bp * 128;
  const CUtensorMap* map = is_v ? &a.vm : &a.km;
  const int nhd = is_v ? a.v_nhd : a.k_nhd;
  int win_b = -1, win = -1, entry = 0;            // the 32 table entries at hand, one per lane
  int n = 0;
  while (ok && w.next(a)) {
    const uint64_t policy = w.r.ntq == 1 ? policy_evict_first() : policy_evict_normal();
    for (int t = w.t0; t < w.t1; ++t, ++n) {
      const int s = n % STAGES;
      const int first = (t * kTile) >> a.shift;
      if (w.b != win_b || (first >> 5) != win) {
        win_b = w.b;
        win = first >> 5;
        const int e = 32 * win + lane;
        entry = e < a.W ? a.tables[(long)w.b * a.W + e] : -1;
      }
      if (n >= STAGES) ok = wait(&empty[s], (n / STAGES - 1) & 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int left = w.r.len - t * kTile;       // slots from here on
      const int nb = max(0, min(np, (left + bp - 1) / bp));
      const int page = __shfl_sync(0xffffffffu, entry, (first + i) & 31);
      if (lane == 0) mbar_expect_tx(&full[s], nb * bp * 128 * HALF * 2);
      __syncwarp();
      if (lane < boxes && i < nb) {
        const int off = (t * kTile) & ((1 << a.shift) - 1) & ~(kTile - 1);
        tma_load_4d(dst0 + s * STAGE, map, 64 * h, nhd ? w.kvh : off, nhd ? off : w.kvh, page, &full[s], policy);
      }
    }
  }
  // An expired wait: the copies in flight land before the CTA may end.
  if (!ok)
    for (int k = max(0, n - STAGES); k < n; ++k) wait(&full[k % STAGES], (k / STAGES) & 1);
}

// The join's descriptor of an item that begins in this CTA (one thread).
template <int MT>
__device__ __forceinline__ void describe(const Args& a, const Walk<MT>& w, const Deal& deal, bool whole) {
  const int c1 = whole ? (int)blockIdx.x : deal.cta_of(w.u - w.t1 + w.r.nt - 1);
  const int4 d = make_int4(blockIdx.x, c1 - (int)blockIdx.x + 1, w.b, w.item);
  if (a.by_item) a.desc[((long)w.b * a.nkv + w.kvh) * a.ntq_max + w.qt] = d;
  else if (!whole) a.desc[blockIdx.x] = d;
}
// Descriptors by CTA: none when no item begins here that others share.
template <int MT>
__device__ __forceinline__ void describe_none(const Args& a, const Walk<MT>& w) {
  if (!a.by_item && !w.open) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
}

// Two neighbouring elements of row `row`, head `head` of the output.
template <int HD, typename TQ>
__device__ __forceinline__ void put2(const Args& a, int row, int head, int d, float x, float y) {
  if constexpr (std::is_same<TQ, float>::value) {
    if (a.frag) {
      const int T = (a.N + 3) / 4;
      act_store(a.frag, row, head * HD + d, T, x, a.frag_umma);
      act_store(a.frag, row, head * HD + d + 1, T, y, a.frag_umma);
      return;
    }
  }
  store2<TQ>(static_cast<TQ*>(a.out) + row * a.o_row + head * a.o_head + d, x, y);
}

// TC: the cache's type. F32: fp32 queries and output over a bf16 cache, the
// queries and the probabilities as three bf16 terms each (24 bits: exact).
template <int HD, typename TC, bool F32, int WM, int WK>
__global__ void __launch_bounds__(Shape<HD, WM, WK, F32>::kThreads, Shape<HD, WM, WK, F32>::kCtas)
    k_paged_attn(const __grid_constant__ Args a) {
  using S = Shape<HD, WM, WK, F32>;
  using TQ = typename std::conditional<F32, float, TC>::type;
  constexpr int MT = S::MT, SW = kTile / WK, KS = HD / 16, ND = HD / 8, NS = SW / 8, NQ = F32 ? 3 : 1;
  extern __shared__ unsigned char pa_smem_raw[];
  unsigned char* ring = pa_smem_raw + ((1024 - (smem_u32(pa_smem_raw) & 1023)) & 1023);
  unsigned char* extra = ring + S::kStages * S::kStage;
  __shared__ long sh_loc[S::kWarps + 3];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], S::kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (tid >= S::kWarps * 32 && lane < 2) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &a.vm : &a.km)) : "memory");
  }
  __syncthreads();
  pdl_wait();          // the kernels before this one have finished
  pdl_launch_next();   // the join may come up meanwhile (it waits for this kernel's end)
  const Start st = a.by_warp ? locate_warp<MT>(a) : locate_cta<MT, S::kThreads>(a, sh_loc);
  const long G = min((long)gridDim.x, st.T);
  if ((long)blockIdx.x >= G) {
    if (tid == 0 && !a.by_item) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  const Deal deal(st.T, G);
  const long u0 = deal.first(blockIdx.x), u1 = deal.first(blockIdx.x + 1);
  Walk<MT> w(st, u0, u1);

  bool ok = true;
  if (warp == S::kWarps) {
    produce<S::kStages, S::kHalf, S::kBox, S::kStage, MT>(a, w, ring, full, empty, ok);
    return;
  }

  // ------------------------------------------------------------ consumer warps
  const int wm = warp / WK, wk = warp % WK;
  const int g = lane >> 2, c4 = lane & 3;
  auto cta_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(S::kWarps * 32) : "memory"); };
  // This lane's ldmatrix rows (keys: 16 slots x 16 dimensions; values: 16
  // slots x 16 dimensions, transposed): 16-byte piece p of slot s lies at
  // (128 s + 16 (s % 8)) ^ 16 p of its box column.
  const int k_slot = wk * SW + (lane & 7) + 8 * (lane >> 4), v_slot = wk * SW + (lane & 7) + 8 * ((lane >> 3) & 1);
  const uint32_t k_off = (k_slot * 128 + ((k_slot & 7) << 4)) ^ (((lane >> 3) & 1) << 4);
  const uint32_t v_off = (v_slot * 128 + ((v_slot & 7) << 4)) ^ ((lane >> 4) << 4);
  int n = 0;
  while (w.next(a)) {
    const Request r = w.r;
    const int q0 = w.qt * MT + 16 * wm + g;        // this lane's queries: q0 and q0 + 8
    const int Mq = r.rows * a.group;
    uint32_t qf[F32 ? 1 : KS][4];
    if constexpr (F32) {
      // The tile's queries in shared memory, as three bf16 terms.
      TC* sq = reinterpret_cast<TC*>(extra);
      cta_sync();   // the region's last readers are done
      constexpr int E = 4;                                // elements of a 16-byte load
      constexpr int NL = MT * HD / E / (S::kWarps * 32);  // loads of a thread, all in flight together
      uint4 f[NL];
#pragma unroll
      for (int y = 0; y < NL; ++y) {
        const int e = tid + y * S::kWarps * 32, m = e / (HD / E), d = E * (e - m * (HD / E));
        const int x = w.qt * MT + m, jj = x / a.group, hh = w.kvh * a.group + x - jj * a.group;
        f[y] = make_uint4(0u, 0u, 0u, 0u);
        if (x < Mq)
          f[y] = *reinterpret_cast<const uint4*>(static_cast<const TQ*>(a.q) + (r.s0 + jj) * a.q_row + hh * a.q_head + d);
      }
#pragma unroll
      for (int y = 0; y < NL; ++y) {
        const int e = tid + y * S::kWarps * 32, m = e / (HD / E), d = E * (e - m * (HD / E));
        float v[4] = {__uint_as_float(f[y].x ^ a.flip), __uint_as_float(f[y].y ^ a.flip),
                      __uint_as_float(f[y].z ^ a.flip), __uint_as_float(f[y].w ^ a.flip)};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          uint32_t p[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            p[z] = Num<bf16>::pack(v[2 * z], v[2 * z + 1]);
            v[2 * z] -= Num<bf16>::lo(p[z]);
            v[2 * z + 1] -= Num<bf16>::hi(p[z]);
          }
          *reinterpret_cast<uint2*>(sq + (k * MT + m) * S::QP + d) = make_uint2(p[0], p[1]);
        }
      }
      cta_sync();
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = q0 + 8 * e, jj = x / a.group, hh = w.kvh * a.group + x - jj * a.group;
        const TQ* src = static_cast<const TQ*>(a.q) + (r.s0 + jj) * a.q_row + hh * a.q_head + 2 * c4;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[k][e] = x < Mq ? *reinterpret_cast<const uint32_t*>(src + 16 * k) ^ a.flip : 0u;
          qf[k][e + 2] = x < Mq ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) ^ a.flip : 0u;
        }
      }
    }
    float o[ND][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    float* const so = reinterpret_cast<float*>(extra + S::kQBytes);   // parts: [WK][MT][OP]
    auto so_ml = [&](int x) { return reinterpret_cast<float2*>(so + x * S::OP + HD); };
    // Adds what the warp's part holds to output and sum; its reference may be an
    // older maximum.
    auto unfold = [&] {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = wk * MT + 16 * wm + g + 8 * e;
        const float2 ml = *so_ml(x);
        const float f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m[e]) * a.scale2);
        if (c4 == 0) l[e] = fmaf(ml.y, f, l[e]);   // (a lane's l is a quarter of the row's)
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const float2 y = *reinterpret_cast<const float2*>(so + x * S::OP + 8 * d + 2 * c4);
          o[d][2 * e] = fmaf(y.x, f, o[d][2 * e]);
          o[d][2 * e + 1] = fmaf(y.y, f, o[d][2 * e + 1]);
        }
      }
    };
    // Output, sum and maximum to the warp's part.
    auto leave = [&] {
      __syncwarp();   // (what it held has been read)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int x = wk * MT + 16 * wm + g + 8 * e;
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
#pragma unroll
        for (int d = 0; d < ND; ++d)
          *reinterpret_cast<float2*>(so + x * S::OP + 8 * d + 2 * c4) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
        if (c4 == 0) *so_ml(x) = make_float2(m[e], l[e]);
      }
      __syncwarp();
    };

    // One unit. Every row sees all slots of a plain one; a tail unit holds
    // slots of the pass itself, or slots past the end; in an odd one, some of
    // the pass's values are no finite numbers.
    constexpr int PLAIN = 0, TAILED = 1, ODD = 2;
    auto unit = [&](auto kind, int t) {
      constexpr bool TAIL = decltype(kind)::value != PLAIN, CLEAN = decltype(kind)::value == ODD;
      const int s = n % S::kStages;
      const uint32_t ks = smem_u32(ring) + s * S::kStage, vs = ks + S::kHalf * S::kBox;
      const int base = t * kTile + wk * SW;         // this warp's first slot
      // ---- scores (fp32 queries: the small terms have a sum of their own, as the
      // tensor cores cut off what they add to a large one: 19 rows over up to 4144
      // slots, 128 dimensions, output off by 5.3e-7, 1.2e-6 without; as fast)
      float x[NS][4], small[F32 ? NS : 1][4] = {};
#pragma unroll
      for (int i = 0; i < NS; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t qk[NQ][4];
        if constexpr (F32) {
          const TC* sq = reinterpret_cast<const TC*>(extra);
#pragma unroll
          for (int e = 0; e < NQ; ++e)
            ldsm_x4(qk[e], smem_u32(sq + (e * MT + 16 * wm + (lane & 7) + 8 * ((lane >> 3) & 1)) * S::QP + 16 * k +
                                    8 * (lane >> 4)));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) qk[0][e] = qf[k][e];
        }
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) {
          uint32_t kb[4];
          ldsm_x4(kb, ((ks + k_off) ^ ((2 * k & 7) << 4)) + (k >> 2) * S::kBox + i * 2048);
#pragma unroll
          for (int e = NQ - 1; e >= 0; --e) {       // the small terms first
            Num<TC>::mma(e > 0 ? small[2 * i] : x[2 * i], qk[e], kb[0], kb[1]);
            Num<TC>::mma(e > 0 ? small[2 * i + 1] : x[2 * i + 1], qk[e], kb[2], kb[3]);
          }
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] += small[i][e];
      }
      // ---- what a row does not see is -infinity (set, not added: what such
      // slots hold, NaN included, does not matter). vis[e]: the slots of the
      // unit that row e sees, one bit each, this lane's own from bit 0 on.
      unsigned long long vis[2] = {0, 0};
      if constexpr (TAIL) {
        const int first = r.p0 - t * kTile;          // the pass's first slot, within the unit
        auto low = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1; };
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = q0 + 8 * e, j = q / a.group;
          if (q < Mq) {
            vis[e] = low(first + j + 1);
            if (a.mask) {
              const unsigned long long bits = a.mask[r.s0 + j];
              vis[e] = low(first) | (first >= 64 || first <= -64 ? 0ull : first >= 0 ? bits << first : bits >> -first);
            }
            vis[e] = (vis[e] & low(r.len - t * kTile)) >> (wk * SW + 2 * c4);
          }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(vis[e >> 1] >> (8 * i + (e & 1)) & 1)) x[i][e] = -INFINITY;
      }
      // ---- running maximum (of q . k; the scale is not negative) and sum
      float ref[2];
      bool raise = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(x[0][2 * e], x[0][2 * e + 1]);
#pragma unroll
        for (int i = 1; i < NS; ++i) mx = fmaxf(mx, fmaxf(x[i][2 * e], x[i][2 * e + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        ref[e] = fmaxf(m[e], mx);
        raise |= ref[e] != m[e];
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = m[e] == -INFINITY ? 0.f : exp2_approx((m[e] - ref[e]) * a.scale2);
          m[e] = ref[e];
          l[e] *= f;
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            o[d][2 * e] *= f;
            o[d][2 * e + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) ref[e] = m[e] == -INFINITY ? 0.f : fmaf(-m[e], a.scale2, (float)Num<TC>::kUp);
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][e] = exp2_approx(fmaf(x[i][e], a.scale2, ref[e >> 1]));
          sum[e >> 1] += x[i][e];
        }
      l[0] += sum[0];
      l[1] += sum[1];
      // ---- output: probabilities (the cache's type, or three bf16 terms) x
      // values. In a tail unit values past the end are cut off; in an odd one
      // the pass's values that are no finite numbers are taken out of the
      // product (a probability 0 times NaN is NaN) and added for the rows that
      // see them.
#pragma unroll
      for (int i = 0; i < NS / 2; ++i) {
        uint32_t p[NQ][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ti = 2 * i + (e >> 1), ei = 2 * (e & 1);
          float y0 = x[ti][ei], y1 = x[ti][ei + 1];
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
            p[k][e] = Num<TC>::pack(y0, y1);
            if (NQ > 1) {
              y0 -= Num<TC>::lo(p[k][e]);
              y1 -= Num<TC>::hi(p[k][e]);
            }
          }
        }
        const int s0 = base + 16 * i + 2 * c4;       // slots of this lane's value pairs: s0, s0 + 1 and s0 + 8, s0 + 9
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if constexpr (TAIL) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            keep[e] = (s0 + 8 * e < r.len ? 0xffffu : 0u) | (s0 + 8 * e + 1 < r.len ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int d = 0; d < ND / 2; ++d) {
          uint32_t vb[4];
          ldsm_x4_trans(vb, ((vs + v_off) ^ ((2 * d & 7) << 4)) + (d >> 2) * S::kBox + i * 2048);
          if constexpr (TAIL) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              vb[e] &= keep[e & 1];
              if constexpr (CLEAN) {
                constexpr uint32_t X = Num<TC>::kExp;
                const int sl = s0 + 8 * (e & 1);
                if ((vb[e] & X) == X && sl >= r.p0) vb[e] &= 0xffff0000u;
                if ((vb[e] >> 16 & X) == X && sl + 1 >= r.p0) vb[e] &= 0xffffu;
              }
            }
          }
          if constexpr (F32) {
            // (the tensor cores cut off what they add, so the sums over units
            // are added here: error 1.5e-6 where it was 4e-6 after 80 units; 11.1
            // us for one of 2057 tokens with 63 queries, 10.5 before)
            float y[2][4] = {};
#pragma unroll
            for (int k = NQ - 1; k >= 0; --k) {
              Num<TC>::mma(y[0], p[k], vb[0], vb[1]);
              Num<TC>::mma(y[1], p[k], vb[2], vb[3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[2 * d][e] += y[0][e], o[2 * d + 1][e] += y[1][e];
          } else {
            Num<TC>::mma(o[2 * d], p[0], vb[0], vb[1]);
            Num<TC>::mma(o[2 * d + 1], p[0], vb[2], vb[3]);
          }
        }
      }
      if constexpr (CLEAN) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            const int slot = base + 8 * i + c, src = (lane & ~3) + (c >> 1);
            const float pa = __shfl_sync(0xffffffffu, c & 1 ? x[i][1] : x[i][0], src);
            const float pb = __shfl_sync(0xffffffffu, c & 1 ? x[i][3] : x[i][2], src);
            // (the other lane's bits start at its own slots)
            const bool sa = __shfl_sync(0xffffffffu, (int)(vis[0] >> (8 * i + (c & 1)) & 1), src);
            const bool sb = __shfl_sync(0xffffffffu, (int)(vis[1] >> (8 * i + (c & 1)) & 1), src);
            if (slot < r.p0 || slot >= r.len) continue;
            const int sl = slot & (kTile - 1);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              uint32_t v;
              asm volatile("ld.shared.b32 %0, [%1];"
                           : "=r"(v)
                           : "r"(vs + (d >> 3) * S::kBox + sl * 128 + (((d & 7) ^ (sl & 7)) << 4) + 4 * c4));
              constexpr uint32_t X = Num<TC>::kExp;
              if ((v & X) == X) {
                if (sa) o[d][0] = fmaf(pa, Num<TC>::lo(v), o[d][0]);
                if (sb) o[d][2] = fmaf(pb, Num<TC>::lo(v), o[d][2]);
              }
              if ((v >> 16 & X) == X) {
                if (sa) o[d][1] = fmaf(pa, Num<TC>::hi(v), o[d][1]);
                if (sb) o[d][3] = fmaf(pb, Num<TC>::hi(v), o[d][3]);
              }
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      ++n;
    };
    auto arrived = [&] {
      if (ok && !wait(&full[n % S::kStages], (n / S::kStages) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
    };
    // Whether this warp's slots hold values of the pass that are no finite
    // numbers and that some row may not see (one row sees all there is).
    auto odd_values = [&](int t) {
      if (r.len - r.p0 <= 1 && !a.mask) return false;
      const uint32_t vs = smem_u32(ring) + n % S::kStages * S::kStage + S::kHalf * S::kBox;
      const int s0 = max(wk * SW, r.p0 - t * kTile), s1 = min((wk + 1) * SW, r.len - t * kTile);
      bool odd = false;
      for (int e = lane; e < (s1 - s0) * 8 * S::kHalf; e += 32) {   // 16-byte pieces, in any order
        const int sl = s0 + e / (8 * S::kHalf), p = e % (8 * S::kHalf);
        uint32_t v[4];
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(vs + (p >> 3) * S::kBox + sl * 128 + (p & 7) * 16));
        constexpr uint32_t X = Num<TC>::kExp;
#pragma unroll
        for (int y = 0; y < 4; ++y) odd |= (v[y] & X) == X || (v[y] >> 16 & X) == X;
      }
      return (bool)__any_sync(0xffffffffu, odd);
    };
    const int plain = max(0, min(r.p0, r.len)) / kTile;   // units whose slots every row sees
    int t = w.t0;
    if (w.qt * MT + 16 * wm >= Mq) {   // no query for this warp: it only keeps the ring going
      for (; t < w.t1; ++t, ++n) {
        arrived();
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[n % S::kStages]);
      }
    }
    auto fold_now = [&] {
      if ((t - w.t0) % S::kFold || t == w.t0) return;
      if (t - w.t0 > S::kFold) unfold();
      leave();
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    };
    for (; t < min(w.t1, plain); ++t) {
      fold_now();
      arrived();
      unit(std::integral_constant<int, PLAIN>{}, t);
    }
    for (; t < w.t1; ++t) {
      fold_now();
      arrived();
      if (odd_values(t)) unit(std::integral_constant<int, ODD>{}, t);
      else unit(std::integral_constant<int, TAILED>{}, t);
    }

    // ---- the end of the piece: everything to this warp's part
    if (w.t1 - w.t0 > S::kFold) unfold();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!ok) l[e] = __int_as_float(0x7fc00000);   // an expired wait: NaN
      if (m[e] != -INFINITY) m[e] = fmaf(m[e], a.scale2, (float)-Num<TC>::kUp);
    }
    leave();
    const bool begins = w.t0 == 0, whole = begins && w.t1 == r.nt;
    if (begins && tid == 0) describe(a, w, deal, whole);
    const long slot = 2l * blockIdx.x + (begins ? 1 : 0);
    float* part = a.part + slot * a.mt_max * HD;
    float2* part_ml = a.part_ml + slot * a.mt_max;
    const float kLn2 = 0.693147180559945f;
    // Joined over the warps that shared out the slots.
    cta_sync();
    for (int e = tid; e < MT * (HD / 4); e += S::kWarps * 32) {
      const int x = e / (HD / 4), d = 4 * (e - x * (HD / 4));
      const int q = w.qt * MT + x;
      if (q >= Mq) break;
      float mm = -INFINITY, ll = 0.f, f[WK];
      float2 ml[WK];
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        ml[k] = *so_ml(k * MT + x);
        mm = fmaxf(mm, ml[k].x);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        f[k] = ml[k].x == -INFINITY ? 0.f : exp2_approx(ml[k].x - mm);
        // (a warp that saw nothing has l = 0; one whose wait expired, NaN)
        ll += ml[k].x == -INFINITY ? ml[k].y : ml[k].y * f[k];
        const float4 y = *reinterpret_cast<const float4*>(so + (k * MT + x) * S::OP + d);
        v.x = fmaf(y.x, f[k], v.x);
        v.y = fmaf(y.y, f[k], v.y);
        v.z = fmaf(y.z, f[k], v.z);
        v.w = fmaf(y.w, f[k], v.w);
      }
      if (whole) {
        const int jj = q / a.group, hh = w.kvh * a.group + q - jj * a.group;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        put2<HD, TQ>(a, r.s0 + jj, hh, d, v.x * inv, v.y * inv);
        put2<HD, TQ>(a, r.s0 + jj, hh, d + 2, v.z * inv, v.w * inv);
        if (a.lse && d == 0) a.lse[(long)(r.s0 + jj) * a.nq + hh] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
      } else {
        *reinterpret_cast<float4*>(part + x * HD + d) = v;
        if (d == 0) part_ml[x] = make_float2(mm, ll);
      }
    }
    cta_sync();   // the region is free again
  }
  if (!ok && lane == 0) report_err(a.err, kErrWait);
  if (tid == 0) describe_none(a, w);
}

// The join of the items that several CTAs share: the parts lie with the CTAs
// first .. first + count - 1. With few items (`wide`: many parts each) one CTA
// per (item, query), its four warps taking the parts in turn and their sums
// added in order; else a warp per (item, query).
constexpr int kJoinThreads = 128;

template <int HD, typename TQ, int MT>
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ Args a) {
  constexpr int V = HD / 32;   // dimensions of a lane
  __shared__ float so[4][HD];
  __shared__ float2 sml[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = a.wide ? blockIdx.y : 4 * blockIdx.y + warp;   // query of the tile
  pdl_launch_next();
  Request r;
  int kvh = 0, qt = 0;
  if (a.by_item) {   // items of requests with fewer rows have no descriptor
    const int b = blockIdx.x / (a.nkv * a.ntq_max), i = blockIdx.x - b * a.nkv * a.ntq_max;
    kvh = i / a.ntq_max;
    qt = i - kvh * a.ntq_max;
    r = request<MT>(a, b);
  }
  pdl_wait();   // (before any return: what follows the join relies on the main kernel's end as well)
  if (a.by_item && qt * MT + x >= r.rows * a.group) return;   // (all of a wide join's CTA)
  const int4 d = a.desc[blockIdx.x];
  if (d.y < 2) return;
  if (!a.by_item) {
    r = request<MT>(a, d.z);
    kvh = d.w / r.ntq;
    qt = d.w - kvh * r.ntq;
  }
  const int q = qt * MT + x;
  if (q >= r.rows * a.group) return;
  auto slot = [&](int k) { return (2l * (d.x + k) + (k == 0 ? 1 : 0)) * a.mt_max + x; };
  const int k0 = a.wide ? warp : 0, step = a.wide ? 4 : 1;
  // A running maximum again, over batches of eight parts loaded together.
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = 0.f;
  for (int kb = k0; kb < d.y; kb += 8 * step) {
    float v[8][V];
    float2 ml[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = kb + i * step;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
      if (k < d.y) {
        ml[i] = a.part_ml[slot(k)];
        const float* p = a.part + slot(k) * HD + V * lane;
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(p);
          v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(p);
          v[i][0] = f.x, v[i][1] = f.y;
        }
      }
    }
    float mm = m;
#pragma unroll
    for (int i = 0; i < 8; ++i) mm = fmaxf(mm, ml[i].x);
    const float f0 = m == -INFINITY ? 0.f : exp2_approx(m - mm);
    m = mm;
    if (m != -INFINITY) l *= f0 == 0.f && l != l ? 1.f : f0;   // (a NaN stays)
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = ml[i].x == -INFINITY ? 0.f : exp2_approx(ml[i].x - m);
      l += ml[i].x == -INFINITY ? ml[i].y : ml[i].y * f;   // (a part that saw nothing has sum 0, a failed one NaN)
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(v[i][e], f, o[e]);
    }
  }
  if (a.wide) {
#pragma unroll
    for (int e = 0; e < V; ++e) so[warp][V * lane + e] = o[e];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp > 0) return;
    m = fmaxf(fmaxf(sml[0].x, sml[1].x), fmaxf(sml[2].x, sml[3].x));
    l = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = sml[k].x == -INFINITY ? 0.f : exp2_approx(sml[k].x - m);
      l += sml[k].x == -INFINITY ? sml[k].y : sml[k].y * f;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf(so[k][V * lane + e], f, o[e]);
    }
  }
  const int jj = q / a.group, hh = kvh * a.group + q - jj * a.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  put2<HD, TQ>(a, r.s0 + jj, hh, V * lane, o[0] * inv, o[1] * inv);
  if constexpr (V == 4) put2<HD, TQ>(a, r.s0 + jj, hh, V * lane + 2, o[2] * inv, o[3] * inv);
  if (a.lse && lane == 0) a.lse[(long)(r.s0 + jj) * a.nq + hh] = l == 0.f ? -INFINITY : m * 0.693147180559945f + logf(l);
}

}  // namespace pa
}  // namespace sf
