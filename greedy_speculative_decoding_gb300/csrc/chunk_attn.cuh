// Attention of a chunk of new tokens over a paged cache: many rows a request,
// so that the products bound it and not the cache's bytes.
//
// The formula is paged_attn.cuh's, and so are an item (request, KV head, tile
// of queries) and the deal of the items' units over the CTAs. Here a unit is 128 slots, an item 256 queries in two
// tiles of 128, and an item has only the units that its last row sees: of a
// prompt's first tokens few. The number of units of item q of a request with g
// query heads a KV head and the pass's first row in slot p0 is
//   ceil((p0 + floor((256 q + 255) / g) + 1) / 128) = floor((2 q + C) / g),
//   C = floor((255 + g (p0 + 128)) / 128),
// whose sums have a closed form, so a CTA finds its units without a plan.
//
// A CTA (one on an SM), twelve warps:
//   * two times four softmax warps, one tile each, a thread per query: they read
//     the scores from tensor memory, write the probabilities in their place, and
//     rescale the output when a row's maximum has outgrown its reference;
//   * a producer warp, which finds the CTA's pieces of items, tells the other
//     warps, and brings keys and values, 128 slots at a time, into a ring of
//     tiles (TMA, 128-byte swizzle);
//   * an MMA warp: S = Q K^T (queries and keys in shared memory) and O += P V
//     (probabilities in tensor memory), tile by tile in turn, so that the tensor
//     cores work on one tile while the other's softmax runs. Their queue holds
//     about four MMAs (256 cycles), so what happens between two of them counts:
//     with the whole warp in the loop, one lane elected for every few MMAs, a
//     wait takes 130 to 160 cycles even when there is nothing to wait for, and
//     two tiles' 32 MMAs and four waits 2200 to 2500 cycles; with the loop in
//     one lane, 2048, which is the tensor cores' rate. (A warp for each tile:
//     the tiles' products mix, both end together, and the tensor cores idle
//     through both softmaxes.)
//   * two warps that look through the values of slots that some row does not
//     see (those past the end among them), as a probability 0 times NaN is NaN:
//     values that are no finite numbers become 0, and the rows that do see them
//     NaN.
// Tensor memory holds both tiles' O and S (P over S), 512 columns at head
// dimension 128.
//
// Measured: 2048 rows over 16384 tokens, 40 / 8 heads of 128, 362 us (1780
// TFLOP/s), of 64 299; a whole prompt of 8192, 28 / 4 heads of 128, 296 (1625);
// nine prompts of 33..4099 tokens 296. Tried, at 128 and 64, for what stood then:
// the maximum of half a unit at a time 458 for 405 and 463 for 320; P apart from
// S, 388 for 317 at 64; a third warpgroup that loads and stores 466 for 392;
// scalar multiplications in place of pairs 416 for 405 and 346 for 319; one
// barrier for all of P 419 for 408 and 350 for 320; the next queries copied beside
// the last softmax 390 for 363 and 319 for 300.
#pragma once

#include "paged_attn_tc.cuh"

namespace sf {
namespace pa {

template <int HD, typename TC>
struct ChunkShape {
  static constexpr int MT = 256;                        // queries of an item
  static constexpr int kSlots = 128;                    // of a unit
  static constexpr int kThreads = 384;
  // Registers of a softmax thread and of the other warps': 2 x 128 x 200 + 128 x 104 = 384 x 168, the launch's (216 and
  // 72: the producer spills, 4 us of nine prompts' 316).
  static constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;
  static constexpr int kHalf = HD / 64;
  static constexpr int kBox = 128 * 128;                // 128 rows of 64 dimensions
  static constexpr int kTileBytes = kHalf * kBox;       // of queries, keys or values
  static constexpr int kStages = HD == 128 ? 4 : 10;
  static constexpr int kStaging = 4096;                 // bytes of a softmax warp: 128 of each row on their way out
  static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 8 * kStaging;
  static constexpr int kO = 0, kS = 2 * HD;             // tensor-memory columns: O of both tiles, S of both
  // As in TcShape: bounds of a reference's lag and the scale of fp16 probabilities, in powers of two.
  static constexpr int kLag = std::is_same<TC, __half>::value ? 3 : 8;
  static constexpr int kUp = std::is_same<TC, __half>::value ? 12 : 0;
  static constexpr int kFold = 128;                     // units after which O moves to the part (16384 slots, as there)
  // Units that an item's beginning counts for (queries in, output out, and the
  // first scores and last output, which nothing runs beside). Nine whole prompts
  // at the 7B shape: 2 356 us, 3 327, 4 319, 5 341.
  static constexpr int kPiece = 4;
  // Units of 128 slots whose keys and values stay in L2 (64 MB of 129; at 96 MB 24576 tokens take 584 us; chunk_walk).
  static constexpr long kRound = (64l << 20) / (kSlots * HD * 4);
};

// The units of a request's items.
struct ItemUnits {
  int g, ntq, last, c1, c0, piece;
  __device__ __forceinline__ ItemUnits() {}
  __device__ __forceinline__ ItemUnits(const Args& a, const Request& r) : g(a.group), ntq(r.ntq), piece(a.piece) {
    const int p0 = max(r.p0, 0);   // (rows in front of slot 0 see nothing and count as if they saw the first slots)
    const int C = (int)((255 + (long)g * (p0 + 128)) >> 7);
    c1 = (int)((unsigned)C / (unsigned)g);
    c0 = C - c1 * g;
    last = (p0 + r.rows + 127) >> 7;
  }
  // Units of item q.
  __device__ __forceinline__ int of(int q) const {
    return q == ntq - 1 ? last : c1 + (int)((unsigned)(2 * q + c0) / (unsigned)g);
  }
  // Units before item n < ntq of a head, items' beginnings included: the sum
  // over q < n of floor((2 q + c0) / g) counts for every v >= 1 the q with
  // 2 q + c0 >= v g.
  __device__ __forceinline__ long before(int n) const {
    if (n == 0) return 0;
    const long M = (unsigned)(2 * (n - 1) + c0) / (unsigned)g;   // the largest term
    const long odd = g & 1 ? (c0 & 1 ? M / 2 : (M + 1) / 2) : (c0 & 1 ? M : 0);
    return (long)n * (piece + c1) + M * n - ((g * (M * (M + 1) / 2) - M * c0 + odd) >> 1);
  }
  __device__ __forceinline__ long head() const { return ntq > 0 ? before(ntq - 1) + piece + last : 0; }
  // The item with unit x of a head (by a warp together).
  __device__ __forceinline__ int find(long x) const {
    int lo = 0, n = ntq;   // the item lies in lo .. lo + n - 1
    while (n > 1) {
      const int step = (n + 31) >> 5, q = lo + step * (int)(threadIdx.x & 31);
      const unsigned in = __ballot_sync(0xffffffffu, q < lo + n && before(q) <= x);
      const int k = 31 - __clz(in);
      n = min(step, n - k * step);
      lo += k * step;
    }
    return lo;
  }
};

// Walks the pieces of items that a CTA's units make up (Walk's counterpart).
struct ChunkWalk {
  long u;          // units before the next piece
  long left;       // units of the CTA from there on
  int b;
  Request r;
  ItemUnits iu;
  int kvh, qt, at; // the item at hand and its units done, its beginning included
  int t0, t1, nt;  // the piece: units t0 .. t1 - 1 of nt
  bool open = false;
  __device__ __forceinline__ bool next(const Args& a) {
    while (left > 0) {
      if (r.ntq == 0 || kvh == a.nkv) {
        r = request<256>(a, ++b);
        iu = ItemUnits(a, r);
        kvh = qt = at = 0;
        continue;
      }
      nt = iu.of(qt);
      const int all = nt + iu.piece, first = at, take = (int)min((long)(all - at), left);
      const int q = qt, h = kvh;
      u += take;
      left -= take;
      at += take;
      if (at == all) {
        at = 0;
        if (++qt == iu.ntq) {
          qt = 0;
          ++kvh;
        }
      }
      if (first + take <= iu.piece) continue;   // (no slots: the item's pieces are the next CTAs')
      item_q = q;
      item_h = h;
      t0 = max(0, first - iu.piece);
      t1 = first + take - iu.piece;
      open = t0 == 0 && t1 < nt;
      return true;
    }
    return false;
  }
  int item_q, item_h;   // query tile and KV head of the piece
};

// Where one of a CTA's shares of the units begins.
struct ShareStart {
  long u, left;   // units before it, and its own
  long base;      // units before its request
  int b;
};
// What the CTA's warps know of its shares, in shared memory.
struct Shares {
  long each, more;   // Deal's
  int rounds;
  ShareStart start[kRounds];
  __device__ __forceinline__ int cta_of(long u) const {
    Deal d(1, 1);
    d.each = each, d.more = more;
    return d.cta_of(u);
  }
};

// A CTA's shares of the units: all threads of the CTA together.
//
// With one share a CTA, all requests and heads are at work at the same time, and
// where their keys and values are more than L2 holds, items bring them from memory
// again. So then the units are dealt out in up to three rounds, one after the
// other over all CTAs (share v = CTA + round * CTAs), if items are enough that a
// round still shares keys and values (eight items a head) and the shares stay long
// (64 units). 40 / 8 heads of 128, us in one round and in rounds: 17000 tokens (66
// MB), 40 items a head (2048 rows) 390 and 391; 24576 584 and 569, 16 items 259 and
// 245; 32768 811 and 758 (without a pause, at the power cap, 927 to 969 and 850 to
// 875 once), 12 items 271 and 250; 65536, 40 items 1690 and 1583 (three), 8 374 and
// 344. Not taken: 24576, 8 items 136 and 141, 2 57 and 80; 32768, 8 items 188 and
// 178, 4 105 and 114; 65536, 6 items 289 and 272, 4 196 and 205. At 64 dimensions,
// where the exponentials bound it, calls ask for one round (32 / 16 heads, 32768
// tokens, 40 items 1120 and 1130, 24 704 and 719, 2 80 and 90).
template <int HD, typename TC>
__device__ __forceinline__ void chunk_walk(const Args& a, long* sh, Shares& shares) {
  using S = ChunkShape<HD, TC>;
  constexpr int NT = S::kThreads, NW = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long mine = 0, cache = 0;   // units; units of all items' longest, of each head
  for (int b = b0; b < b1; ++b) {
    const ItemUnits iu(a, request<256>(a, b));
    mine += a.nkv * iu.head();
    if (iu.ntq > 0) cache += (long)a.nkv * iu.last;
  }
  long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (a.rounds > 1) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) cache += __shfl_xor_sync(0xffffffffu, cache, o);
  }
  if (lane == 31) {
    sh[warp] = incl;
    sh[NW + warp] = cache;
  }
  __syncthreads();
  long before = 0, T = 0;
  cache = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += sh[w];
    T += sh[w];
    cache += sh[NW + w];
  }
  int rounds = 1;
  while (rounds < a.rounds && cache > rounds * S::kRound && T >= 8 * cache && T >= 64l * (rounds + 1) * gridDim.x) ++rounds;
  const long G = min((long)rounds * gridDim.x, T);
  const Deal deal(max(T, 1l), max(G, 1l));
  if (tid == 0) {
    shares.each = deal.each;
    shares.more = deal.more;
    shares.rounds = rounds;
  }
  const long lo = before + incl - mine;
  for (int i = 0; i < rounds; ++i) {
    const long v = blockIdx.x + (long)i * gridDim.x, u0 = v < G ? deal.first(v) : -1;
    if (tid == 0 && v >= G) shares.start[i] = ShareStart{0, 0, 0, 0};
    if (u0 >= lo && u0 < lo + mine) {
      long base = lo;
      for (int b = b0; b < b1; ++b) {
        const long n = a.nkv * ItemUnits(a, request<256>(a, b)).head();
        if (u0 < base + n) {
          shares.start[i] = ShareStart{u0, deal.first(v + 1) - u0, base, b};
          break;
        }
        base += n;
      }
    }
  }
  __syncthreads();
}
// The walk over a share (by a warp together).
__device__ __forceinline__ ChunkWalk walk_from(const Args& a, const ShareStart& s) {
  ChunkWalk w;
  w.u = s.u;
  w.left = s.left;
  w.b = s.b;
  if (s.left > 0) {
    w.r = request<256>(a, w.b);
    w.iu = ItemUnits(a, w.r);
    const long rest = s.u - s.base, head = w.iu.head();
    w.kvh = (int)Deal::div(rest, head);
    w.qt = w.iu.find(rest - w.kvh * head);
    w.at = (int)(rest - w.kvh * head - w.iu.before(w.qt));
  }
  return w;
}

// A piece of an item as the producer warp hands it to the others.
struct Piece {
  int s0, rows, len, p0;   // of the request
  int kvh, q;              // KV head, query tile
  int t0, t1;              // units; none: there are no more pieces
  int whole;               // all of the item's units
  int v;                   // the share
};
// Places for pieces. The ring of tiles lets the producer be at most six units, so
// six pieces, ahead of the MMA warp, the warps that look at values and the first
// tile; but not of the second tile's warps, which it does not hold back over pieces
// that have no queries for them. So the softmax warps say when they are done with a
// place (kPieceWarps of them), and the producer waits for that before it writes the
// place anew.
constexpr int kPieces = 16, kPieceWarps = 8, kChecks = 8;

// The join's descriptor of an item that begins in share v (one thread).
__device__ __forceinline__ void describe(const Args& a, const ChunkWalk& w, int v, const Shares& shares, bool whole) {
  const int c1 = whole ? v : shares.cta_of(w.u - w.t1 + w.nt - 1);
  const int4 d = make_int4(v, c1 - v + 1, w.b, w.item_h * w.r.ntq + w.item_q);
  if (!whole) a.desc[v] = d;
}
// None begins there that others share.
__device__ __forceinline__ void describe_none(const Args& a, int v) { a.desc[v] = make_int4(0, 0, 0, 0); }

// A wait ran out: every row of the CTA's pieces becomes NaN (one warp, which
// finds the pieces by itself).
template <int HD, typename TC>
__device__ __noinline__ void leave_nan(const Args& a, const Shares& shares) {
  const int lane = threadIdx.x & 31;
  const float nan = __int_as_float(0x7fc00000);
  for (int round = 0; round < shares.rounds; ++round) {
    ChunkWalk w = walk_from(a, shares.start[round]);
    const int v = blockIdx.x + round * gridDim.x;
    while (w.next(a)) {
      const bool whole = w.t0 == 0 && w.t1 == w.nt;
      if (lane == 0 && w.t0 == 0) describe(a, w, v, shares, whole);
      const long slot = 2l * v + (w.t0 == 0 ? 1 : 0);
      for (int i = lane; i < 256; i += 32) {
        const int q = w.item_q * 256 + i, j = q / a.group, hh = w.item_h * a.group + q - j * a.group;
        if (q >= w.r.rows * a.group) break;
        if (!whole) {
          a.part_ml[slot * a.mt_max + i] = make_float2(0.f, nan);
          continue;
        }
        TC* dst = static_cast<TC*>(a.out) + (w.r.s0 + j) * a.o_row + hh * a.o_head;
        for (int d = 0; d < HD; d += 2) *reinterpret_cast<uint32_t*>(dst + d) = Num<TC>::pack(nan, nan);
        if (a.lse) a.lse[(long)(w.r.s0 + j) * a.nq + hh] = nan;
      }
    }
    if (lane == 0 && !w.open) describe_none(a, v);
  }
  if (lane == 0)
    for (int round = shares.rounds; round < a.rounds; ++round) describe_none(a, blockIdx.x + round * gridDim.x);
  report_err(a.err, kErrWait);
}

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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// As wait, without a call (setmaxnreg's register counts allow none), for a
// converged warp; once a wait has run out (ok false) no further one is begun.
// The lanes do not vote on it: that would cost 100 cycles a wait. Whoever gave up
// goes on without waiting, to the end of the piece at least, but frees no tile any
// more (a copy into one that is on its way already may not be begun); the CTA's
// rows become NaN in the end. (The bound is an argument of the call, for a test
// that makes waits run out. As a constant: nine prompts 313 us, 297 so; 64 chunks of
// 200 rows at 64 dimensions 239 and 227.)
__device__ __forceinline__ void await(bool& ok, uint64_t* bar, uint32_t parity, uint32_t polls) {
  if (ok) ok = mbar_wait(bar, parity, polls);
  __syncwarp();
}

template <int HD, typename TC>
__global__ void __launch_bounds__(ChunkShape<HD, TC>::kThreads, 1) k_chunk_attn(const __grid_constant__ Args a) {
  using S = ChunkShape<HD, TC>;
  constexpr int NS = S::kStages, SL = S::kSlots;
  extern __shared__ unsigned char pa_smem_raw[];
  unsigned char* const qbuf = pa_smem_raw + ((1024 - (smem_u32(pa_smem_raw) & 1023)) & 1023);   // both tiles' queries
  unsigned char* const ring = qbuf + 2 * S::kTileBytes;
  __shared__ long sh_loc[2 * (S::kThreads / 32)];
  __shared__ Shares s_shares;
  // full: a tile of the ring has landed; empty: it may be loaded anew; checked: a unit's values may be used.
  __shared__ __align__(8) uint64_t full[NS], empty[NS], checked[kChecks], q_full[2], s_full[2], p_full[2][2], o_done[2], drain;
  __shared__ __align__(8) uint64_t piece_full[kPieces], piece_empty[kPieces];
  __shared__ Piece s_piece[kPieces];
  __shared__ int s_odd[kPieces];   // the first slot with a value that is no finite number, among those looked at
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_fail;   // a wait has run out
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < kChecks; ++i) mbar_init(&checked[i], 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 4);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x][0], 4);
      mbar_init(&p_full[x][1], 4);
      mbar_init(&o_done[x], 1);
    }
    mbar_init(&drain, 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], kPieceWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == 8 && lane < 2) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &a.vm : &a.km)) : "memory");
  }
  if (tid == 0) s_fail = 0;
  if (warp == 9) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_launch_next();
  chunk_walk<HD, TC>(a, sh_loc, s_shares);
  bool ok = true;
  // Piece i of the CTA, for the other warps; no units at the end. (A warp that has
  // given up sees the end.)
  auto piece_at = [&](int i) {
    await(ok, &piece_full[i % kPieces], i / kPieces & 1, a.polls);
    ok = __all_sync(0xffffffffu, ok);
    Piece p = s_piece[i % kPieces];
    if (!ok) p.t1 = p.t0 = 0, s_fail = 1;
    return p;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kOtherRegs));
    if (warp == 8) {
      // -------------------------------------------------------- producer warp
      const int bp = min(1 << a.shift, SL);           // slots of a box
      const int np = SL / bp;                         // boxes of a column
      const int bi = lane % np, h = lane / np;        // this lane's box of a tile: np * kHalf <= 16 lanes
      const uint32_t dst0 = smem_u32(ring) + h * S::kBox + bi * bp * 128;
      const uint64_t policy = policy_evict_normal();
      int win_b = -1, win = -1, entry = 0;            // the 32 table entries at hand, one per lane
      int s = 0, phase = 1, loaded = 0;               // (a new barrier's phase 1 counts as past)
      int piece = 0, round = -1;
      ChunkWalk w;
      w.left = 0;
      while (true) {
        const bool more = ok && w.next(a);
        if (ok && !more && round + 1 < s_shares.rounds) {        // (this share is done)
          if (lane == 0 && round >= 0 && !w.open) describe_none(a, blockIdx.x + round * gridDim.x);
          w = walk_from(a, s_shares.start[++round]);
          continue;
        }
        const int v = blockIdx.x + round * gridDim.x;
        // Its place (also to tell of an end because a wait ran out, unless this one does).
        const bool place = __all_sync(0xffffffffu, mbar_wait(&piece_empty[piece % kPieces], piece / kPieces & 1 ^ 1, a.polls));
        if (!place) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const bool whole = more && w.t0 == 0 && w.t1 == w.nt;
          s_odd[piece % kPieces] = INT32_MAX;
          s_piece[piece % kPieces] =
              more ? Piece{w.r.s0, w.r.rows, w.r.len, w.r.p0, w.item_h, w.item_q, w.t0, w.t1, whole, v} : Piece{};
          mbar_arrive(&piece_full[piece % kPieces]);
          if (more && w.t0 == 0) describe(a, w, v, s_shares, whole);
        }
        ++piece;
        if (!more) break;
        // Its queries towards L2: the softmax warps load them when they are done with the piece before.
        for (int i = lane; i < 256; i += 32) {
          const int q = w.item_q * 256 + i, j = q / a.group, hh = w.item_h * a.group + q - j * a.group;
          if (q < w.r.rows * a.group) {
            const TC* p = static_cast<const TC*>(a.q) + (w.r.s0 + j) * a.q_row + hh * a.q_head;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
            if (HD == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 64));
          }
        }
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const int first = (t * SL) >> a.shift;
          if (w.b != win_b || (first >> 5) != win) {
            win_b = w.b;
            win = first >> 5;
            const int e = 32 * win + lane;
            entry = e < a.W ? a.tables[(long)w.b * a.W + e] : -1;
          }
          const int left = w.r.len - t * SL;          // slots from here on
          const int nb = max(0, min(np, (left + bp - 1) / bp));
          const int page = __shfl_sync(0xffffffffu, entry, (first + bi) & 31);
          const int off = (t * SL) & ((1 << a.shift) - 1);
#pragma unroll
          for (int v = 0; v < 2; ++v) {               // keys, then values
            await(ok, &empty[s], phase, a.polls);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_expect_tx(&full[s], nb * bp * 128 * S::kHalf);
            __syncwarp();
            const int nhd = v ? a.v_nhd : a.k_nhd;
            if (h < S::kHalf && bi < nb)
              tma_load_4d(dst0 + s * S::kTileBytes, v ? &a.vm : &a.km, 64 * h, nhd ? w.item_h : off,
                          nhd ? off : w.item_h, page, &full[s], policy);
            ++loaded;
            if (++s == NS) s = 0, phase ^= 1;
          }
        }
      }
      if (lane == 0) {
        if (!w.open) describe_none(a, blockIdx.x + max(round, 0) * gridDim.x);
        for (int r = s_shares.rounds; r < a.rounds; ++r) describe_none(a, blockIdx.x + r * gridDim.x);
      }
      if (!ok) s_fail = 1;
      // The copies in flight land before the CTA may end, whatever the others did.
      for (int k = max(0, loaded - NS); k < loaded; ++k) mbar_wait(&full[k % NS], (k / NS) & 1, kWaitPolls);
    } else if (warp == 9) {
      // ------------------------------------------------------------- MMA warp
      // One lane does it all.
      if (elect_one()) {
        constexpr uint32_t id_s = tc_idesc<TC>(128, SL, false), id_o = tc_idesc<TC>(128, HD, true);
        const uint64_t dq = sw128_desc(smem_u32(qbuf)), dk = sw128_desc(smem_u32(ring));
        const uint64_t dv = sw128_desc_mn(smem_u32(ring), S::kBox);
        auto wait_for = [&](uint64_t* bar, uint32_t parity) {
          if (ok && !mbar_wait(bar, parity, 1)) ok = mbar_wait(bar, parity, a.polls);
          tc_fence_after();
        };
        // S of tile x with the keys in stage s; the last tile frees the stage (unless a wait has run out).
        auto scores = [&](int x, int s, bool last) {
          const uint64_t q = dq + (uint64_t)(x * (S::kTileBytes >> 4)), d = dk + (uint64_t)(s * (S::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint64_t o = ((k >> 2) * S::kBox + 32 * (k & 3)) >> 4;
            umma_bf16(tmem + S::kS + SL * x, q + o, d + o, id_s, k > 0);
          }
          umma_commit(&s_full[x]);
          if (last && ok) umma_commit(&empty[s]);
        };
        // O of tile x += P V for half h of the unit's slots, the values in stage s.
        auto output = [&](int x, int s, int h, uint32_t keep) {
          const uint64_t d = dv + (uint64_t)(s * (S::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < SL / 32; ++k) {
            const int kk = h * (SL / 32) + k;
            umma_bf16_tmem_a(tmem + S::kO + HD * x, tmem + S::kS + SL * x + 8 * kk, d + (2048 * kk >> 4), id_o,
                             kk > 0 ? 1u : keep);
          }
        };
        int s = 0, phase = 0, n = 0;                    // stage, units
        uint32_t piece[2] = {0, 0}, done[2] = {0, 0};   // parities of each tile's next piece and unit
        auto advance = [&] { if (++s == NS) s = 0, phase ^= 1; };
        for (int i = 0;; ++i) {
          wait_for(&piece_full[i % kPieces], i / kPieces & 1);
          if (!ok) break;
          const Piece w = s_piece[i % kPieces];
          const int units = w.t1 - w.t0;
          if (units == 0) break;
          const int tiles = w.rows * a.group - w.q * 256 > 128 ? 2 : 1;
          wait_for(&full[s], phase);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x == tiles) break;
            wait_for(&q_full[x], piece[x]);
            piece[x] ^= 1;
            scores(x, s, x == tiles - 1);
          }
          advance();
          for (int u = 0; u < units; ++u, ++n) {
            const int sv = s;
            const bool more = u + 1 < units;
            advance();
            wait_for(&checked[n % kChecks], n / kChecks & 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x == tiles) break;
              const bool last = x == tiles - 1;
              wait_for(&p_full[x][0], done[x]);
              output(x, sv, 0, u % S::kFold ? 1u : 0u);
              wait_for(&p_full[x][1], done[x]);
              done[x] ^= 1;
              output(x, sv, 1, 1u);
              if (last && ok) umma_commit(&empty[sv]);
              if (more) {
                if (x == 0) wait_for(&full[s], phase);
                scores(x, s, last);
              } else {
                umma_commit(&o_done[x]);
              }
            }
            if (more) advance();
          }
        }
        if (!ok) s_fail = 1;
        // What was issued ends before the CTA does, also when a wait has run out.
        umma_commit(&drain);
        mbar_wait(&drain, 0, kWaitPolls);
      }
      __syncwarp();
    } else {
      // ------------------------------------------- warps that look at values
      constexpr int PP = HD / 8;                      // 16-byte pieces of a slot
      constexpr uint32_t X = Num<TC>::kExp;
      const int me = tid - 320;                       // 0 .. 63
      int s = 1, phase = 0, n = 0;                    // (keys in one stage, values in the next)
      for (int piece = 0;; ++piece) {
        const Piece w = piece_at(piece);
        if (w.t1 == 0) break;
        // From slot `seen` on some row of the item does not see a slot.
        const int seen = w.p0 + w.q * 256 / a.group + 1;
        for (int t = w.t0; t < w.t1; ++t, ++n) {
          await(ok, &full[s], phase, a.polls);
          const int s0 = min(max(seen - t * SL, 0), SL), s1 = min(max(w.len - t * SL, 0), SL);
          if (s0 < SL) {
            unsigned char* vs = ring + s * S::kTileBytes;
            auto at = [&](int sl, int p) {            // in any order within a slot
              return reinterpret_cast<uint4*>(vs + (p >> 3) * S::kBox + sl * 128 + (p & 7) * 16);
            };
            auto bad = [](uint32_t v) { return (v & X) == X || (v >> 16 & X) == X; };
            auto clean = [](uint32_t v) { return ((v & X) == X ? 0u : v & 0xffffu) | ((v >> 16 & X) == X ? 0u : v & 0xffff0000u); };
            // Zero times each, added up: NaN if one of them is no finite number (two
            // elements an instruction; looking at every exponent took nine whole
            // prompts at the 7B shape 354 us, 319 so).
            using T2 = typename std::conditional<std::is_same<TC, bf16>::value, __nv_bfloat162, __half2>::type;
            const uint32_t zero = 0;
            const T2 none = *reinterpret_cast<const T2*>(&zero);
            T2 sum[4] = {none, none, none, none};
#pragma unroll 8
            for (int e = s0 * PP + me; e < SL * PP; e += 64) {
              const uint4 v = *at(e / PP, e % PP);
              sum[0] = __hfma2(*reinterpret_cast<const T2*>(&v.x), none, sum[0]);
              sum[1] = __hfma2(*reinterpret_cast<const T2*>(&v.y), none, sum[1]);
              sum[2] = __hfma2(*reinterpret_cast<const T2*>(&v.z), none, sum[2]);
              sum[3] = __hfma2(*reinterpret_cast<const T2*>(&v.w), none, sum[3]);
            }
            const T2 both = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
            const float total = __low2float(both) + __high2float(both);
            if (total != total) {
              int odd = INT32_MAX;
              for (int e = s0 * PP + me; e < SL * PP; e += 64) {
                uint4* const p = at(e / PP, e % PP);
                const uint4 v = *p;
                if (bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w)) {
                  *p = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
                  if (e / PP < s1) odd = min(odd, t * SL + e / PP);
                }
              }
              if (odd != INT32_MAX) atomicMin(&s_odd[piece % kPieces], odd);
              fence_proxy_async();
            }
          }
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&checked[n % kChecks]);
          s += 2;
          if (s >= NS) s -= NS, phase ^= 1;
        }
      }
      if (!ok) s_fail = 1;
    }
  } else {
    // ----------------------------------------------------------- softmax warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
    const int x = warp >> 2, row = tid & 127;                 // the tile, and the query of it = tensor-memory lane
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_s = lanes + S::kS + SL * x, t_o = lanes + S::kO + HD * x;
    unsigned char* const qs = qbuf + x * S::kTileBytes;
    int n = 0, my_pieces = 0;                                 // units and pieces of this tile
    auto s_wait = [&] {
      await(ok, &s_full[x], n & 1, a.polls);
      tc_fence_after();
    };
    // The piece's queries into shared memory (rows past the end: zeros).
    auto load_queries = [&](const Piece& w) {
      constexpr int PP = HD / 8, RW = 32 / PP;                // pieces of a row, rows of a load
      constexpr long kNone = INT64_MIN;
      const int q = w.q * 256 + 128 * x + row, j = q / a.group, hh = w.kvh * a.group + q - j * a.group;
      const long off = q < w.rows * a.group ? (w.s0 + j) * a.q_row + hh * a.q_head : kNone;
      const int p = lane % PP;
      uint4 f[32 / RW];                                       // (all on their way together)
#pragma unroll
      for (int i = 0; i < 32 / RW; ++i) {
        const long o = __shfl_sync(0xffffffffu, off, RW * i + lane / PP);
        f[i] = make_uint4(0u, 0u, 0u, 0u);
        if (o != kNone) f[i] = *reinterpret_cast<const uint4*>(static_cast<const TC*>(a.q) + o + 8 * p);
      }
#pragma unroll
      for (int i = 0; i < 32 / RW; ++i) {
        f[i].x ^= a.flip, f[i].y ^= a.flip, f[i].z ^= a.flip, f[i].w ^= a.flip;
        const int r = 32 * (warp & 3) + RW * i + lane / PP;
        *reinterpret_cast<uint4*>(qs + (p >> 3) * S::kBox + r * 128 + (((p & 7) ^ (r & 7)) << 4)) = f[i];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
    };
    // The warp is done with piece i's place, its first odd slot among it.
    auto release = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[i % kPieces]);
    };
    // The next piece with queries for this tile, its queries on their way.
    int i = 0;
    auto next_piece = [&] {
      while (true) {
        const Piece p = piece_at(i);
        if (p.t1 == 0) return p;
        if (p.rows * a.group - p.q * 256 > 128 * x) {
          load_queries(p);
          return p;
        }
        release(i);
        ++i;
      }
    };
    for (Piece w = next_piece(); w.t1 != 0;) {
      const int q = w.q * 256 + 128 * x + row, j = q / a.group, hh = w.kvh * a.group + q - j * a.group;
      const int Mq = w.rows * a.group;
      const bool live = q < Mq, warp_live = (q & ~31) < Mq;
      const int out_row = w.s0 + j;
      const int lim = live ? w.p0 + j + 1 : INT32_MAX;      // slots that the row sees (0 .. lim - 1)
      const int lim_warp = __shfl_sync(0xffffffffu, lim, 0);  // (the least: rows see more and more)
      const int t0 = w.t0, t1 = w.t1;
      const bool whole = w.whole;
      const long slot = 2l * w.v + (t0 == 0 ? 1 : 0);
      float* const part = a.part + (slot * a.mt_max + 128 * x + row) * HD;     // (of a live row)
      float2* const part_ml = a.part_ml + slot * a.mt_max + 128 * x + row;
      float m = -INFINITY, l = 0.f;
      bool folded = false;                                    // the part holds sums
      auto unit = [&](int t) {
        s_wait();
        if (warp_live) {
          uint32_t v[SL];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, v + 32 * c);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < SL; ++i) asm volatile("" : "+r"(v[i]));   // (read behind the wait only)
          // ---- what the row does not see is -infinity
          if ((t + 1) * SL > lim_warp) {
            const int vis = lim - t * SL;
#pragma unroll
            for (int i = 0; i < SL; ++i)
              if (i >= vis) v[i] = 0xff800000u;
          }
          // ---- maximum; a new reference when it has outgrown the old one
          float mx4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 4]));
#pragma unroll
          for (int i = 8; i < SL; i += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) mx4[y] = fmaxf(fmaxf(mx4[y], __uint_as_float(v[i + y])), __uint_as_float(v[i + y + 4]));
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const bool grow = m != -INFINITY && (mx - m) * a.scale2 > (float)S::kLag;
          if (__any_sync(0xffffffffu, grow)) {                // (each row by itself: its result does not depend on the others)
            const float f = grow ? exp2_approx((m - mx) * a.scale2) : 1.f;
            if (grow) m = mx;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(t_o + 16 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                asm volatile("" : "+r"(o[i]));
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              }
              tmem_st16(t_o + 16 * c, o);
            }
            tmem_st_wait();
          }
          if (m == -INFINITY) m = mx;                         // (what came before saw nothing: O is 0)
          const float ref = m == -INFINITY ? 0.f : fmaf(-m, a.scale2, (float)S::kUp);
          const uint64_t sc2 = pair(a.scale2, a.scale2), ref2 = pair(ref, ref);
          uint64_t l2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = 64 * c + 2 * i;
              const float2 y = unpair(fma2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, ref2));
              const float p0 = exp2_approx(y.x), p1 = exp2_approx(y.y);
              l2[i & 3] = add2(l2[i & 3], pair(p0, p1));
              p[i] = Num<TC>::pack(p0, p1);
            }
            tmem_st32(t_s + 32 * c, p);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x][c]);        // (the product with one half runs beside the other's exponentials)
          }
          const float2 ls = unpair(add2(add2(l2[0], l2[1]), add2(l2[2], l2[3])));
          l += ls.x + ls.y;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane < 2) mbar_arrive(&p_full[x][lane]);
        }
        ++n;
      };
      // Between two units: O and l move to the part (`first`: which holds
      // nothing yet), whose reference may be an older maximum.
      auto fold = [&](bool first) {
        s_wait();   // (the next unit's scores lie behind the last output)
        const float2 ml = live && !first ? *part_ml : make_float2(-INFINITY, 0.f);
        const float f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m) * a.scale2);
        if (live) *part_ml = make_float2(m, fmaf(ml.y, f, l));
        l = 0.f;
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(t_o + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(o[i]));
            if (live) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                float4* const p = reinterpret_cast<float4*>(part + 16 * c + i);
                const float4 y = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
                *p = make_float4(fmaf(y.x, f, __uint_as_float(o[i])), fmaf(y.y, f, __uint_as_float(o[i + 1])),
                                 fmaf(y.z, f, __uint_as_float(o[i + 2])), fmaf(y.w, f, __uint_as_float(o[i + 3])));
              }
            }
            __syncwarp();
          }
        }
      };
#pragma unroll 1
      for (int t = t0; t < t1; ++t) {
        if ((t - t0) % S::kFold == 0 && t > t0) {
          fold(!folded);
          folded = true;
        }
        unit(t);
      }
      // ---- O is there, and all that is to be known of the piece; only then is the
      // next one looked for, over any number of pieces that other tiles have alone.
      // (Its queries go where this one's were, whose scores have been read. Loaded
      // before the wait, with the search behind it: 322 us for nine prompts, 315 so.)
      await(ok, &o_done[x], my_pieces & 1, a.polls);
      tc_fence_after();
      ++my_pieces;
      const int odd = s_odd[i % kPieces];
      release(i++);
      w = next_piece();
      float f = 0.f;                                          // of what lies in the part
      if (folded && live) {
        const float2 ml = *part_ml;
        f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m) * a.scale2);
        l = fmaf(ml.y, f, l);
      }
      if (odd < lim) l = __int_as_float(0x7fc00000);   // the row sees a value that is no number: NaN
      if (m != -INFINITY) m = fmaf(m, a.scale2, (float)-S::kUp);
      if (warp_live) {
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        // 128 bytes of each row (32 words a lane, its row's) through shared
        // memory, so that a store is four rows' 128 bytes (a lane's own row at a
        // time would be 32 rows' 16 bytes: items' ends took 4 us).
        unsigned char* const sw = ring + NS * S::kTileBytes + warp * S::kStaging;
        char* const dst = !live ? nullptr
                          : whole ? reinterpret_cast<char*>(static_cast<TC*>(a.out) + out_row * a.o_row + hh * a.o_head)
                                  : reinterpret_cast<char*>(part);
        auto put = [&](const uint32_t* y, int at) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(sw + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), k = lane & 7;
            char* const d = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
            const uint4 v = *reinterpret_cast<const uint4*>(sw + r * 128 + ((k ^ (r & 7)) << 4));
            if (d) *reinterpret_cast<uint4*>(d + at + 16 * k) = v;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < HD / 64; ++c) {
          uint32_t o[64];
          __syncwarp();
          tmem_ld32(t_o + 64 * c, o);
          tmem_ld32(t_o + 64 * c + 32, o + 32);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(o[i]));
          if (folded && live) {
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const float4 y = *reinterpret_cast<const float4*>(part + 64 * c + i);
              o[i] = __float_as_uint(fmaf(y.x, f, __uint_as_float(o[i])));
              o[i + 1] = __float_as_uint(fmaf(y.y, f, __uint_as_float(o[i + 1])));
              o[i + 2] = __float_as_uint(fmaf(y.z, f, __uint_as_float(o[i + 2])));
              o[i + 3] = __float_as_uint(fmaf(y.w, f, __uint_as_float(o[i + 3])));
            }
          }
          // (a row that saw nothing: l = 0 and O = 0)
          if (whole) {
            uint32_t y[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              y[i] = Num<TC>::pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            put(y, 128 * c);
          } else {
            put(o, 256 * c);
            put(o + 32, 256 * c + 128);
          }
        }
        if (live && whole && a.lse)
          a.lse[(long)out_row * a.nq + hh] = l == 0.f ? -INFINITY : m * 0.693147180559945f + logf(l);
        if (live && !whole) *part_ml = make_float2(m, l);
      }
      tc_fence_before();   // O has been read: the next piece's first product may replace it
    }
    if (!ok) s_fail = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (warp == 0 && s_fail) leave_nan<HD, TC>(a, s_shares);
}

// The join of the items that several CTAs share: the parts lie with the CTAs
// first .. first + count - 1, and every CTA that one begins in has a descriptor.
// A warp takes two queries of an item (a lane HD / 32 dimensions), four parts on
// their way, so that nearly all of an item's CTAs are there at once: 6 us after nine
// whole prompts at the 7B shape, 21 with a warp and a launched CTA for every item's
// every query. Few items have many parts each: 30 rows of 16384 tokens, 28 / 4
// heads of 128, the call 35 us, with four queries a warp and two parts 54, with one and eight
// 32 (but nine prompts 300 for 296).
constexpr int kChunkJoinThreads = 256, kChunkJoinQueries = 2 * kChunkJoinThreads / 32;
template <int HD, typename TC>
__global__ void __launch_bounds__(kChunkJoinThreads) k_chunk_join(const __grid_constant__ Args a) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31, x0 = blockIdx.y * kChunkJoinQueries + (threadIdx.x >> 5) * 2;
  pdl_launch_next();
  pdl_wait();   // (before any return: what follows the join relies on the main kernel's end as well)
  const int4 d = a.desc[blockIdx.x];
  if (d.y < 2) return;
  const Request r = request<256>(a, d.z);
  const int kvh = d.w / r.ntq, qt = d.w - kvh * r.ntq, Mq = r.rows * a.group;
  if (qt * 256 + x0 >= Mq) return;
  float m[2], l[2], o[2][V];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) o[i][e] = 0.f;
  }
#pragma unroll 4
  for (int k = 0; k < d.y; ++k) {
    const long slot = (2l * (d.x + k) + (k == 0 ? 1 : 0)) * a.mt_max + x0;
    float2 ml[2];
    float v[2][V];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
      if (qt * 256 + x0 + i < Mq) {
        ml[i] = a.part_ml[slot + i];
        const float* p = a.part + (slot + i) * HD + V * lane;
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(p);
          v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(p);
          v[i][0] = f.x, v[i][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mm = fmaxf(m[i], ml[i].x);
      const float f0 = m[i] == -INFINITY ? 0.f : exp2_approx(m[i] - mm), f1 = ml[i].x == -INFINITY ? 0.f : exp2_approx(ml[i].x - mm);
      // (a part that saw nothing has sum 0, one whose row sees a value that is no number NaN)
      l[i] = (m[i] == -INFINITY || l[i] != l[i] ? l[i] : l[i] * f0) + (ml[i].x == -INFINITY || ml[i].y != ml[i].y ? ml[i].y : ml[i].y * f1);
      m[i] = mm;
#pragma unroll
      for (int e = 0; e < V; ++e) o[i][e] = fmaf(v[i][e], f1, o[i][e] * f0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int q = qt * 256 + x0 + i;
    if (q >= Mq) return;
    const int j = q / a.group, hh = kvh * a.group + q - j * a.group;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    TC* dst = static_cast<TC*>(a.out) + (r.s0 + j) * a.o_row + hh * a.o_head + V * lane;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(Num<TC>::pack(o[i][0] * inv, o[i][1] * inv), Num<TC>::pack(o[i][2] * inv, o[i][3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = Num<TC>::pack(o[i][0] * inv, o[i][1] * inv);
    if (a.lse && lane == 0) a.lse[(long)(r.s0 + j) * a.nq + hh] = l[i] == 0.f ? -INFINITY : m[i] * 0.693147180559945f + logf(l[i]);
  }
}

}  // namespace pa
}  // namespace sf
