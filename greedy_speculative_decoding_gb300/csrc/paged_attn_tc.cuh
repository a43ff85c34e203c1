// Paged attention for many queries per KV head (several rows times the query
// heads that share the KV head), on the tcgen05 tensor cores: tiles of 128
// queries. The work is dealt out as in paged_attn.cuh; beside the producer warp
// a CTA has
//   * an MMA warp: S = Q K^T (128 x 64) and O += P V, queries, probabilities
//     and both accumulators in tensor memory, keys and values in shared memory
//     (the values with the slots as the MMA's K side). Queries in shared memory
//     took all its bandwidth during S. The scores of a unit come behind the
//     output of the one two before, whose S and P they replace: a unit's scores
//     there means that output complete;
//   * four softmax warps, a thread per query row: row maximum and sum without
//     shuffles. O is rescaled only when a row's maximum has grown by more than
//     2^kLag since its reference was set, so seldom after the first unit.
//     Probabilities of 16-bit queries are rounded to the cache's type, by half a
//     step each; with a lagging reference that includes the largest, which is
//     exactly a power of two in the mma.sync kernel. bf16 has the range for a
//     lag of 2^8; fp16 probabilities are taken times 2^12 and may lag by 2^3, so
//     that the largest stay below 2^15 and those down to 2^-26 of it keep their
//     bits (the others are off by 2^-37 of it at most).
//   * fp32 queries and their probabilities are three bf16 terms each (24 bits:
//     exact), so three products in place of one, the small terms first. The
//     tensor cores cut off what they add to the output (54 units of 12 products
//     left it 8e-6 too small), so it moves every 16 units to sums in shared
//     memory that are rounded (of 16-bit queries every 256 units).
//
// mma.sync reaches 590 TFLOP/s on this GPU (measured, four or more warps an
// SM); the 45 queries of a 9-row verify with 5 heads per KV head, padded to 48,
// need 430 of them to keep up with the cache's bytes, 128 queries 1150. A unit
// takes 1.07 thousand cycles here (600 the softmax warps' arithmetic: 64
// exponentials a thread are 512 cycles of an SM quarter's unit; the rest
// waits and hand-overs), its bytes 1.4 thousand at head dimension 128. Eight
// sequences of 4096 to 8192 tokens, head_dim 128, 128 queries: 48 us (530
// TFLOP/s; mma.sync in tiles of 32: 126 us), in fp16 51, as its references are
// raised more often; 45 queries: 41 us (67). With fp32 queries 75 us (mma.sync
// in tiles of 16: 236 us) and 67 us (94): the products are 1.6 thousand cycles a
// unit there, the terms of the probabilities nearly as many again in the softmax
// warps, behind the products; the sums' 4 us are the price of an error of 3e-6.
#pragma once

#include "paged_attn.cuh"

namespace sf {
namespace pa {

template <int HD, typename TC, bool F32>
struct TcShape {
  static constexpr int MT = 128;
  static constexpr int kThreads = 192;                 // 4 softmax warps, producer, MMA
  static constexpr int kHalf = HD / 64;
  static constexpr int kBox = kTile * 128;
  static constexpr int kStage = 2 * kHalf * kBox;
  // Tensor-memory columns (32 bits): O, two S (P of a unit over its S), the
  // queries; fp32 queries and probabilities as three 16-bit terms. At head
  // dimension 64 two CTAs share an SM where that fits (the softmax of one alone
  // takes longer than its units' bytes).
  static constexpr int kLag = std::is_same<TC, __half>::value ? 3 : 8;   // (in powers of two, as kUp)
  static constexpr int kUp = std::is_same<TC, __half>::value ? 12 : 0;
  static constexpr int kTerms = F32 ? 3 : 1;
  static constexpr int kSCols = F32 ? 96 : 64;           // of S (64), then of P (32 a term)
  static constexpr int kO = 0, kS = HD, kQ = HD + 2 * kSCols;
  static constexpr int kQTerm = HD / 2;
  static constexpr int kCtas = HD == 64 && !F32 ? 2 : 1, kCols = 512 / kCtas;
  // Units after which O moves to the sums. Of 16-bit queries the sums are the
  // piece's place in the workspace (over 2^20 slots in one CTA outputs were 0.5%
  // too small without). With fp32 queries the call says after how many (Args::fold).
  static constexpr int kFold = 256;
  static constexpr int kSums = F32 ? MT * HD * 4 : 0;
  static constexpr int kStages = !F32 ? 6 : HD == 64 ? 10 : 4;
  static constexpr int kSmem = 1024 + kStages * kStage + kSums;
  // (as in paged_attn.cuh: 64 sequences of 100 to 2000 tokens, 8 KV heads, 45
  // queries: 64.8 us, 93.2 with none, 71.8 with 4, 68.3 with 14)
  static constexpr int kPiece = 8;
  static_assert(kQ + kTerms * kQTerm <= kCols, "tensor memory");
};

// B operand with the slots as K: rows of 128 bytes are 64 dimensions of one
// slot (the MN side contiguous), 8 slots to a 1024-byte swizzle atom. Leading
// offset: from 64 dimensions to the next 64 (one box); stride: from 8 slots to
// the next 8.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t saddr, uint32_t box_bytes) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(box_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

template <typename TC>
__host__ __device__ constexpr uint32_t tc_idesc(int M, int N, bool b_mn) {
  const uint32_t fmt = std::is_same<TC, bf16>::value ? 1 : 0;   // operand type: bf16 or fp16
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// 64 fp32 values as three 16-bit terms, the largest first, into tensor-memory
// columns `pitch` apart (the values become the rest, about 2^-24 of them).
template <int PITCH, typename TC>
__device__ __forceinline__ void put_terms(uint32_t taddr, float (&x)[64]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      p[i] = Num<TC>::pack(x[2 * i], x[2 * i + 1]);
      x[2 * i] -= Num<TC>::lo(p[i]);
      x[2 * i + 1] -= Num<TC>::hi(p[i]);
    }
    tmem_st32(taddr + PITCH * k, p);
  }
}

// TC: the cache's type. F32: fp32 queries and output over a bf16 cache.
template <int HD, typename TC, bool F32>
__global__ void __launch_bounds__(TcShape<HD, TC, F32>::kThreads, TcShape<HD, TC, F32>::kCtas)
    k_paged_attn_tc(const __grid_constant__ Args a) {
  using S = TcShape<HD, TC, F32>;
  using TQ = typename std::conditional<F32, float, TC>::type;
  constexpr int MT = S::MT;
  extern __shared__ unsigned char pa_smem_raw[];
  unsigned char* ring = pa_smem_raw + ((1024 - (smem_u32(pa_smem_raw) & 1023)) & 1023);
  __shared__ long sh_loc[S::kThreads / 32 + 2];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], s_full[2], p_full[2], o_done[2], q_full, drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_keep[2];     // the unit adds to what the softmax put into O (see odd values)
  __shared__ float s_sum[F32 ? MT : 1];   // the part of l that goes with the sums
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 4);
      mbar_init(&o_done[b], 1);
      s_keep[b] = 0;
    }
    mbar_init(&q_full, 4);
    mbar_init(&drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == 4 && lane < 2) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &a.vm : &a.km)) : "memory");
  }
  if (warp == 5) {
    tmem_alloc(&s_tmem, S::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_wait();
  pdl_launch_next();
  const Start st = a.by_warp ? locate_warp<MT>(a) : locate_cta<MT, S::kThreads>(a, sh_loc);
  const long G = min((long)gridDim.x, st.T);
  const bool idle = (long)blockIdx.x >= G;
  const Deal deal(max(st.T, 1l), max(G, 1l));
  const long u0 = deal.first(blockIdx.x), u1 = idle ? u0 : deal.first(blockIdx.x + 1);
  Walk<MT> w(st, u0, u1);
  bool ok = true;

  if (warp == 4) {
    // ---------------------------------------------------------- producer warp
    produce<S::kStages, S::kHalf, S::kBox, S::kStage, MT>(a, w, ring, full, empty, ok);
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA warp
    // The whole warp runs the loop and one lane issues: control flow and
    // descriptors are the same in all lanes, and the shuffles and votes say so
    // to the compiler, which then keeps the descriptors in uniform registers
    // (moving them there for every MMA took 100 cycles an MMA).
    constexpr uint32_t id_s = tc_idesc<TC>(MT, kTile, false), id_o = tc_idesc<TC>(MT, HD, true);
    const uint32_t utmem = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk = sw128_desc(__shfl_sync(0xffffffffu, smem_u32(ring), 0));
    const uint64_t dv = sw128_desc_mn(__shfl_sync(0xffffffffu, smem_u32(ring) + S::kHalf * S::kBox, 0), S::kBox);
    bool good = true;
    auto await = [&](uint64_t* bar, uint32_t parity) {
      if (good) good = __all_sync(0xffffffffu, wait(bar, parity));
    };
    auto scores = [&](int n) {   // S of unit n
      const int s = n % S::kStages;
      await(&full[s], (n / S::kStages) & 1);
      tc_fence_after();
      const uint64_t d = dk + (uint64_t)(s * (S::kStage >> 4));
      const uint32_t t = utmem + S::kS + S::kSCols * (n & 1);
      if (elect_one()) {
#pragma unroll
        for (int i = S::kTerms - 1; i >= 0; --i)   // the small terms first
#pragma unroll
          for (int k = 0; k < HD / 16; ++k)
            umma_bf16_tmem_a(t, utmem + S::kQ + S::kQTerm * i + 8 * k,
                             d + (((k >> 2) * S::kBox + 32 * (k & 3)) >> 4), id_s, i < S::kTerms - 1 || k > 0);
        umma_commit(&s_full[n & 1]);
      }
      __syncwarp();
    };
    int n = 0, piece = 0;
    while (__shfl_sync(0xffffffffu, (int)(good && w.next(a)), 0)) {
      const int units = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0);
      await(&q_full, piece++ & 1);
      tc_fence_after();
      scores(n);   // (both S are free: the units before have handed over their P)
      if (units > 1) scores(n + 1);
      for (int u = 0; u < units; ++u, ++n) {
        await(&p_full[n & 1], (n >> 1) & 1);
        if (!good) break;
        tc_fence_after();
        const uint32_t keep = (F32 ? u & (a.fold - 1) : u % S::kFold) ? 1u : (uint32_t)__shfl_sync(0xffffffffu, s_keep[n & 1], 0);
        const uint64_t d = dv + (uint64_t)(n % S::kStages * (S::kStage >> 4));
        const uint32_t t = utmem + S::kS + S::kSCols * (n & 1);
        if (elect_one()) {
#pragma unroll
          for (int i = S::kTerms - 1; i >= 0; --i)
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              umma_bf16_tmem_a(utmem + S::kO, t + 32 * i + 8 * k, d + (2048 * k >> 4), id_o,
                               i < S::kTerms - 1 || k > 0 ? 1u : keep);
          umma_commit(&empty[n % S::kStages]);
          umma_commit(&o_done[n & 1]);
        }
        __syncwarp();
        if (u + 2 < units) scores(n + 2);
      }
    }
    if (!good) {   // an expired wait: what was issued ends before the CTA does
      if (elect_one()) umma_commit(&drain);
      wait(&drain, 0);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- softmax warps
    const int row = tid;                                  // query of the tile = tensor-memory lane
    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    float4* const sums = reinterpret_cast<float4*>(ring + S::kStages * S::kStage) + row;   // (128 apart)
    auto sync4 = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    int n = 0;
    // Waits for unit k's output, k the unit before the one at hand. (Two
    // barriers in turn: at that point the barrier is in unit k's phase or the
    // next, never further, so that the parity tells.)
    auto o_wait = [&](int k) {
      if (ok && !wait(&o_done[k & 1], (k >> 1) & 1)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    };
    while (w.next(a)) {
      const Request r = w.r;
      const int Mq = r.rows * a.group;
      const int q = w.qt * MT + row, j = q / a.group, hh = w.kvh * a.group + q - j * a.group;
      const bool live = q < Mq, warp_live = w.qt * MT + 32 * warp < Mq;
      const unsigned long long bits = a.mask && live ? a.mask[r.s0 + j] : 0;
      // The row's query (rows past the end: zeros).
      if (warp_live) {
        const TQ* src = static_cast<const TQ*>(a.q) + (r.s0 + j) * a.q_row + hh * a.q_head;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          constexpr int W = 16 * sizeof(TQ);              // 32-bit words of 64 dimensions
          uint32_t v[W];
#pragma unroll
          for (int i = 0; i < W / 4; ++i) {
            uint4 f = make_uint4(0u, 0u, 0u, 0u);
            if (live) f = *reinterpret_cast<const uint4*>(src + 64 * c + (64 * 4 / W) * i);
            v[4 * i] = f.x ^ a.flip, v[4 * i + 1] = f.y ^ a.flip, v[4 * i + 2] = f.z ^ a.flip, v[4 * i + 3] = f.w ^ a.flip;
          }
          __syncwarp();
          if constexpr (F32) {
            float x[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] = __uint_as_float(v[i]);
            put_terms<S::kQTerm, TC>(lanes + S::kQ + 32 * c, x);
          } else {
            tmem_st32(lanes + S::kQ + 32 * c, v);
          }
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full);
      float m = -INFINITY, l = 0.f;
      bool folded = false;                                // the sums hold a part of O
      if constexpr (F32) s_sum[row] = 0.f;
      const long slot = 2l * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      float* const part = a.part + (slot * a.mt_max + row) * HD;     // (of a live row)
      float2* const part_ml = a.part_ml + slot * a.mt_max + row;
      // 16-bit queries, between two units: O and l move to the part (`first`:
      // which holds nothing yet), whose reference may be an older maximum.
      auto fold = [&](bool first) {
        o_wait(n - 1);
        const float2 ml = live && !first ? *part_ml : make_float2(-INFINITY, 0.f);
        const float f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m) * a.scale2);
        if (live) *part_ml = make_float2(m, fmaf(ml.y, f, l));
        l = 0.f;
        if (warp_live) {
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t v[16];
            tmem_ld16(lanes + S::kO + 16 * c, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
            if (live) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                float4* const p = reinterpret_cast<float4*>(part + 16 * c + i);
                const float4 y = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
                *p = make_float4(fmaf(y.x, f, __uint_as_float(v[i])), fmaf(y.y, f, __uint_as_float(v[i + 1])),
                                 fmaf(y.z, f, __uint_as_float(v[i + 2])), fmaf(y.w, f, __uint_as_float(v[i + 3])));
              }
            }
            __syncwarp();
          }
        }
      };
      // One unit: every row sees all slots of a plain one; a tail unit holds
      // slots of the pass itself, or slots past the end. (Apart, so that the
      // plain units' loop is short straight code.)
      auto unit = [&](auto kind, int t) {
        constexpr bool TAIL = decltype(kind)::value;
        const int b = n & 1;
        if (ok && !wait(&s_full[b], (n >> 1) & 1)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        float x[kTile];
        if (warp_live) {
          uint32_t v[4][16];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld16(lanes + S::kS + S::kSCols * b + 16 * c, v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kTile; ++i) {
            asm volatile("" : "+r"(v[i >> 4][i & 15]));   // (read behind the wait only)
            x[i] = __uint_as_float(v[i >> 4][i & 15]);
          }
        }
        // ---- what the row does not see is -infinity
        unsigned long long vis = ~0ull;
        if constexpr (TAIL) {
          const int first = r.p0 - t * kTile;             // the pass's first slot, within the unit
          auto low = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1; };
          vis = low(first + j + 1);
          if (a.mask) vis = low(first) | (first >= 64 || first <= -64 ? 0ull : first >= 0 ? bits << first : bits >> -first);
          vis = live ? vis & low(r.len - t * kTile) : 0ull;
          if (warp_live) {
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (!((i < 32 ? (uint32_t)vis : (uint32_t)(vis >> 32)) >> (i & 31) & 1)) x[i] = -INFINITY;
          }
        }
        if (warp_live) {
          // ---- maximum; a new reference when it has outgrown the old one
          float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i < kTile; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], x[i]);
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          const bool grow = m != -INFINITY && (mx - m) * a.scale2 > (float)S::kLag;
          if (__any_sync(0xffffffffu, grow)) {            // (then for every row whose maximum is a new one)
            const bool raise = m != -INFINITY && mx > m;
            const float f = raise ? exp2_approx((m - mx) * a.scale2) : 1.f;
            if (raise) m = mx;
            l *= f;
            o_wait(n - 1);   // (never at the piece's first unit: m was -infinity)
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              uint32_t v[16];
              tmem_ld16(lanes + S::kO + 16 * c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                asm volatile("" : "+r"(v[i]));
                v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              }
              tmem_st16(lanes + S::kO + 16 * c, v);
            }
            tmem_st_wait();
            if (F32 && folded) {
              s_sum[row] *= f;
#pragma unroll 4
              for (int c = 0; c < HD / 4; ++c) {
                const float4 y = sums[128 * c];
                sums[128 * c] = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
              }
            }
          }
          if (m == -INFINITY) m = mx;                     // (what came before saw nothing: O is 0)
          const float ref = m == -INFINITY ? 0.f : fmaf(-m, a.scale2, (float)S::kUp);
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kTile; ++i) {
            x[i] = exp2_approx(fmaf(x[i], a.scale2, ref));
            l4[i & 3] += x[i];
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        }
        // ---- O starts anew with the piece and after moving to the sums
        const bool fresh = (F32 ? (t - w.t0) & (a.fold - 1) : (t - w.t0) % S::kFold) == 0;
        if constexpr (F32) {
          if (fresh && t > w.t0) {
            o_wait(n - 1);
            if (warp_live) {
#pragma unroll 1
              for (int c = 0; c < HD / 16; ++c) {
                uint32_t v[16];
                tmem_ld16(lanes + S::kO + 16 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                  asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]));
                  float4* const p = sums + 128 * (4 * c + i / 4);
                  const float4 y = folded ? *p : make_float4(0.f, 0.f, 0.f, 0.f);
                  *p = make_float4(y.x + __uint_as_float(v[i]), y.y + __uint_as_float(v[i + 1]),
                                   y.z + __uint_as_float(v[i + 2]), y.w + __uint_as_float(v[i + 3]));
                }
              }
            }
            folded = true;
            s_sum[row] += l;
            l = 0.f;
          }
        }
        // ---- values of a tail unit: slots past the end become 0; values of
        // the pass that are no finite numbers (odd: a probability 0 times NaN
        // is NaN) are added to O here for the rows that see them, and become 0.
        int keep = 0;
        if constexpr (TAIL) {
          unsigned char* vs = ring + n % S::kStages * S::kStage + S::kHalf * S::kBox;
          if (ok && !wait(&full[n % S::kStages], (n / S::kStages) & 1)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          constexpr int PP = 8 * S::kHalf;                // 16-byte pieces of a slot
          const int s0 = min(max(0, r.p0 - t * kTile), kTile), s1 = min(max(0, r.len - t * kTile), kTile);
          auto piece = [&](int sl, int p) {               // in any order within a slot
            return reinterpret_cast<uint4*>(vs + (p >> 3) * S::kBox + sl * 128 + (p & 7) * 16);
          };
          for (int e = tid; e < (kTile - s1) * PP; e += 128) *piece(s1 + e / PP, e % PP) = make_uint4(0u, 0u, 0u, 0u);
          constexpr uint32_t X = Num<TC>::kExp;
          auto bad = [](uint32_t v) { return ((v & X) == X ? 1 : 0) | ((v >> 16 & X) == X ? 2 : 0); };
          if (r.len - r.p0 > 1 || a.mask) {
            int odd = 0;
            for (int e = tid; e < (s1 - s0) * PP; e += 128) {
              const uint4 v = *piece(s0 + e / PP, e % PP);
              odd |= bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w);
            }
            int any;
            __syncwarp();
            asm volatile(
                "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.aligned.pred q, 1, 128, p;\n"
                " selp.s32 %0, 1, 0, q;\n}"
                : "=r"(any)
                : "r"(odd)
                : "memory");
            if (any) {
              if (warp_live) {
                float p[kTile];                           // (indexed at run time: local memory)
#pragma unroll
                for (int i = 0; i < kTile; ++i) p[i] = x[i];
                if (!fresh) o_wait(n - 1);
#pragma unroll 1
                for (int c = 0; c < HD / 16; ++c) {
                  uint32_t v[16];
                  if (fresh) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0u;
                  } else {
                    tmem_ld16(lanes + S::kO + 16 * c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
                  }
#pragma unroll 1
                  for (int sl = s0; sl < s1; ++sl) {
                    if (!(vis >> sl & 1)) continue;
#pragma unroll
                    for (int h = 0; h < 8; ++h) {         // dimensions 16 c + 2 h, + 1
                      const int d = 16 * c + 2 * h;
                      const uint32_t y = *reinterpret_cast<const uint32_t*>(
                          vs + (d >> 6) * S::kBox + sl * 128 + (((d >> 3 & 7) ^ (sl & 7)) << 4) + 2 * (d & 7));
                      if (bad(y) & 1) v[2 * h] = __float_as_uint(fmaf(p[sl], Num<TC>::lo(y), __uint_as_float(v[2 * h])));
                      if (bad(y) & 2)
                        v[2 * h + 1] = __float_as_uint(fmaf(p[sl], Num<TC>::hi(y), __uint_as_float(v[2 * h + 1])));
                    }
                  }
                  __syncwarp();
                  tmem_st16(lanes + S::kO + 16 * c, v);
                }
                tmem_st_wait();
              }
              keep = 1;
              __syncwarp();
              sync4();   // everyone has read them
              for (int e = tid; e < (s1 - s0) * PP; e += 128) {
                uint4 v = *piece(s0 + e / PP, e % PP);
                auto clean = [&](uint32_t y) {
                  return (bad(y) & 1 ? 0u : y & 0xffffu) | (bad(y) & 2 ? 0u : y & 0xffff0000u);
                };
                *piece(s0 + e / PP, e % PP) = make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
              }
            }
          }
          fence_proxy_async();
        }
        // ---- probabilities, in the cache's type (of fp32 queries: three terms)
        if (warp_live) {
          if constexpr (F32) {
            put_terms<32, TC>(lanes + S::kS + S::kSCols * b, x);
          } else {
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) p[i] = Num<TC>::pack(x[2 * i], x[2 * i + 1]);
            tmem_st32(lanes + S::kS + S::kSCols * b, p);
          }
          tmem_st_wait();
        }
        if (tid == 0 && fresh) s_keep[b] = keep;       // (the MMA warp reads it where O starts anew)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
        ++n;
      };
      const int plain = max(0, min(r.p0, r.len)) / kTile;   // units whose slots every row sees
      int t = w.t0;
      auto fold_now = [&] {
        if (!F32 && (t - w.t0) % S::kFold == 0 && t > w.t0) {
          fold(!folded);
          folded = true;
        }
      };
      for (; t < min(w.t1, plain); ++t) {
        fold_now();
        unit(std::false_type{}, t);
      }
      for (; t < w.t1; ++t) {
        fold_now();
        unit(std::true_type{}, t);
      }

      // ---- the end of the piece (both barriers are then past its units)
      if (w.t1 - w.t0 > 1) o_wait(n - 2);
      o_wait(n - 1);
      float f = 0.f;                             // of what lies in the part
      if (F32) {
        l += s_sum[row];
      } else if (folded && live) {
        const float2 ml = *part_ml;
        f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m) * a.scale2);
        l = fmaf(ml.y, f, l);
      }
      if (!ok) l = __int_as_float(0x7fc00000);   // an expired wait: NaN
      if (m != -INFINITY) m = fmaf(m, a.scale2, (float)-S::kUp);
      const bool begins = w.t0 == 0, whole = begins && w.t1 == r.nt;
      if (begins && tid == 0) describe(a, w, deal, whole);
      if (warp_live) {
        const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
        TQ* dst = static_cast<TQ*>(a.out) + (r.s0 + j) * a.o_row + hh * a.o_head;
#pragma unroll 1
        for (int c = 0; c < HD / 16; ++c) {
          uint32_t v[16];
          __syncwarp();
          tmem_ld16(lanes + S::kO + 16 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
          if (F32 && folded) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 y = sums[128 * (4 * c + i / 4)];
              v[i] = __float_as_uint(__uint_as_float(v[i]) + y.x);
              v[i + 1] = __float_as_uint(__uint_as_float(v[i + 1]) + y.y);
              v[i + 2] = __float_as_uint(__uint_as_float(v[i + 2]) + y.z);
              v[i + 3] = __float_as_uint(__uint_as_float(v[i + 3]) + y.w);
            }
          }
          if (!live) continue;
          if (!F32 && folded) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 y = *reinterpret_cast<const float4*>(part + 16 * c + i);
              v[i] = __float_as_uint(fmaf(y.x, f, __uint_as_float(v[i])));
              v[i + 1] = __float_as_uint(fmaf(y.y, f, __uint_as_float(v[i + 1])));
              v[i + 2] = __float_as_uint(fmaf(y.z, f, __uint_as_float(v[i + 2])));
              v[i + 3] = __float_as_uint(fmaf(y.w, f, __uint_as_float(v[i + 3])));
            }
          }
          // (a row that saw nothing: l = 0 and O = 0)
          if (whole && F32) {
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              put2<HD, float>(a, r.s0 + j, hh, 16 * c + i, __uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
          } else if (whole) {
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              o[i] = Num<TC>::pack(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + 16 * c) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + 16 * c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(part + 16 * c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
        }
        if (live && whole && a.lse)
          a.lse[(long)(r.s0 + j) * a.nq + hh] = l == 0.f ? -INFINITY : m * 0.693147180559945f + logf(l);
        if (live && !whole) *part_ml = make_float2(m, l);
      }
      tc_fence_before();   // O has been read: the next piece's first product may replace it
    }
    if (!ok && lane == 0) report_err(a.err, kErrWait);
    if (tid == 0) describe_none(a, w);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

}  // namespace pa
}  // namespace sf
