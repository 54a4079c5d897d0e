// prefix_sm100.cu -- one-token attention of a whole batch over one shared
// prefix: the B G query rows of a KV head (G = Hq / Hkv heads of B sequences)
// are the rows of one matrix product with the prefix's keys, so a K/V tile is
// read once for up to 256 rows instead of once per sequence.
//
// Per KV head this is forward attention of B G rows over Np keys without a
// mask, cut along the keys into splits that write normalised fp32 partials
// (cache_decode.cu merges them with the sequences' own keys by log-sum-exp):
//   S = Q K^T, t = s scale log2 e, p = 2^(t - m), l = sum p, O = P V / l.
//
// Bound by HBM up to 256 rows: 64 KB of K and V per 128-key tile against 16.8
// MFLOP on the tensor cores and 32768 exponentials; by the tensor cores and the
// exponentials beyond, when several row blocks read one tile from L2.
//
// Measured (bf16, 32 query and 8 KV heads of 128), the whole call with the sequences' own caches and the
// merge, in a CUDA graph with pauses, below the power cap: 64 sequences behind 32768 keys with up to 1024 of
// their own, 337 MB and 35 GFLOP, 63.5 us, 5.3 TB/s or 0.81 of a plain copy; 250 behind 8192 with up to 512
// E4M3 ones, 240 MB and 35 GFLOP, 72.9 us.  One call after another for seconds, at the cap: 74 and 82 us.
//
// The machinery is the forward kernel's (fwd_sm100.cu): a persistent CTA per
// SM; one or two 128-row query tiles; one thread issuing TMA loads of K and V
// into a two-stage ring, one issuing tcgen05 MMAs with S, P and O in TMEM, and
// a warpgroup per query tile with one row per thread.  What differs:
//  * a query tile packs 128 / G whole sequences: its TMA box is 64 columns x G
//    heads x (128 / G) sequences of q [B, Hq, d], so row r is head r % G of
//    sequence r / G.  Rows past G (128 / G), up to 127, hold whatever the
//    shared memory held; a row's results never reach another row's;
//  * with one query tile, a K/V tile is taken in two halves of 64 keys with an S
//    buffer each (S_h, P_h over its first columns): while a row's exponentials of
//    one half run, the tensor core multiplies the other half's P and refills its S
//    (1.57 us a K/V tile; 1.75 us with one S buffer of 128 keys, whose softmax and
//    products take turns).  Two query tiles overlap each other that way, and the
//    shorter products of halves only cost them (1.95 us a K/V tile; 2.4 us in
//    halves);
//  * the output is fp32, staged 32 columns at a time and written by a TMA box of
//    the same shape into o_part [B, Hq, S, d].
#include <cuda.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "serving.h"
#include "sm100.cuh"

namespace fa {
namespace {

using namespace sm100;

constexpr int kBM = 128;     // rows of a query tile (= TMEM lanes)
constexpr int kBN = 128;     // keys per K/V tile
constexpr int kStages = 2;   // K/V ring depth
// With one query tile, up to so many query rows of a KV head, or so many keys, P is taken as two 16-bit
// values (launch_d).  One pair of limits for both types and head sizes, each measured at a point or two.
constexpr int kRestRows = 32, kRestKeys = 1024;
// Register split with two query tiles: launched at 168 per thread (384 x 168 = 64512), the
// load/MMA warpgroup drops to 104 and the softmax warpgroups rise to 200 (2 x 128 x 200 +
// 128 x 104 = 64512).  One query tile (256 threads) needs no split.
constexpr int kRegsSoftmax = 200;
constexpr int kRegsControl = 104;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale O when m grows by more than 2^8
// fp16 weights are kept 2^7 larger (m lowered by 7): at most 2^15, normal down to 2^-21 of the reference,
// and off by 2^-32 of it at most below.  Unlifted, a key 2^-25 below another counted in l and not in O: of
// 20000 such keys behind one whose value was 0 nothing was left.
template <typename T>
constexpr float kLift = Elem<T>::kBf16 ? 0.f : 7.f;

// 2^x for two values on the FMA and integer pipes, as exp2_fma2 (sm100.cuh) does it but by a
// degree-5 minimax polynomial (gen_exp2_poly.py 5; relative error 2.4e-7 against the 7.5e-5 of degree
// 3): a prefix may hold a single key, whose LSE is log2 of one such value and is kept to fp32 here.
__device__ __forceinline__ float2 exp2_fma2_fine(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 t = __fadd2_rn(x, make_float2(12582912.f, 12582912.f));
  const float2 n = __fadd2_rn(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), x);
  float2 q = make_float2(1.327647245e-03f, 1.327647245e-03f);
  q = __ffma2_rn(q, f, make_float2(9.675540961e-03f, 9.675540961e-03f));
  q = __ffma2_rn(q, f, make_float2(5.550713092e-02f, 5.550713092e-02f));
  q = __ffma2_rn(q, f, make_float2(2.402212024e-01f, 2.402212024e-01f));
  q = __ffma2_rn(q, f, make_float2(6.931469440e-01f, 6.931469440e-01f));
  q = __ffma2_rn(q, f, make_float2(1.000000119e+00f, 1.000000119e+00f));
  return make_float2(__int_as_float(__float_as_int(q.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(q.y) + (__float_as_int(t.y) << 23)));
}
// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Of every eight column pairs of a score block, how many take it instead of ex2.approx (measured at
// 0, 2, 3 and 4: one query tile is fastest at 2 by 0.3 us in 34, two at 0 by 2.5 %).
template <int NT>
__device__ __forceinline__ float2 exp2_pair(float2 x, int pair) {
  constexpr int K = NT == 1 ? 2 : 0;
  if (((pair + 1) * K) / 8 != (pair * K) / 8) return exp2_fma2_fine(x);
  return make_float2(ex2(x.x), ex2(x.y));
}

template <int D, int NT, bool REST>
struct Smem {
  static constexpr int kPanel = 128 * 128;  // one [128 rows][128 bytes] swizzled panel
  static constexpr int kTile = (D / 64) * kPanel;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + NT * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffStage = kOffV + kStages * kTile;  // 32 fp32 columns per query tile
  static constexpr int kOffBar = kOffStage + NT * kPanel;
  enum { kBarQ = 0, kBarKFull = 1, kBarKEmpty = 3, kBarVFull = 5, kBarVEmpty = 7, kBarS = 9, kBarP = 13, kBarDrain = 17,
         kBarQEmpty = 18, kBarOFree = 19, kBarStageFull = 21, kBarStageDone = 23, kNumBars = 25 };
  // kBarS / kBarP + 2 t + h: S (P) of half h of query tile t is there.  S completes once more per work
  // than there are tiles: the last time when the last PV of that half has finished.
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmem + 4;
  static constexpr int kBytes = kOffAbort + 4 + 1024;  // + slack to align the base to 1024 B
  static_assert(kBytes <= 232448, "shared memory per CTA exceeded");
  static constexpr int kThreads = 128 * (NT + 1);
  static constexpr int kHalves = NT == 1 ? 2 : 1;  // S buffers of a query tile
  static constexpr int kWidth = kBN / kHalves;     // their keys
  static_assert(!REST || kHalves == 2, "the rest of P lies in the free half of an S buffer's columns");
  // TMEM columns: S_t, then O_t
  static constexpr uint32_t col_s(int t) { return 128u * t; }
  static constexpr uint32_t col_o(int t) { return 128u * NT + 128u * t; }
  static constexpr uint32_t kCols = 256u * NT;
};

struct Params {
  float* lse_part;  // [B,Hq,S]
  int B, Hq, Hkv, Np, G, seqs;  // seqs = 128 / G sequences per query tile
  int S, chunk;                 // splits and their keys
  int row_blocks;               // NT query tiles each
  int num_work;                 // S * Hkv * row_blocks
  float scale_log2;  // positive: masked scores are -inf before it multiplies them
  int* status;
};

// Work w: row blocks of one (split, KV head) are neighbours, so the CTAs that share its K/V tiles
// run together.
struct Work {
  int rb, hk, s;
};
__device__ __forceinline__ Work work_at(const Params& p, int w) {
  return Work{w % p.row_blocks, (w / p.row_blocks) % p.Hkv, w / (p.row_blocks * p.Hkv)};
}

template <typename T, int D, int NT, bool REST>
__global__ void __launch_bounds__(Smem<D, NT, REST>::kThreads, 1)
    prefix_sm100_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO, Params p) {
  using L = Smem<D, NT, REST>;
  constexpr int kWarpLoad = 4 * NT, kWarpMma = 4 * NT + 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* gb = smem_raw + (sb - raw);
  auto bar = [&](int i) { return sb + L::kOffBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + L::kOffAbort);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto blocks_of = [&](const Work& x) {  // K/V tiles of a split
    return (min(p.chunk, p.Np - x.s * p.chunk) + kBN - 1) / kBN;
  };

  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i)
      mbar_init(bar(i), (i >= L::kBarP && i < L::kBarP + 4) || (i >= L::kBarOFree && i < L::kBarStageDone) ? kBM : 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(sb + L::kOffTmem, L::kCols);
    tmem_relinquish();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmO);
  }
  // behind every earlier grid; and the caches' partials, launched next as a programmatic dependent,
  // share no output with this kernel and may fill SMs as its CTAs leave
  wait_for_earlier_grids();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(gb + L::kOffTmem);

  if (warp >= kWarpLoad) {
   if constexpr (NT == 2) regs_decrease<kRegsControl>();
   if (warp == kWarpLoad) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(p.G * p.seqs * 128 * (D / 64));  // of one query tile's boxes
      int last_k[kStages] = {-1, -1}, last_v[kStages] = {-1, -1};
      int last_q = -1;
      int g = 0;  // K/V tiles loaded so far by this CTA (ring position)
      int wl = 0;
      for (int w = blockIdx.x; w < p.num_work; w += gridDim.x, ++wl) {
        const Work x = work_at(p, w);
        const int nblk = blocks_of(x), key0 = x.s * p.chunk;
        // the previous work's last score MMAs must have read Q before it is replaced
        if (wl > 0 && !mbar_wait(bar(L::kBarQEmpty), (wl - 1) & 1, abort_flag, p.status)) break;
        mbar_expect_tx(bar(L::kBarQ), NT * q_bytes);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::kOffQ + t * L::kTile + pn * L::kPanel, &tmQ, bar(L::kBarQ), 64 * pn, x.hk * p.G,
                        (x.rb * NT + t) * p.seqs, 0);
        last_q = wl;
        bool stop = false;
        for (int j = 0; j < nblk; ++j, ++g) {
          const int st = g & 1, u = g >> 1;
          if (u > 0 && !mbar_wait(bar(L::kBarKEmpty + st), (u - 1) & 1, abort_flag, p.status)) {
            stop = true;
            break;
          }
          mbar_expect_tx(bar(L::kBarKFull + st), L::kTile);
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::kOffK + st * L::kTile + pn * L::kPanel, &tmK, bar(L::kBarKFull + st), 64 * pn, x.hk,
                        key0 + j * kBN, 0);
          last_k[st] = u;
          if (u > 0 && !mbar_wait(bar(L::kBarVEmpty + st), (u - 1) & 1, abort_flag, p.status)) {
            stop = true;
            break;
          }
          mbar_expect_tx(bar(L::kBarVFull + st), L::kTile);
#pragma unroll
          for (int pn = 0; pn < D / 64; ++pn)
            tma_load_4d(sb + L::kOffV + st * L::kTile + pn * L::kPanel, &tmV, bar(L::kBarVFull + st), 64 * pn, x.hk,
                        key0 + j * kBN, 0);
          last_v[st] = u;
        }
        if (stop) break;
      }
      if (*abort_flag) {
        // let every copy this thread issued land before the CTA releases its shared memory
        if (last_q >= 0) wait_drain(bar(L::kBarQ), last_q & 1, p.status);
        for (int st = 0; st < kStages; ++st) {
          if (last_k[st] >= 0) wait_drain(bar(L::kBarKFull + st), last_k[st] & 1, p.status);
          if (last_v[st] >= 0) wait_drain(bar(L::kBarVFull + st), last_v[st] & 1, p.status);
        }
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr bool kBf16 = Elem<T>::kBf16;
      constexpr uint32_t idq = idesc_f16(kBf16, kBM, L::kWidth, false);
      constexpr uint32_t idv = idesc_f16(kBf16, kBM, D, true);
      auto qk = [&](int t, int h, int st) {  // scores of keys kWidth h .. of the tile
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = (kk >> 2) * L::kPanel + (kk & 3) * 32;
          const uint64_t a = sdesc_sw128(sb + L::kOffQ + t * L::kTile + ko, 16, 1024);
          const uint64_t bd = sdesc_sw128(sb + L::kOffK + st * L::kTile + ko + h * (L::kWidth * 128), 16, 1024);
          mma_ss(tbase + L::col_s(t) + L::kWidth * h, a, bd, idq, kk > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](int t, int h, int st, bool first) {
#pragma unroll
        for (int kk = 0; kk < L::kWidth / 16; ++kk) {
          // V stored [keys][d]: B is N(=d)-major; 16 keys = two 8-row groups of 128 B
          const uint64_t bd =
              sdesc_sw128(sb + L::kOffV + st * L::kTile + (h * (L::kWidth / 16) + kk) * 2048, L::kPanel, 1024);
          mma_ts(tbase + L::col_o(t), tbase + L::col_s(t) + L::kWidth * h + kk * 8, bd, idv, (!first || kk > 0) ? 1u : 0u);
          if constexpr (REST)  // and what rounding P left, in the second half of S's columns
            mma_ts(tbase + L::col_o(t), tbase + L::col_s(t) + L::kWidth * h + L::kWidth / 2 + kk * 8, bd, idv, 1u);
        }
      };
      bool ok = true;
      int g = 0;  // K/V tiles consumed so far by this CTA; P barriers complete once per tile
      int wl = 0;
      for (int w = blockIdx.x; ok && w < p.num_work; w += gridDim.x, ++wl) {
        const int nblk = blocks_of(work_at(p, w));
        ok = mbar_wait(bar(L::kBarQ), wl & 1, abort_flag, p.status) &&
             mbar_wait(bar(L::kBarKFull + (g & 1)), (g >> 1) & 1, abort_flag, p.status);
        // the previous epilogue has read O_t: only then may S complete again (its waiters tell two
        // neighbouring completions apart, not three) and O_t be overwritten
        for (int t = 0; ok && t < NT && wl > 0; ++t)
          ok = mbar_wait(bar(L::kBarOFree + t), (wl - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < L::kHalves; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            qk(t, h, g & 1);
            mma_commit(bar(L::kBarS + 2 * t + h));
          }
        mma_commit(bar(L::kBarKEmpty + (g & 1)));
        if (nblk == 1) mma_commit(bar(L::kBarQEmpty));
        for (int j = 0; ok && j < nblk; ++j, ++g) {
          const int st = g & 1, u = g >> 1;
          const bool more = j + 1 < nblk;
          const int st1 = (g + 1) & 1, u1 = (g + 1) >> 1;
          ok = mbar_wait(bar(L::kBarVFull + st), u & 1, abort_flag, p.status);
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              ok = ok && mbar_wait(bar(L::kBarP + 2 * t + h), g & 1, abort_flag, p.status);
              if (ok) {
                tc_fence_after();
                pv(t, h, st, j == 0 && h == 0);
                if (more && h == 0 && t == 0) ok = mbar_wait(bar(L::kBarKFull + st1), u1 & 1, abort_flag, p.status);
              }
              if (ok) {
                if (more) {
                  tc_fence_after();
                  qk(t, h, st1);  // overwrites S_h / P_h of the tile after its PV, in issue order
                }
                mma_commit(bar(L::kBarS + 2 * t + h));
              }
            }
          if (!ok) break;
          if (!more) mma_commit(bar(L::kBarVEmpty + st));  // inside a work the softmax warps free V (below)
          if (more && j + 2 == nblk) mma_commit(bar(L::kBarQEmpty));  // last score MMAs issued
        }
      }
      // no MMA may still run when TMEM is released
      mma_commit(bar(L::kBarDrain));
      wait_drain(bar(L::kBarDrain), 0, p.status);
    }
   }
  } else {
    if constexpr (NT == 2) regs_increase<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax + epilogue
    const int t = warp >> 2;
    const int wq = warp & 3;
    const int rr = wq * 32 + lane;  // row of the query tile
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tbase + lane_off + L::col_s(t);
    const uint32_t tO = tbase + lane_off + L::col_o(t);
    const float c = p.scale_log2;
    bool ok = true;
    int g = 0;  // K/V tiles processed so far by this CTA; S has completed g + wl times
    int wl = 0;
    for (int w = blockIdx.x; ok && w < p.num_work; w += gridDim.x, ++wl) {
      const Work x = work_at(p, w);
      const int nblk = blocks_of(x), key0 = x.s * p.chunk;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < nblk; ++j, ++g) {
#pragma unroll 1
        for (int h = 0; h < L::kHalves; ++h) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarS + 2 * t + h), (g + wl) & 1, abort_flag, p.status));
          if (!ok) break;
          if (t == NT - 1 && h == L::kHalves - 1 && wq == 0 && lane == 0 && j != 0) {
            // the last S of tile g is complete, and with it every MMA issued before it: the score
            // MMAs of tile g (its K stage is free) and the PV of tile g - 1 (its V stage is)
            mbar_arrive(bar(L::kBarKEmpty + (g & 1)));
            mbar_arrive(bar(L::kBarVEmpty + ((g - 1) & 1)));
          }
          tc_fence_after();
          const uint32_t tSh = tS + L::kWidth * h;
          float s[L::kWidth];
          {
            uint32_t r[L::kWidth / 32][32];
#pragma unroll
            for (int q = 0; q < L::kWidth / 32; ++q) tmem_ld32(tSh + 32 * q, r[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < L::kWidth / 32; ++q) {
              reg_fence(r[q]);
#pragma unroll
              for (int i = 0; i < 32; ++i) s[32 * q + i] = __uint_as_float(r[q][i]);
            }
          }
          const int lim = p.Np - (key0 + j * kBN + L::kWidth * h);  // keys of this S inside the prefix
          if (lim < L::kWidth) {
#pragma unroll
            for (int i = 0; i < L::kWidth; ++i)
              if (i >= lim) s[i] = -INFINITY;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < L::kWidth; i += 8) {
            mx[0] = max3_nan(mx[0], s[i], s[i + 1]);
            mx[1] = max3_nan(mx[1], s[i + 2], s[i + 3]);
            mx[2] = max3_nan(mx[2], s[i + 4], s[i + 5]);
            mx[3] = max3_nan(mx[3], s[i + 6], s[i + 7]);
          }
          const float mxs = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * c;
          const bool resc = mxs > m_ref + kRescaleThreshold;
          const float corr = resc ? ex2(m_ref - mxs) : 1.f;
          if (resc) m_ref = mxs;
          l *= corr;
          const float mu = (m_ref == -INFINITY ? 0.f : m_ref) - kLift<T>;
          const float2 c2 = make_float2(c, c), nm2 = make_float2(-mu, -mu);
          float2 rs0 = make_float2(0.f, 0.f), rs1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < L::kWidth / 32; ++q) {
            uint32_t pk[16], pr[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const int c0 = 32 * q + 2 * i;
              const float2 xa = __ffma2_rn(make_float2(s[c0], s[c0 + 1]), c2, nm2);
              const float2 xb = __ffma2_rn(make_float2(s[c0 + 2], s[c0 + 3]), c2, nm2);
              const float2 a = exp2_pair<NT>(xa, 16 * q + i), bb = exp2_pair<NT>(xb, 16 * q + i + 1);
              rs0 = __fadd2_rn(rs0, a);
              rs1 = __fadd2_rn(rs1, bb);
              pk[i] = Elem<T>::pack(a.x, a.y);
              pk[i + 1] = Elem<T>::pack(bb.x, bb.y);
              if constexpr (REST) {
                const float2 ha = Elem<T>::unpack(pk[i]), hb = Elem<T>::unpack(pk[i + 1]);
                pr[i] = Elem<T>::pack(a.x - ha.x, a.y - ha.y);
                pr[i + 1] = Elem<T>::pack(bb.x - hb.x, bb.y - hb.y);
              }
            }
            tmem_st16(tSh + 16 * q, pk);
            if constexpr (REST) tmem_st16(tSh + L::kWidth / 2 + 16 * q, pr);
          }
          l += (rs0.x + rs0.y) + (rs1.x + rs1.y);
          // a NaN or +inf score makes the row NaN, also where the polynomial would clamp it away
          if (!(mxs < INFINITY)) l = NAN;
          if (__any_sync(0xffffffffu, resc && j + h > 0)) {
            if constexpr (L::kHalves == 2) {
              // the other half's last PV must have finished (with one S buffer this S is behind it)
              ok = __all_sync(0xffffffffu,
                              mbar_wait(bar(L::kBarS + 2 * t + (h ^ 1)), (g + wl + h) & 1, abort_flag, p.status));
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t r[32];
              tmem_ld32(tO + q * 32, r);
              tmem_wait_ld();
              reg_fence(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
              tmem_st32(tO + q * 32, r);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(L::kBarP + 2 * t + h));
        }
        if (!ok) break;
      }
      // the last PV has finished (of both halves: the first's was committed before the second's)
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarS + 2 * t + L::kHalves - 1), (g + wl) & 1, abort_flag,
                                                  p.status));
      if (!ok) break;
      uint32_t r[D];
      // O_t: TMEM -> registers, then hand the TMEM columns back to the MMA thread at once
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < D / 32; ++q) tmem_ld32(tO + q * 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * q));
      tmem_wait_ld();
#pragma unroll
      for (int q = 0; q < D / 32; ++q) reg_fence(*reinterpret_cast<uint32_t(*)[32]>(r + 32 * q));
      tc_fence_before();
      mbar_arrive(bar(L::kBarOFree + t));

      const int b0 = (x.rb * NT + t) * p.seqs;  // first sequence of this query tile
      if (m_ref == -INFINITY && l == l) l = 0.f;  // every score -inf (clamped exponentials aside): O = 0, LSE = -inf
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int b = b0 + rr / p.G;
      if (rr < p.G * p.seqs && b < p.B) {
        const long li = ((long)b * p.Hq + x.hk * p.G + rr % p.G) * p.S + x.s;
        if (FA_IN_BOUNDS(p.status, li, (long)p.B * p.Hq * p.S))
          p.lse_part[li] = ((m_ref == -INFINITY ? 0.f : m_ref) - kLift<T> + log2f(l)) * kLn2;
      }
      const uint32_t half = sb + L::kOffStage + t * L::kPanel;
#pragma unroll
      for (int pn = 0; pn < D / 32; ++pn) {
        const int u = wl * (D / 32) + pn;  // uses of this tile's stage so far
        if (u > 0)
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarStageDone + t), (u - 1) & 1, abort_flag, p.status));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          auto f = [&](int i) { return __float_as_uint(__uint_as_float(r[32 * pn + 4 * k + i]) * inv); };
          st_shared_v4(half + rr * 128 + ((k ^ (rr & 7)) << 4), f(0), f(1), f(2), f(3));
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(L::kBarStageFull + t));
        if (wq == 0 && lane == 0) {
          ok = mbar_wait(bar(L::kBarStageFull + t), u & 1, abort_flag, p.status);
          if (ok) {
            if (b0 < p.B) {  // a block's second tile may hold no sequence
              tma_store_4d(&tmO, half, 32 * pn, x.s, x.hk * p.G, b0);
              bulk_commit();
              bulk_wait_read_all();
            }
            mbar_arrive(bar(L::kBarStageDone + t));
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
    }
    // stores must be complete before the CTA exits
    if (wq == 0 && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tbase, L::kCols);
  }
}

template <typename T, int D, int NT, bool REST>
cudaError_t launch(const CacheDecodeArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.Hkv, seqs = kBM / G, S = a.prefix_splits;
  const int type = Elem<T>::kBf16 ? kMapBf16 : kMapF16;
  CUtensorMap mq, mk, mv, mo;
  {
    const uint64_t dims[4] = {D, (uint64_t)a.Hq, (uint64_t)a.B, 1};
    const uint64_t st[3] = {D * 2, (uint64_t)a.Hq * D * 2, (uint64_t)a.B * a.Hq * D * 2};
    const uint32_t box[4] = {64, (uint32_t)G, (uint32_t)seqs, 1};
    if (!make_map_box(&mq, a.q, type, dims, st, box)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[4] = {D, (uint64_t)S, (uint64_t)a.Hq, (uint64_t)a.B};
    const uint64_t st[3] = {D * 4, (uint64_t)S * D * 4, (uint64_t)a.Hq * S * D * 4};
    const uint32_t box[4] = {32, 1, (uint32_t)G, (uint32_t)seqs};
    if (!make_map_box(&mo, a.o_part, kMapF32, dims, st, box)) return cudaErrorInvalidValue;
  }
  if (!make_map(&mk, a.kp, Elem<T>::kBf16, D, a.Hkv, a.Np, 1, kBN) ||
      !make_map(&mv, a.vp, Elem<T>::kBf16, D, a.Hkv, a.Np, 1, kBN))
    return cudaErrorInvalidValue;
  const int rows = (a.B + NT * seqs - 1) / (NT * seqs);
  const long long work = (long long)rows * a.Hkv * a.prefix_splits;
  if (work > (1ll << 30)) return cudaErrorInvalidValue;
  // A scale of 0 would make NaN of a masked score.  The smallest positive number in its place leaves -inf as
  // it is and takes any finite score to below 2^-20, whose weight is 1 as for a score of 0.  (Scaling the last
  // tile's scores before they are masked does as well, but costs prefixes of two query tiles 1.6 to 3.9 %.)
  const float scale_log2 = std::max(a.scale * kLog2e, 0x1p-149f);
  Params p{a.lse_part, a.B, a.Hq, a.Hkv, a.Np, G, seqs, S, a.prefix_chunk, rows, (int)work, scale_log2, a.status};
  auto kern = prefix_sm100_kernel<T, D, NT, REST>;
  constexpr int smem = Smem<D, NT, REST>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = (int)std::min<long long>(work, a.prefix_ctas);
  return launch_dependent(kern, dim3(grid), Smem<D, NT, REST>::kThreads, smem, s, mq, mk, mv, mo, p);
}

template <typename T, int D>
cudaError_t launch_d(const CacheDecodeArgs& a, cudaStream_t s) {
  const int G = a.Hq / a.Hkv;
  // Rounding P to 16 bits costs an output as much as its own rounding does: over many outputs 1.41 times
  // the error of the last rounding alone, over the few of a small batch up to 1.6.  Multiplying P's rest
  // too takes that back and half as many products more.  Two query tiles, whose softmax spills for it with
  // heads of 128, go without at any length (64 sequences behind 32768 bf16 keys: error 1.40 and 64 us, with the
  // rest 1.00 and 79; 250 behind 8192: 1.16 and 76, 1.01 and 98).
  if (a.B > kBM / G) return launch<T, D, 2, false>(a, s);
  // One tile takes it for the few rows of a small batch (1.83 us a K/V tile instead of 1.57) and behind a
  // short prefix, where a call is mostly launches (32 sequences behind 1000 keys 15.1 us and 1.00 times the
  // error of one rounding, without it 14.7 and 1.30).
  return a.B * G <= kRestRows || a.Np <= kRestKeys ? launch<T, D, 1, true>(a, s) : launch<T, D, 1, false>(a, s);
}

template <typename T>
cudaError_t launch_t(const CacheDecodeArgs& a, cudaStream_t s) {
  return a.d == 128 ? launch_d<T, 128>(a, s) : launch_d<T, 64>(a, s);
}

}  // namespace

cudaError_t launch_prefix_sm100(const CacheDecodeArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<__half>(a, s);
}

}  // namespace fa
