// cache_decode.cu -- one-token attention over a key/value cache in 16 bits or
// in E4M3 (fp8_cache.cu's rows), as split partials, and the log-sum-exp merge
// of those partials with a shared prefix's (prefix_sm100.cu).
//
// For a query row q of head h and the cached keys j of its sequence,
//   t_j = scale log2(e) s^k_j (q . c^k_j),   p_j = 2^(t_j - m),
//   l = sum p_j,   o = sum p_j s^v_j c^v_j / l,   lse = ln 2 (m + log2 l)
// with codes c and scales s of an E4M3 cache (s = 1 and c the values themselves
// in 16 bits).  The codes are never multiplied out: s^k_j joins the score and
// s^v_j the weight, so a key costs its d + 4 bytes twice.
//
// Work.  The keys of the batch, in blocks of kBlock, sequence after sequence, are
// one line of W blocks, W from the lengths on the device; of the C CTAs (C <= W) of
// each KV head, CTA i takes the blocks from i W / C to (i + 1) W / C, whatever
// sequences they belong to, and leaves one partial (O, LSE of the group's rows) per
// sequence that it touches, in its head's slot b + i -- along the line either
// summand grows, so no two partials share one; a sequence that one CTA has whole, without
// a prefix, goes straight to the outputs (1000 sequences of up to 1000 keys: 259 us, 269 through the merge; for
// groups of 9 to 16 heads, whose CTAs have no register left, 500 of 700 36.2 and 35.9, so they do not).  Every CTA has the same keys to read
// however ragged the batch, and the CTAs of the Hkv heads, neighbours in the grid,
// read the same tokens' rows together (a line through the heads as well, whose CTAs
// stand at different tokens, lost 13 % of the bandwidth).
//
// Small batches (SOLO): a cluster of up to 8 CTAs per sequence and KV head shares
// that sequence's blocks out and merges through distributed shared memory, with the
// few partials of a shared prefix if there is one: one launch instead of two, and
// no workspace of its own.
//
// A CTA.  The group's Hq / Hkv query rows share every byte it reads.  Each of the
// four warps streams its own kStep keys of a block through its own two cp.async
// buffers (no block barrier until a sequence's end) with its own running (m, l, O);
// the warps merge through shared memory while the next block arrives.  Bound by
// HBM reads of the cache as long as the arithmetic per key is small, which shapes
// the rest:
//  * The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that
//    keys and columns of d fill the MMA's 16 rows and the group its 8 columns
//    (two column blocks for groups of 9 to 16): half the MMAs, exponentials and
//    accumulators of padding the group to 16 rows.
//  * m is a reference that stays until a score exceeds it by more than 2^6:
//    then every lane's maximum is reduced and O, l rescaled; otherwise a block
//    costs one vote.
//
// E4M3 operands.  E4M3 values are exact in fp16, so codes are converted in
// registers (cvt.rn.f16x2.e4m3x2) and multiplied as m16n8k16 fp16 products:
//  * K: an 8 x 16-byte ldmatrix gives a thread four consecutive codes of a key;
//    the order in which the MMA's k index runs over d is free as long as q
//    follows it, so q is loaded in that order.
//  * V: the transposing ldmatrix moves 16-bit units, here two neighbouring
//    columns of one key; a byte permutation per register gives the key pairs of
//    either column, so rows r and r + 8 of an MMA are columns 2 r and 2 r + 1.
//  * q in bf16 is scaled by a power of two per row that brings its largest
//    value to [2^14, 2^15): conversion to fp16 is then exact for every element
//    within 2^-30 of the row's largest and off by at most 2^-39 of it below.
//  * the weights p_j s^v_j are fp16 in units of 2^(e - 8), where 2^e exceeds
//    every s^v seen so far: at most 2^14 (p up to 2^6), relative error 2^-11
//    down to 2^-22 of 2^e, absolute 2^-33 of it below.
// Measured (bf16, 32 query and 8 KV heads of 128), with the merge: 64 sequences of up to 32768 keys, 3.34 GB,
// 496 to 504 us, 6.7 to 6.6 TB/s or 1.03 to 1.01 of a plain copy; in a CUDA graph one of 32768 18.2 us, 16 of
// up to 2000 15.3 us.  With 9 to 16 query heads a KV head, heads of 128 spill up to 104 bytes a thread.
//
// l sums the unrounded p_j.  fp16 weights of a 16-bit cache are kept 2^8 larger
// (m lowered by 8) for the same reason: at most 2^14, normal down to 2^-22.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr float kStale = 6.f;  // log2 units that a score may exceed the reference m by
// Rounding the weights to 16 bits costs an output as much as its own rounding does: over many outputs
// 1.41 times the error of the last rounding alone, over the few of a small batch up to 1.6.  With REST
// the rounding errors are multiplied too, and only the last rounding shows.  A 16-bit cache always takes
// it (its loads hide it); an E4M3 cache with bf16 output never (its weights are rounded to fp16: 64 sequences
// of 32768 keys, 1.01 times the error of one rounding), with fp16 output up to so many rows (32 sequences of
// 3000 keys, 16 heads, d = 64: 39.6 us with, 33.6 without).
constexpr int kRestRows = 256;
constexpr int kMinUnit = -112;  // smallest e of the weights' unit (all powers of two below stay normal)

// A warp's two buffers of kStep keys each.  Two of them (99 KB in flight on an SM of three CTAs) leave
// room for a third CTA: three of 32 keys were 2 % slower on 32768-key sequences and up to 30 % on
// short ones.  E4M3 rows of 128 values, 64 sequences of 32768 keys and 16 of 2000: 32 keys and three CTAs an
// SM 496 and 15.3 us, 16 keys and four CTAs (128 registers) 500 and 19.2, 16 keys and three 528 and 19.1.
template <int D, bool F8>
struct Ring {
  static constexpr int kRow = D * (F8 ? 1 : 2);          // bytes of a K or V row
  static constexpr int kStep = kRow <= 128 ? 32 : 16;    // keys per block
  static constexpr int kTile = kStep * kRow;
  static constexpr int kStage = 2 * kTile + (F8 ? 2 * kStep * 4 : 0);  // K, V, their scales
  static constexpr int kBlocks = kStep / 16;
};
template <int D, bool F8, int NB>
struct Smem {
  static constexpr int kOffM = 4 * 2 * Ring<D, F8>::kStage;  // m, l [4][8 NB] fp32, then the offset of each warp's O
  static constexpr int kBytes = kOffM + 4 * 8 * NB * 2 * 4 + 4 * 4;
  static constexpr int kOffSolo = (kBytes + 15) / 16 * 16;  // SOLO: this CTA's O [8 NB][D] and LSE [8 NB]
  static constexpr int kSoloBytes = kOffSolo + 8 * NB * (D + 1) * 4;
  static_assert(8 * NB * D * 4 <= Ring<D, F8>::kStage, "a warp's O is merged through its free buffer");
};

// Byte offset of 16-byte chunk `c` of row `r` in a tile of ROW-byte rows, chunks permuted so that
// one chunk of eight consecutive rows (ldmatrix) touches every bank once.
template <int ROW>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * ROW + ((c ^ (ROW >= 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
// Four E4M3 codes (low byte first) as two fp16 pairs; exact.
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
// Transpose of an 8 x 8 matrix of 16-bit values held as ldmatrix leaves it.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Maximum and sum over the lanes that hold the same query rows (lane & 3 equal).
__device__ __forceinline__ float rows_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float rows_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// A run of blocks of one sequence, as one warp sees it.
struct Item {
  int b;
  int first, hi;     // this warp's keys: kStep from first + i kBlock on, below hi
  int nblk;
  int pos;           // place of the run's first block on the line
  int blk, blks;     // that block within the sequence, and the sequence's blocks
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Shared memory of the cluster's CTA `rank` at this CTA's address `addr`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}

template <typename T, int D, bool F8, int NB, bool REST, bool SOLO>
__global__ void __launch_bounds__(kThreads, cache_ctas_per_sm(D, F8, NB == 2)) cache_decode_kernel(CacheDecodeArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using R = Ring<D, F8>;
  using L = Smem<D, F8, NB>;
  using M = typename std::conditional<F8, __half, T>::type;  // MMA operand type
  constexpr int MB = R::kBlocks;
  constexpr int kBlock = 4 * R::kStep;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  int rank = 0, ranks = 1;  // SOLO: place in the cluster
  if constexpr (SOLO) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    ranks = p.solo;
  }
  const int unit = SOLO ? blockIdx.x / ranks : blockIdx.x;
  const int hk = unit % p.Hkv, cta = unit / p.Hkv;  // SOLO: cta is the sequence
  // behind every earlier grid but a prefix kernel's, which itself started behind all others; the merge,
  // launched next, may become resident
  if (!p.after_prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
  if constexpr (!SOLO) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const uint32_t ring = smem_u32(smem) + warp * 2 * R::kStage;
  const uint8_t* const ring_g = smem + warp * 2 * R::kStage;
  float* const red_m = reinterpret_cast<float*>(smem + L::kOffM);
  float* const red_l = red_m + 4 * 8 * NB;
  uint32_t* const red_at = reinterpret_cast<uint32_t*>(red_l + 4 * 8 * NB);
  const long row_bytes = (long)p.Hkv * R::kRow;

  // W, this CTA's part [begin, end) of the line, and the sequence that begin lies in.  Every warp for
  // itself: a lane sums the blocks of a stretch of sequences, and the one whose stretch holds begin walks it
  auto length = [&](int b) { return FA_IN_BOUNDS(p.status, b, p.B) ? min(max(p.seqlens[b], 0), p.Nk_max) : 0; };
  auto blocks = [&](int n) { return (n + kBlock - 1) / kBlock; };
  int begin, end, W = 0, C = 0;  // W < 2^31: a block of a head takes 4 KB at least
  int cb = 0, cblk = 0, cn = 0, cpos;  // the cursor: block cblk of sequence cb, of cn keys, at place cpos
  if constexpr (SOLO) {
    cb = cta;
    cn = length(cb);
    const int nb = blocks(cn);
    cpos = cblk = begin = (int)((long long)rank * nb / ranks);
    end = (int)((long long)(rank + 1) * nb / ranks);
  } else {
    const int per = (p.B + 31) / 32;
    const int b0 = min(lane * per, p.B), b1 = min(b0 + per, p.B);
    int mine = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) mine += blocks(length(b));
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    W = __shfl_sync(0xffffffffu, upto, 31);
    C = min(p.cache_ctas / p.Hkv, W);  // a CTA without a block would be a gap in its neighbours' spans
    begin = cta < C ? (int)((long long)cta * W / C) : W;
    end = cta < C ? (int)((long long)(cta + 1) * W / C) : W;
    int at = upto - mine;  // place of sequence b0
    const bool here = begin < end && at <= begin && begin < upto;
    if (here) {
      cb = b0;
      cn = length(cb);
      while (begin >= at + blocks(cn)) {
        at += blocks(cn);
        cn = length(++cb);
      }
      cblk = begin - at;
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    cb = __shfl_sync(0xffffffffu, cb, who & 31);
    cn = __shfl_sync(0xffffffffu, cn, who & 31);
    cblk = __shfl_sync(0xffffffffu, cblk, who & 31);
    cpos = begin;
  }
  // the line's next run within [cpos, end)
  auto next = [&](Item& it) {
    if (cpos >= end) return false;
    while (cblk == blocks(cn)) {  // this sequence is done, or has no key
      cn = length(++cb);
      cblk = 0;
    }
    it.b = cb;
    it.pos = cpos;
    it.blk = cblk;
    it.blks = blocks(cn);
    const int take = min(it.blks - cblk, end - cpos);
    it.first = cblk * kBlock + warp * R::kStep;
    it.hi = min((cblk + take) * kBlock, cn);
    it.nblk = it.first < it.hi ? (it.hi - it.first + kBlock - 1) / kBlock : 0;
    cpos += take;
    cblk += take;
    return true;
  };
  constexpr int kC = R::kRow / 16, kRows = 32 / kC;  // chunks per row, rows per pass of the warp
  const int lr = lane / kC, lc = lane % kC;
  // the loads run one block ahead of the products: `src` is the next block that this warp loads
  struct {
    const uint8_t *k, *v;    // this lane's chunk of row lr
    const float *ks, *vs;    // the scales of row lane % kStep
    int keys;                // rows of the block that are inside, kStep or more if it is full
    int left;                // blocks of its item still to load
  } src;
  src.left = 0;
  const long kstride = (long)kBlock * row_bytes;
  // (of the checking build: 16 bytes of K and of V, and a key's two scales, lie inside the cache)
  auto inside = [&](const uint8_t* k, const uint8_t* v) {
    const long last = (long)p.B * p.Nk_max * row_bytes - 15;
    return FA_IN_BOUNDS(p.status, k - static_cast<const uint8_t*>(p.k), last) &&
           FA_IN_BOUNDS(p.status, v - static_cast<const uint8_t*>(p.v), last);
  };
  auto inside_scales = [&](const float* ks, const float* vs) {
    const long all = (long)p.B * p.Hkv * p.Nk_max;
    return FA_IN_BOUNDS(p.status, ks - p.k_scale, all) && FA_IN_BOUNDS(p.status, vs - p.v_scale, all);
  };
  auto aim = [&](const Item& it) {
    const long row = ((long)it.b * p.Nk_max + it.first + lr) * p.Hkv + hk;
    src.k = static_cast<const uint8_t*>(p.k) + row * R::kRow + 16 * lc;
    src.v = static_cast<const uint8_t*>(p.v) + row * R::kRow + 16 * lc;
    if constexpr (F8) {
      const long at = ((long)it.b * p.Hkv + hk) * p.Nk_max + it.first + lane % R::kStep;
      src.ks = p.k_scale + at;
      src.vs = p.v_scale + at;
    }
    src.keys = it.hi - it.first;
    src.left = it.nblk;
  };
  auto load = [&](int stage) {
    const uint32_t st = ring + stage * R::kStage;
    if (src.keys >= R::kStep) {
      const uint8_t *pk = src.k, *pv = src.v;
#pragma unroll
      for (int j = 0; j < R::kStep / kRows; ++j) {
        if (inside(pk, pv)) {
          cp_async16(st + chunk_at<R::kRow>(lr + j * kRows, lc), pk, true);
          cp_async16(st + R::kTile + chunk_at<R::kRow>(lr + j * kRows, lc), pv, true);
        }
        pk += kRows * row_bytes;
        pv += kRows * row_bytes;
      }
    } else {  // a sequence's last block: rows past its end as zeros
#pragma unroll 1
      for (int j = 0; j < R::kStep / kRows; ++j) {
        const int r = lr + j * kRows;
        const long off = r < src.keys ? j * kRows * row_bytes : 0;
        const bool ok = r < src.keys && inside(src.k + off, src.v + off);
        cp_async16(st + chunk_at<R::kRow>(r, lc), ok ? src.k + off : static_cast<const uint8_t*>(p.k), ok);
        cp_async16(st + R::kTile + chunk_at<R::kRow>(r, lc), ok ? src.v + off : static_cast<const uint8_t*>(p.v), ok);
      }
    }
    if constexpr (F8) {
      const int r = lane % R::kStep;
      const bool ok = r < src.keys && inside_scales(src.ks, src.vs);
      cp_async4(st + 2 * R::kTile + 4 * r, ok ? src.ks : p.k_scale, ok);
      cp_async4(st + 2 * R::kTile + 4 * (R::kStep + r), ok ? src.vs : p.v_scale, ok);
      src.ks += kBlock;
      src.vs += kBlock;
    }
    src.k += kstride;
    src.v += kstride;
    src.keys -= kBlock;
    --src.left;
  };
  // q as B fragments: column n = lane / 4 of block nb is query row 8 nb + n.  16-bit: k index =
  // d; E4M3: k pairs 2c and 2c + 8 of step j are d = 16 j + 4 c + {0, 1} and {2, 3}, c = lane & 3
  uint32_t qf[NB][D / 16][2];
  auto load_q = [&](const Item& it) {
    const uint16_t* gq = static_cast<const uint16_t*>(p.q) + ((long)it.b * p.Hq + (long)hk * G) * D;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = 8 * nb + (lane >> 2), c = lane & 3;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        qf[nb][j][0] = qf[nb][j][1] = 0u;
        if (row < G && FA_IN_BOUNDS(p.status, (long)it.b * p.Hq + (long)hk * G + row, (long)p.B * p.Hq)) {
          const uint16_t* q0 = gq + (long)row * D + 16 * j;
          if constexpr (F8) {
            const uint2 w = *reinterpret_cast<const uint2*>(q0 + 4 * c);
            qf[nb][j][0] = w.x;
            qf[nb][j][1] = w.y;
          } else {
            qf[nb][j][0] = *reinterpret_cast<const uint32_t*>(q0 + 2 * c);
            qf[nb][j][1] = *reinterpret_cast<const uint32_t*>(q0 + 8 + 2 * c);
          }
        }
      }
    }
  };

  float* const solo_o = reinterpret_cast<float*>(smem + L::kOffSolo);
  float* const solo_lse = solo_o + 8 * NB * D;
  Item cur;
  bool have = next(cur);
  if (SOLO && !have && tid < G) solo_lse[tid] = -INFINITY;
  int c0 = 0;  // buffer of the current item's first block
  if (have) {
    aim(cur);
    if (cur.nblk > 0) load(0);
    cp_async_commit();
    load_q(cur);
  }
  while (have) {
    Item nxt;
    const bool more = next(nxt);

    float cq[NB][2];  // scale log2(e) of rows 8 nb + 2 c + {0, 1}, without q's power of two
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float unmul = 1.f;
      if constexpr (F8 && Elem<T>::kBf16) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = Elem<T>::unpack(qf[nb][j][e]);
            amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        amax = quad_max(amax);
        // exponent of amax, kept where both powers of two are normal numbers
        const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 126);
        const float mul = pow2(14 - ex);
        unmul = pow2(ex - 14);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = Elem<T>::unpack(qf[nb][j][e]);
            qf[nb][j][e] = Elem<__half>::pack(f.x * mul, f.y * mul);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        cq[nb][e] = p.scale * kLog2e * __shfl_sync(0xffffffffu, unmul, (2 * (lane & 3) + e) * 4);
    }

    // O^T: acc[nb][i] holds columns 16 i + .. of d (rows of the MMA) for query rows 2 c + {0, 1}
    float acc[NB][D / 16][4];
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nb][e] = -INFINITY;
        l[nb][e] = 0.f;
      }
    }
    constexpr float kLift = !F8 && !Elem<T>::kBf16 ? 8.f : 0.f;  // fp16 weights of a 16-bit cache
    int ev = kMinUnit;  // E4M3: 2^ev exceeds every V scale of this warp's keys so far

    for (int i = 0; i < max(cur.nblk, 1); ++i) {
      cp_async_wait<0>();
      __syncwarp();  // block i is there, and every lane is done with the block before it
      const int stage = (c0 + i) & 1;
      if (src.left == 0 && more) aim(nxt);
      if (src.left > 0) load(cur.nblk == 0 ? stage : stage ^ 1);
      cp_async_commit();
      if (cur.nblk == 0) break;
      const uint32_t st = ring + stage * R::kStage;
      const int key0 = cur.first + i * kBlock;

      float sc[MB][NB][4];  // keys 16 mb + lane / 4 + {0, 8}, rows 8 nb + 2 c + {0, 1}
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sc[mb][nb][0] = sc[mb][nb][1] = sc[mb][nb][2] = sc[mb][nb][3] = 0.f;
        if constexpr (F8) {
#pragma unroll
          for (int j = 0; j < D / 16; j += 2) {
            uint32_t r[4];
            ldsm_x4(st + chunk_at<R::kRow>(16 * mb + (lane & 15), j + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[4];
              e4m3x4_to_h2(r[2 * h], a[0], a[2]);
              e4m3x4_to_h2(r[2 * h + 1], a[1], a[3]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) mma16816<M>(sc[mb][nb], a, qf[nb][j + h][0], qf[nb][j + h][1]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            uint32_t a[4];
            ldsm_x4(st + chunk_at<R::kRow>(16 * mb + (lane & 15), 2 * j + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<M>(sc[mb][nb], a, qf[nb][j][0], qf[nb][j][1]);
          }
        }
      }
      float vs[MB][2];
      float vmax = 0.f;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ks = 1.f;
          vs[mb][e] = 1.f;
          if constexpr (F8) {
            const float* sp =
                reinterpret_cast<const float*>(ring_g + (st - ring) + 2 * R::kTile) + 16 * mb + 8 * e + (lane >> 2);
            ks = sp[0];
            vs[mb][e] = sp[R::kStep];
            vmax = fmaxf(vmax, vs[mb][e]);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            sc[mb][nb][2 * e] *= cq[nb][0] * ks;
            sc[mb][nb][2 * e + 1] *= cq[nb][1] * ks;
          }
        }
      if (key0 + R::kStep > cur.hi) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (key0 + 16 * mb + 8 * e + (lane >> 2) >= cur.hi) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) sc[mb][nb][2 * e] = sc[mb][nb][2 * e + 1] = -INFINITY;
            }
      }
      float mx[NB][2];
      bool grow = F8 && vmax >= pow2(ev);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nb][e] = fmaxf(sc[0][nb][e], sc[0][nb][2 + e]);
#pragma unroll
          for (int mb = 1; mb < MB; ++mb) mx[nb][e] = fmaxf(mx[nb][e], fmaxf(sc[mb][nb][e], sc[mb][nb][2 + e]));
          grow = grow || mx[nb][e] > m[nb][e] + kStale;
        }
      if (__any_sync(0xffffffffu, grow)) {
        float down = 1.f;
        if constexpr (F8) {  // the weights' unit grows: O follows
          const int en = max((int)(__float_as_uint(rows_max(vmax)) >> 23) - 126, ev);  // at most 129
          down = ev - en < -126 ? 0.f : pow2(ev - en);
          ev = en;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[nb][e], rows_max(mx[nb][e]));
            corr[e] = m[nb][e] == -INFINITY ? 0.f : ex2(m[nb][e] - mn);
            m[nb][e] = mn;
            l[nb][e] *= corr[e];
            corr[e] *= down;
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nb][k][e] *= corr[e & 1];
        }
      }
      // P^T as B fragments, and (REST) what their rounding left
      uint32_t pb[MB][NB][2], pr[MB][NB][2];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float vf = F8 ? vs[mb][e] * pow2(8 - ev) : 1.f;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float mu0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0] - kLift;
            const float mu1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1] - kLift;
            const float p0 = ex2(sc[mb][nb][2 * e] - mu0), p1 = ex2(sc[mb][nb][2 * e + 1] - mu1);
            l[nb][0] += p0;
            l[nb][1] += p1;
            const float w0 = F8 ? p0 * vf : p0, w1 = F8 ? p1 * vf : p1;
            const uint32_t hi = Elem<M>::pack(w0, w1);
            pb[mb][nb][e] = transpose8(hi);
            if constexpr (REST) {
              const float2 h = Elem<M>::unpack(hi);
              pr[mb][nb][e] = transpose8(Elem<M>::pack(w0 - h.x, w1 - h.y));
            }
          }
        }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if constexpr (F8) {
#pragma unroll
          for (int k = 0; k < D / 16; k += 2) {
            uint32_t r[4];  // keys 0-7 and 8-15 of 16-byte chunks k and k + 1
            ldsm_x4_t(st + R::kTile + chunk_at<R::kRow>(16 * mb + (lane & 15), k + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t a[4];
              e4m3x4_to_h2(__byte_perm(r[2 * h], 0, 0x3120), a[0], a[1]);
              e4m3x4_to_h2(__byte_perm(r[2 * h + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma16816<M>(acc[nb][k + h], a, pb[mb][nb][0], pb[mb][nb][1]);
                if constexpr (REST) mma16816<M>(acc[nb][k + h], a, pr[mb][nb][0], pr[mb][nb][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4];  // (keys, columns) halves in the order (0, 0), (0, 8), (8, 0), (8, 8)
            ldsm_x4_t(st + R::kTile + chunk_at<R::kRow>(16 * mb + (lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1)),
                      a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              mma16816<M>(acc[nb][k], a, pb[mb][nb][0], pb[mb][nb][1]);
              if constexpr (REST) mma16816<M>(acc[nb][k], a, pr[mb][nb][0], pr[mb][nb][1]);
            }
          }
        }
      }
    }
    c0 += cur.nblk;  // the next item's first block is in buffer c0 & 1 or on its way there
    if (more) load_q(nxt);

    // merge the four warps: each leaves O [8 NB][D] in its free buffer, m and l [4][8 NB], fp32
    __syncwarp();
    const uint32_t at = (warp * 2 + ((c0 & 1) ^ 1)) * R::kStage;
    float* const own = reinterpret_cast<float*>(smem + at);
    if (lane == 0) red_at[warp] = at;
    const float back = F8 ? pow2(ev - 8) : 1.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nb + 2 * (lane & 3) + e;
        const float ls = rows_sum(l[nb][e]);
        if (lane < 4) {
          red_m[warp * 8 * NB + row] = m[nb][e];
          red_l[warp * 8 * NB + row] = ls;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // MMA rows lane / 4 and lane / 4 + 8
          const int col0 = 16 * k + (F8 ? 2 * (lane >> 2) : (lane >> 2)), col1 = F8 ? col0 + 1 : col0 + 8;
          own[row * D + col0] = acc[nb][k][e] * back;
          own[row * D + col1] = acc[nb][k][2 + e] * back;
        }
      }
    __syncthreads();
    const long slots = (long)p.Hkv * (p.B + gridDim.x / p.Hkv);
    const long slot = (long)hk * (p.B + gridDim.x / p.Hkv) + cur.b + cta;
    const bool straight = !SOLO && NB == 1 && p.prefix_splits == 0 && cur.blk == 0 && cur.pos + cur.blks <= end;
    // whoever has a sequence's first block knows which CTAs have the others
    if (!SOLO && tid == 0 && cur.blk == 0 && hk == 0 && FA_IN_BOUNDS(p.status, cur.b, p.B))
      p.spans[cur.b] = make_int2(cta, (int)(((long long)(cur.pos + cur.blks) * C - 1) / W));
    for (int idx = 4 * tid; idx < G * D; idx += 4 * kThreads) {
      const int g = idx / D;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, red_m[w * 8 * NB + g]);
      const float mu = mx == -INFINITY ? 0.f : mx;  // every score -inf (l = 0) or NaN (l NaN)
      float lt = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // a warp with no finite score has l and O of 0 or NaN in any unit
        const float f = red_m[w * 8 * NB + g] == -INFINITY ? 1.f : ex2(red_m[w * 8 * NB + g] - mu);
        const float4 x = *reinterpret_cast<const float4*>(smem + red_at[w] + 4 * idx);
        lt += red_l[w * 8 * NB + g] * f;
        o.x += x.x * f;
        o.y += x.y * f;
        o.z += x.z * f;
        o.w += x.w * f;
      }
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      const float4 part = lt == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      const float lse = (mu - (mx == -INFINITY ? 0.f : kLift) + log2f(lt)) * kLn2;
      if constexpr (SOLO) {
        *reinterpret_cast<float4*>(solo_o + idx) = part;
        if (idx % D == 0) solo_lse[g] = lse;
      } else if (straight) {
        const long row = (long)cur.b * p.Hq + (long)hk * G + g;
        if (FA_IN_BOUNDS(p.status, row, (long)p.B * p.Hq)) {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + idx % D) =
              make_uint2(Elem<T>::pack(part.x, part.y), Elem<T>::pack(part.z, part.w));
          if (idx % D == 0) p.lse[row] = lse;
        }
      } else if (FA_IN_BOUNDS(p.status, slot, slots)) {
        *reinterpret_cast<float4*>(p.o_cache + slot * G * D + idx) = part;
        if (idx % D == 0) p.lse_cache[slot * G + g] = lse;
      }
    }
    __syncthreads();  // the free buffers may be loaded into again
    cur = nxt;
    have = more;
  }
  cp_async_wait<0>();
  if constexpr (SOLO) {
    if (p.after_prefix) asm volatile("griddepcontrol.wait;" ::: "memory");
    cluster_sync();
    const uint32_t so = smem_u32(solo_o), sl = smem_u32(solo_lse);
    for (int idx = 4 * (rank * kThreads + tid); idx < G * D; idx += 4 * kThreads * ranks) {
      const int g = idx / D, col = idx - g * D;
      const long row = (long)cta * p.Hq + (long)hk * G + g;
      if (!FA_IN_BOUNDS(p.status, row, (long)p.B * p.Hq)) continue;
      const float* const plse = p.lse_part + row * p.prefix_splits;
      const float* const po = p.o_part + row * p.prefix_splits * D + col;
      float mx = -INFINITY;
      for (int r = 0; r < ranks; ++r) mx = fmaxf(mx, cluster_load(cluster_addr(sl + 4 * g, r)));
      for (int i = 0; i < p.prefix_splits; ++i) mx = fmaxf(mx, plse[i]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float lse, float4 x) {
        const float w = ex2((lse - mu) * kLog2e);
        l += w;
        o.x += w * x.x;
        o.y += w * x.y;
        o.z += w * x.z;
        o.w += w * x.w;
      };
      for (int r = 0; r < ranks; ++r) {
        const float lse = cluster_load(cluster_addr(sl + 4 * g, r));
        if (lse != -INFINITY) add(lse, cluster_load4(cluster_addr(so + 4 * idx, r)));  // else nothing was left there
      }
#pragma unroll 4
      for (int i = 0; i < p.prefix_splits; ++i) add(plse[i], *reinterpret_cast<const float4*>(po + (long)i * D));
      const float inv = l == 0.f ? 0.f : 1.f / l;
      if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);  // no key: O = 0, LSE = -inf
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + col) =
          make_uint2(Elem<T>::pack(o.x * inv, o.y * inv), Elem<T>::pack(o.z * inv, o.w * inv));
      if (col == 0) p.lse[row] = mu + logf(l);
    }
    cluster_sync();  // no CTA leaves while another may read its shared memory
    return;
  }
  // after a prefix kernel this grid must not end before that one has, since the merge waits only for
  // this one
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Merge: WARPS warps per (h_q, b), each over every WARPS-th of the row's partials (the prefix's splits,
// then the cache's slots): the first kAhead of them, all loaded together, then one by one.
constexpr int combine_threads(int warps) { return warps > 4 ? 32 * warps : 128; }
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(combine_threads(WARPS)) cache_combine_kernel(CacheDecodeArgs p) {
  constexpr int kWarps = combine_threads(WARPS) / 32;
  __shared__ float red[kWarps][D];
  __shared__ float red_m[kWarps], red_l[kWarps];
  constexpr int kCols = D / 32;  // columns per lane
  constexpr int kAhead = WARPS <= 2 ? 8 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WARPS;
  const long row = (long)blockIdx.x * (kWarps / WARPS) + warp / WARPS;  // b Hq + h
  const long nrows = (long)p.B * p.Hq;
  if (WARPS == 1 && row >= nrows) return;
  bool any = row < nrows;  // (two warps a row: an odd number of rows leaves two without)
  const int Sp = p.prefix_splits, G = p.Hq / p.Hkv;
  const int b = (int)(row / p.Hq), h = (int)(row - (long)b * p.Hq), hk = h / G;
  const bool has = any && FA_IN_BOUNDS(p.status, b, p.B) && p.seqlens[any ? b : 0] > 0;
  // (no early start for what follows: the next pass's CTAs, taking their places among this kernel's,
  // came to lie unevenly on the SMs and cost 3 % of a long decode)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 span = has ? p.spans[b] : make_int2(0, -1);
  if (Sp == 0 && G <= 8 && span.x == span.y) any = false;  // one CTA had it whole
  if (WARPS == 1 && !any) return;
  const int live = any ? Sp + span.y - span.x + 1 : 0;
  const long slot0 = ((long)hk * (p.B + p.cache_ctas / p.Hkv) + b + span.x) * G + (h - hk * G);  // then G apart
  auto inside = [&](int s) {  // (of the checking build)
    const long slots = (long)p.Hkv * (p.B + p.cache_ctas / p.Hkv);
    return s < Sp ? FA_IN_BOUNDS(p.status, row * Sp + s, nrows * Sp)
                  : FA_IN_BOUNDS(p.status, slot0 + (long)(s - Sp) * G, slots * G);
  };
  auto lse_of = [&](int s) { return s < Sp ? p.lse_part[row * Sp + s] : p.lse_cache[slot0 + (long)(s - Sp) * G]; };
  auto load = [&](int s, float (&x)[kCols]) {
    const float* src =
        (s < Sp ? p.o_part + (row * Sp + s) * D : p.o_cache + (slot0 + (long)(s - Sp) * G) * D) + lane * kCols;
    if constexpr (D == 128) {
      const float4 f = *reinterpret_cast<const float4*>(src);
      x[0] = f.x;
      x[1] = f.y;
      x[2] = f.z;
      x[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(src);
      x[0] = f.x;
      x[1] = f.y;
    }
  };
  float lse[kAhead], x[kAhead][kCols];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int s = part + i * WARPS;
    lse[i] = -INFINITY;
#pragma unroll
    for (int c = 0; c < kCols; ++c) x[i][c] = 0.f;
    if (s < live && inside(s)) {
      lse[i] = lse_of(s);
      load(s, x[i]);
    }
  }
  float mx = lse[0];
#pragma unroll
  for (int i = 1; i < kAhead; ++i) mx = fmaxf(mx, lse[i]);
  float l = 0.f, o[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = 0.f;
  auto add = [&](float v, const float (&y)[kCols], float mu) {
    const float w = ex2((v - mu) * kLog2e);
    l += w;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] += w * y[c];
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) add(lse[i], x[i], mx == -INFINITY ? 0.f : mx);
  for (int s = part + kAhead * WARPS; s < live && inside(s); s += WARPS) {
    const float v = lse_of(s);
    load(s, x[0]);
    if (v > mx) {
      const float corr = mx == -INFINITY ? 1.f : ex2((mx - v) * kLog2e);  // l and O are 0 or NaN without a maximum
      mx = v;
      l *= corr;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] *= corr;
    }
    add(v, x[0], mx == -INFINITY ? 0.f : mx);
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) red[warp][lane * kCols + c] = o[c];
    if (lane == 0) {
      red_m[warp] = mx;
      red_l[warp] = l;
    }
    __syncthreads();
    const int first = warp - part;  // this row's warps: first .. first + WARPS - 1
    if (part > 0 || !any) return;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, red_m[first + w]);
    l = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; ++c) o[c] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float m = red_m[first + w], f = m == -INFINITY ? 1.f : ex2((m - mx) * kLog2e);
      l += f * red_l[first + w];
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[c] += f * red[first + w][lane * kCols + c];
    }
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int c = 0; c < kCols; ++c) o[c] = l == 0.f ? 0.f : o[c] * inv;  // no key: O = 0, LSE = -inf
  if (!FA_IN_BOUNDS(p.status, row, nrows)) return;
  uint32_t* go = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + lane * kCols);
#pragma unroll
  for (int c = 0; c < kCols / 2; ++c) go[c] = Elem<T>::pack(o[2 * c], o[2 * c + 1]);
  if (lane == 0) p.lse[row] = (mx == -INFINITY ? 0.f : mx) + logf(l);
}

template <typename T, int D, bool F8, int NB, bool REST>
cudaError_t launch_part(const CacheDecodeArgs& a, cudaStream_t s) {
  using L = Smem<D, F8, NB>;
  if (a.solo > 0) {
    auto kern = cache_decode_kernel<T, D, F8, NB, REST, true>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSoloBytes);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(kern, dim3(a.B * a.Hkv * a.solo), a.solo, kThreads, L::kSoloBytes, s, a);
  }
  auto kern = cache_decode_kernel<T, D, F8, NB, REST, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(a.cache_ctas), kThreads, L::kBytes, s, a);
}

template <typename T, int D, bool F8, bool REST>
cudaError_t launch_part_w(const CacheDecodeArgs& a, cudaStream_t s) {
  // groups of 9 to 16 query heads take two column blocks
  return a.Hq / a.Hkv > 8 ? launch_part<T, D, F8, 2, REST>(a, s) : launch_part<T, D, F8, 1, REST>(a, s);
}
template <typename T, int D>
cudaError_t launch_part_d(const CacheDecodeArgs& a, cudaStream_t s) {
  if (!a.k_scale) return launch_part_w<T, D, false, true>(a, s);
  if constexpr (!Elem<T>::kBf16) {
    if (a.B * (long)a.Hq <= kRestRows) return launch_part_w<T, D, true, true>(a, s);
  }
  return launch_part_w<T, D, true, false>(a, s);
}

template <typename T, int D>
cudaError_t launch_combine(const CacheDecodeArgs& a, cudaStream_t s) {
  const long rows = (long)a.B * a.Hq;
  // The more warps a row the more partials it may have, and the fewer rows there are to fill the SMs.  As
  // measured, us a call with 1, 2, 4 and 16 warps: 32 rows of 55 partials 32.7, 22.1, 20.1, 18.3; 512 of 4 47.4,
  // 47.4, 47.3, 49.0; 2048 of 12 57.1, 54.9, 54.3, 65.2; 8000 of 3 35.6, 39.0, 41.9, 78.9.
  const long parts = a.prefix_splits + a.cache_ctas / ((long)a.B * a.Hkv);
  const bool few = rows <= 4l * device_sm_count();
  const int warps = few ? (parts > 16 ? 16 : 4) : parts > 8 ? 2 : 1;
  const int per = combine_threads(warps) / 32 / warps;  // rows a CTA
  const long ctas = (rows + per - 1) / per;
  if (ctas > 0x7fffffffL) return cudaErrorInvalidValue;
  auto kern = warps == 16 ? cache_combine_kernel<T, D, 16>
              : warps == 4 ? cache_combine_kernel<T, D, 4>
              : warps == 2 ? cache_combine_kernel<T, D, 2>
                           : cache_combine_kernel<T, D, 1>;
  return launch_dependent(kern, dim3((unsigned)ctas), combine_threads(warps), 0, s, a);
}

}  // namespace

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t s) {
  if (a.bf16)
    return a.d == 128 ? launch_part_d<__nv_bfloat16, 128>(a, s)
                      : launch_part_d<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_part_d<__half, 128>(a, s) : launch_part_d<__half, 64>(a, s);
}

cudaError_t launch_cache_combine(const CacheDecodeArgs& a, cudaStream_t s) {
  if (a.bf16) return a.d == 128 ? launch_combine<__nv_bfloat16, 128>(a, s) : launch_combine<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_combine<__half, 128>(a, s) : launch_combine<__half, 64>(a, s);
}

}  // namespace fa
