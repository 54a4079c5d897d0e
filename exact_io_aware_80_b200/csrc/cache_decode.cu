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
// Partial pass: one CTA per (split, KV head, sequence).  The group's Hq / Hkv
// query rows (padded to the 16-row MMA shape) share every byte the CTA reads.
// Tiles of 64 keys stream through a cp.async ring; each of the four warps takes
// 16 keys of a tile with its own running (m, l, O), merged through shared
// memory at the end.  Bound by HBM reads of the cache.
//
// E4M3 operands.  E4M3 values are exact in fp16, so codes are converted in
// registers (cvt.rn.f16x2.e4m3x2) and multiplied as m16n8k16 fp16 products:
//  * K: the four threads of a key's row read 16 consecutive codes each; the
//    order in which the MMA's k index runs over d is free as long as q follows
//    it, so q is loaded in the same order.
//  * V: the transposing ldmatrix moves 16-bit units, here two neighbouring
//    columns of one key; a byte permutation per register gives the key pairs of
//    either column, so an n8 block of the MMA holds every second column.
//  * q in bf16 is scaled by a power of two per row that brings its largest
//    value to [2^14, 2^15): conversion to fp16 is then exact for every element
//    within 2^-30 of the row's largest and off by at most 2^-39 of it below.
//  * the weights p_j s^v_j are fp16 in units of 2^(e - 14), where 2^e exceeds
//    every s^v seen so far: at most 2^14, relative error 2^-11 down to 2^-28 of
//    the unit's largest, absolute 2^-39 of it below.  l sums the unrounded p_j.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kTileN = 64;  // keys per tile
constexpr int kStages = 3;
constexpr int kRows = 16;  // MMA rows: the group's query heads, zero-padded

// Byte offset of 16-byte chunk `c` of key row `r` in a tile of E4M3 rows of D bytes.  Chunks are
// permuted so that both the K reads (two rows x four chunks per quarter-warp) and the V reads
// (ldmatrix: one chunk of eight rows) touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk8(int r, int c) {
  if constexpr (D == 128)
    return r * 128 + ((c ^ (((r & 1) << 2) | ((r >> 1) & 3))) << 4);
  else
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D>
__device__ __forceinline__ void load_codes_async(uint32_t smem, const uint8_t* g, int row0, int nrows, long ld,
                                                 int tid) {
  constexpr int kC = D / 16;
#pragma unroll
  for (int e = tid; e < kTileN * kC; e += kThreads) {
    const int r = e / kC, c = e % kC;
    const bool ok = row0 + r < nrows;
    cp_async16(smem + chunk8<D>(r, c), g + (ok ? (long)(row0 + r) * ld + 16 * c : 0), ok);
  }
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}

// Two E4M3 codes (low byte first) as an fp16 pair; exact.
__device__ __forceinline__ uint32_t e4m3_to_h2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_to_h2_hi(uint32_t four) { return e4m3_to_h2(four >> 16); }

// q's rows lane / 4 and lane / 4 + 8 as fp16 A fragments in the order of the K codes: MMA step
// 4 g + i of 16-key-column group g takes, for the thread with c = lane & 3, columns
// 64 g + 16 c + 4 i .. + 3.  Returns 2^-k of the power of two each row was multiplied by.
template <typename T, int D>
__device__ __forceinline__ void load_q8(uint32_t (&qf)[D / 16][4], float (&unscale)[2], const uint16_t* gq, int G,
                                        int lane) {
  const int c = lane & 3;
  float x[2][D / 4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = (lane >> 2) + 8 * e;
    float amax = 0.f;
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (r < G) w = *reinterpret_cast<const uint4*>(gq + (long)r * D + 64 * g + 16 * c + 8 * k);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = Elem<T>::unpack(u[i]);
          x[e][16 * g + 8 * k + 2 * i] = f.x;
          x[e][16 * g + 8 * k + 2 * i + 1] = f.y;
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
    amax = quad_max(amax);
    float mul = 1.f;
    unscale[e] = 1.f;
    if constexpr (Elem<T>::kBf16) {
      // exponent of amax, kept where both powers of two are normal numbers
      int ex = (int)(__float_as_uint(amax) >> 23) - 127;
      ex = min(max(ex, -100), 126);
      mul = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
      unscale[e] = __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
    }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) x[e][i] *= mul;
  }
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const int i = 4 * s;
    qf[s][0] = Elem<__half>::pack(x[0][i], x[0][i + 1]);
    qf[s][1] = Elem<__half>::pack(x[1][i], x[1][i + 1]);
    qf[s][2] = Elem<__half>::pack(x[0][i + 2], x[0][i + 3]);
    qf[s][3] = Elem<__half>::pack(x[1][i + 2], x[1][i + 3]);
  }
}

template <typename T, int D, bool F8>
struct Smem {
  static constexpr int kTile = kTileN * D * (F8 ? 1 : 2);
  static constexpr int kScales = F8 ? 2 * kTileN * 4 : 0;
  static constexpr int kStage = 2 * kTile + kScales;  // K, V, then their scales
  static constexpr int kOffStage = F8 ? 0 : kRows * D * 2;  // 16-bit: q first
  static constexpr int kPipe = kOffStage + kStages * kStage;
  static constexpr int kRed = kOffStage + (4 * kRows * D + 8 * kRows) * 4;
  static constexpr int kBytes = kPipe > kRed ? kPipe : kRed;
};

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kThreads) cache_decode_kernel(CacheDecodeArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using L = Smem<T, D, F8>;
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int G = p.Hq / p.Hkv;
  const int S = p.prefix_splits + p.num_splits;
  int n = p.seqlens[b];
  n = n < 0 ? 0 : (n > p.Nk_max ? p.Nk_max : n);
  const int lo = s * p.chunk;
  const int hi = min(lo + p.chunk, n);
  // the merge, launched next as a programmatic dependent, may become resident; it waits for this
  // grid's end before it reads a partial
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (hi > lo) {
    const int ntiles = (hi - lo + kTileN - 1) / kTileN;
    const long ldk = (long)p.Hkv * D;
    const uint16_t* gq = static_cast<const uint16_t*>(p.q) + ((long)b * p.Hq + (long)hk * G) * D;
    const long base = ((long)b * p.Nk_max * p.Hkv + hk) * D;
    const long sbase = ((long)b * p.Hkv + hk) * p.Nk_max;

    auto load_tile = [&](int t) {
      const uint32_t st = sb + L::kOffStage + (t % kStages) * L::kStage;
      if constexpr (F8) {
        load_codes_async<D>(st, static_cast<const uint8_t*>(p.k) + base, lo + t * kTileN, hi, ldk, tid);
        load_codes_async<D>(st + L::kTile, static_cast<const uint8_t*>(p.v) + base, lo + t * kTileN, hi, ldk, tid);
        const int r = tid & 63, key = lo + t * kTileN + r;
        const bool ok = key < hi;
        const float* src = tid < 64 ? p.k_scale : p.v_scale;
        cp_async4(st + 2 * L::kTile + tid * 4, src + sbase + (ok ? key : 0), ok);
      } else {
        load_tile_async<kTileN, D, kThreads>(st, static_cast<const uint16_t*>(p.k) + base, lo + t * kTileN, hi, ldk,
                                             tid);
        load_tile_async<kTileN, D, kThreads>(st + L::kTile, static_cast<const uint16_t*>(p.v) + base, lo + t * kTileN,
                                             hi, ldk, tid);
      }
    };
    if constexpr (!F8) load_tile_async<kRows, D, kThreads>(sb, gq, 0, G, D, tid);
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) {
      if (t < ntiles) load_tile(t);
      cp_async_commit();
    }

    using M = typename std::conditional<F8, __half, T>::type;  // MMA operand type
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY};
    float l_run[2] = {0.f, 0.f};
    uint32_t qf[D / 16][4];
    float c[2] = {p.scale * kLog2e, p.scale * kLog2e};
    if constexpr (F8) {
      float un[2];
      load_q8<T, D>(qf, un, gq, G, lane);
      c[0] *= un[0];
      c[1] *= un[1];
    }
    int ev = -112;  // E4M3: 2^ev exceeds every V scale of this warp's keys so far

    for (int t = 0; t < ntiles; ++t) {
      if (t + kStages - 1 < ntiles) load_tile(t + kStages - 1);
      cp_async_commit();
      cp_async_wait<kStages - 1>();
      __syncthreads();
      const uint32_t st = sb + L::kOffStage + (t % kStages) * L::kStage;
      if constexpr (!F8) {
        if (t == 0) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) frag_a<kRows>(qf[kk], sb, 0, kk * 16, lane);
        }
      }
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if constexpr (F8) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int g = 0; g < D / 64; ++g) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(st + chunk8<D>(warp * 16 + nb * 8 + (lane >> 2), 4 * g + (lane & 3))));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma16816<M>(sc[nb], qf[4 * g + i], e4m3_to_h2(w[i]), e4m3_to_h2_hi(w[i]));
          }
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t bb[4];
          frag_b_nk<kTileN>(bb, st, warp * 16, kk * 16, lane);
          mma16816<M>(sc[0], qf[kk], bb[0], bb[1]);
          mma16816<M>(sc[1], qf[kk], bb[2], bb[3]);
        }
      }
      // scores in log2 units; this thread's keys are 8 nb + 2 (lane & 3) + {0, 1} of the warp's 16
      float vsc[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
      const int key0 = lo + t * kTileN + warp * 16;
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        float ks[2] = {1.f, 1.f};
        if constexpr (F8) {
          const int kc = warp * 16 + 8 * nb + 2 * (lane & 3);
          const float* sp = reinterpret_cast<const float*>(smem + (st - sb) + 2 * L::kTile);
          const float2 k2 = *reinterpret_cast<const float2*>(sp + kc);
          const float2 v2 = *reinterpret_cast<const float2*>(sp + kTileN + kc);
          ks[0] = k2.x;
          ks[1] = k2.y;
          vsc[nb][0] = v2.x;
          vsc[nb][1] = v2.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nb][e] *= c[e >> 1] * ks[e & 1];
          if (key0 + 8 * nb + 2 * (lane & 3) + (e & 1) >= hi) sc[nb][e] = -INFINITY;
        }
      }
      float corr[2], mu[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float rm = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]), fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
        const float mnew = fmaxf(m_run[e], quad_max(rm));
        mu[e] = (mnew == -INFINITY) ? 0.f : mnew;
        corr[e] = ex2(m_run[e] - mu[e]);
        m_run[e] = mnew;
        l_run[e] *= corr[e];
      }
      float vf[2][2] = {{1.f, 1.f}, {1.f, 1.f}};  // weight of p_j: s^v_j in units of 2^(ev - 14)
      if constexpr (F8) {
        const float vm = quad_max(fmaxf(fmaxf(vsc[0][0], vsc[0][1]), fmaxf(vsc[1][0], vsc[1][1])));
        const int en = max((int)(__float_as_uint(fmaxf(vm, 0.f)) >> 23) - 126, ev);  // at most 129
        if (en > ev) {  // the unit grows: O follows
          const float down = ev - en < -126 ? 0.f : __uint_as_float((uint32_t)(ev - en + 127) << 23);
          corr[0] *= down;
          corr[1] *= down;
          ev = en;
        }
        const float unit = __uint_as_float((uint32_t)(14 - ev + 127) << 23);
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          vf[nb][0] = vsc[nb][0] * unit;
          vf[nb][1] = vsc[nb][1] * unit;
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const float p0 = ex2(sc[nb][0] - mu[0]), p1 = ex2(sc[nb][1] - mu[0]);
        const float p2 = ex2(sc[nb][2] - mu[1]), p3 = ex2(sc[nb][3] - mu[1]);
        l_run[0] += p0 + p1;
        l_run[1] += p2 + p3;
        pa[nb * 2 + 0] = Elem<M>::pack(p0 * vf[nb][0], p1 * vf[nb][1]);
        pa[nb * 2 + 1] = Elem<M>::pack(p2 * vf[nb][0], p3 * vf[nb][1]);
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] *= corr[e >> 1];
      if constexpr (F8) {
        // matrices of one ldmatrix.x4: keys 0-7 and 8-15 of 16-byte chunks 2 np and 2 np + 1
#pragma unroll
        for (int np = 0; np < D / 32; ++np) {
          uint32_t r[4];
          const int row = warp * 16 + (lane & 15);
          ldsm_x4_t(st + L::kTile + chunk8<D>(row, 2 * np + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // chunk 2 np + k: columns 16 (2 np + k) + {even, odd}
            const uint32_t a = __byte_perm(r[2 * k], 0, 0x3120), bq = __byte_perm(r[2 * k + 1], 0, 0x3120);
            mma16816<M>(acc[4 * np + 2 * k], pa, e4m3_to_h2(a), e4m3_to_h2(bq));
            mma16816<M>(acc[4 * np + 2 * k + 1], pa, e4m3_to_h2_hi(a), e4m3_to_h2_hi(bq));
          }
        }
      } else {
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
          uint32_t bb[4];
          frag_b_kn<kTileN>(bb, st + L::kTile, warp * 16, np * 16, lane);
          mma16816<M>(acc[2 * np], pa, bb[0], bb[1]);
          mma16816<M>(acc[2 * np + 1], pa, bb[2], bb[3]);
        }
      }
      __syncthreads();
    }
    cp_async_wait<0>();
    __syncthreads();

    // merge the four warps: per warp m[16], l[16], O[16][D] (fp32) in the stage buffers
    float* red_o = reinterpret_cast<float*>(smem + L::kOffStage);  // [4][16][D]
    float* red_m = red_o + 4 * kRows * D;                          // [4][16]
    float* red_l = red_m + 4 * kRows;                              // [4][16]
    const int r0 = lane >> 2;
    const float back = F8 ? __uint_as_float((uint32_t)(ev - 14 + 127) << 23) : 1.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float l = quad_sum(l_run[e]);
      if ((lane & 3) == 0) {
        red_m[warp * kRows + r0 + 8 * e] = m_run[e];
        red_l[warp * kRows + r0 + 8 * e] = l;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      // E4M3: block i holds the even (odd) columns of 16-byte chunk i / 2
      const int c0 = F8 ? 16 * (i >> 1) + (i & 1) + 4 * (lane & 3) : 8 * i + 2 * (lane & 3);
      const int c1 = F8 ? c0 + 2 : c0 + 1;
      float* o0 = red_o + (warp * kRows + r0) * D;
      float* o1 = red_o + (warp * kRows + r0 + 8) * D;
      o0[c0] = acc[i][0] * back;
      o0[c1] = acc[i][1] * back;
      o1[c0] = acc[i][2] * back;
      o1[c1] = acc[i][3] * back;
    }
    __syncthreads();
    const long nparts = (long)p.B * p.Hq * S;
    const long part0 = ((long)b * p.Hq + (long)hk * G) * S + p.prefix_splits + s;
    for (int idx = tid; idx < G * D; idx += kThreads) {
      const int g = idx / D, col = idx % D;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, red_m[w * kRows + g]);
      const float mu = mx == -INFINITY ? 0.f : mx;  // every score -inf (l = 0) or NaN (l NaN)
      float l = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(red_m[w * kRows + g] - mu);
        l += red_l[w * kRows + g] * f;
        o += red_o[(w * kRows + g) * D + col] * f;
      }
      const long oi = part0 + (long)g * S;
      if (FA_IN_BOUNDS(p.status, oi, nparts)) {
        p.o_part[oi * D + col] = l == 0.f ? 0.f : o / l;
        if (col == 0) p.lse_part[oi] = (mu + log2f(l)) * kLn2;
      }
    }
  }
  // launched as a programmatic dependent of the prefix kernel: this grid must not end before that
  // one has, since the merge waits only for this one (without the launch attribute the wait
  // returns at once)
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Merge: one CTA per (h_q, b), its four warps each over a quarter of the live splits.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) cache_combine_kernel(CacheDecodeArgs p) {
  __shared__ float red[4][D];
  __shared__ float red_m[4], red_l[4];
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.prefix_splits + p.num_splits;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int n = p.seqlens[b];
  n = n < 0 ? 0 : (n > p.Nk_max ? p.Nk_max : n);
  const int live = p.prefix_splits + (n + p.chunk - 1) / p.chunk;
  const long base = ((long)b * p.Hq + h) * S;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  if (FA_IN_BOUNDS(p.status, base + S - 1, (long)p.B * p.Hq * S)) {
    for (int s = warp; s < live; s += 4) {
      const float x = p.lse_part[base + s] * kLog2e;
      const float mn = fmaxf(m, x);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const float corr = ex2(m - mu), w = ex2(x - mu);
      m = mn;
      l = l * corr + w;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = o[i] * corr + w * p.o_part[(base + s) * D + i * 32 + lane];
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) red[warp][i * 32 + lane] = o[i];
  if (lane == 0) {
    red_m[warp] = m;
    red_l[warp] = l;
  }
  __syncthreads();
  const int col = threadIdx.x;
  if (col >= D) return;
  const float mx = fmaxf(fmaxf(red_m[0], red_m[1]), fmaxf(red_m[2], red_m[3]));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float lt = 0.f, ot = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = ex2(red_m[w] - mu);
    lt += red_l[w] * f;
    ot += red[w][col] * f;
  }
  const long row = (long)b * p.Hq + h;
  const float out = lt == 0.f ? 0.f : ot / lt;  // no key: O = 0, LSE = -inf
  uint16_t* go = static_cast<uint16_t*>(p.o) + row * D;
  T v;
  if constexpr (Elem<T>::kBf16) v = __float2bfloat16_rn(out); else v = __float2half_rn(out);
  if (FA_IN_BOUNDS(p.status, row, (long)p.B * p.Hq)) {
    go[col] = *reinterpret_cast<uint16_t*>(&v);
    if (col == 0) p.lse[row] = (mu + log2f(lt)) * kLn2;
  }
}

template <typename T, int D, bool F8>
cudaError_t launch_part(const CacheDecodeArgs& a, int after_prefix, cudaStream_t s) {
  auto kern = cache_decode_kernel<T, D, F8>;
  constexpr int smem = Smem<T, D, F8>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.num_splits, a.Hkv, a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  if (after_prefix) {
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int D>
cudaError_t launch_part_d(const CacheDecodeArgs& a, int after_prefix, cudaStream_t s) {
  return a.k_scale ? launch_part<T, D, true>(a, after_prefix, s) : launch_part<T, D, false>(a, after_prefix, s);
}

template <typename T, int D>
cudaError_t launch_combine(const CacheDecodeArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.Hq, a.B);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_combine_kernel<T, D>, a);
}

}  // namespace

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, int after_prefix, cudaStream_t s) {
  if (a.bf16)
    return a.d == 128 ? launch_part_d<__nv_bfloat16, 128>(a, after_prefix, s)
                      : launch_part_d<__nv_bfloat16, 64>(a, after_prefix, s);
  return a.d == 128 ? launch_part_d<__half, 128>(a, after_prefix, s) : launch_part_d<__half, 64>(a, after_prefix, s);
}

cudaError_t launch_cache_combine(const CacheDecodeArgs& a, cudaStream_t s) {
  if (a.bf16) return a.d == 128 ? launch_combine<__nv_bfloat16, 128>(a, s) : launch_combine<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_combine<__half, 128>(a, s) : launch_combine<__half, 64>(a, s);
}

}  // namespace fa
