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
// query rows share every byte the CTA reads.  Each of the four warps streams
// its own blocks of kStep keys through its own cp.async ring (no block barrier
// until the end) with its own running (m, l, O); the warps merge through shared
// memory.  Bound by HBM reads of the cache as long as the arithmetic per key is
// small, which shapes the rest:
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
constexpr int kMinUnit = -112;  // smallest e of the weights' unit (all powers of two below stay normal)

// Shape of a warp's ring: kStep keys a block, kStages blocks.  Two of 32 keys leave room for three CTAs
// on an SM (99 KB in flight); three of 32 were 2 % slower on 32768-key sequences and up to 30 % on
// short ones, three of 16 as fast there and 8 % slower here.  Persistent CTAs that load the next
// item's first block under the merge gained 3 % on 500-key sequences and cost 13 % on ragged long ones.
template <int D, bool F8>
struct Ring {
  static constexpr int kRow = D * (F8 ? 1 : 2);          // bytes of a K or V row
  static constexpr int kStep = kRow <= 128 ? 32 : 16;    // keys per block
  static constexpr int kStages = 2;
  static constexpr int kTile = kStep * kRow;
  static constexpr int kStage = 2 * kTile + (F8 ? 2 * kStep * 4 : 0);  // K, V, their scales
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kBlocks = kStep / 16;
};
template <int D, bool F8, int NB>
struct Smem {
  static constexpr int kRed = (4 * 8 * NB * (D + 2)) * 4;
  static constexpr int kBytes = 4 * Ring<D, F8>::kWarp > kRed ? 4 * Ring<D, F8>::kWarp : kRed;
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

template <typename T, int D, bool F8, int NB>
__global__ void __launch_bounds__(kThreads) cache_decode_kernel(CacheDecodeArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using R = Ring<D, F8>;
  using M = typename std::conditional<F8, __half, T>::type;  // MMA operand type
  constexpr int MB = R::kBlocks;
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
    const uint32_t ring = smem_u32(smem) + warp * R::kWarp;
    const uint8_t* const ring_g = smem + warp * R::kWarp;
    const long row_bytes = (long)p.Hkv * R::kRow;
    const long base = ((long)b * p.Nk_max * p.Hkv + hk) * R::kRow;
    const uint8_t* const gk = static_cast<const uint8_t*>(p.k) + base;
    const uint8_t* const gv = static_cast<const uint8_t*>(p.v) + base;
    const long sbase = ((long)b * p.Hkv + hk) * p.Nk_max;
    // this warp's blocks: keys lo + (4 i + warp) kStep ..
    const int first = lo + warp * R::kStep;
    const int nblk = first < hi ? (hi - first + 4 * R::kStep - 1) / (4 * R::kStep) : 0;

    constexpr int kC = R::kRow / 16, kRows = 32 / kC;  // chunks per row, rows per pass of the warp
    const int lr = lane / kC, lc = lane % kC;
    auto load = [&](int i) {
      const uint32_t st = ring + (i % R::kStages) * R::kStage;
      const int key0 = first + i * 4 * R::kStep;
      if (key0 + R::kStep <= hi) {
        const uint8_t* pk = gk + (long)(key0 + lr) * row_bytes + 16 * lc;
        const uint8_t* pv = gv + (long)(key0 + lr) * row_bytes + 16 * lc;
#pragma unroll
        for (int j = 0; j < R::kStep / kRows; ++j) {
          cp_async16(st + chunk_at<R::kRow>(lr + j * kRows, lc), pk, true);
          cp_async16(st + R::kTile + chunk_at<R::kRow>(lr + j * kRows, lc), pv, true);
          pk += kRows * row_bytes;
          pv += kRows * row_bytes;
        }
      } else {  // the last block: rows past hi as zeros
#pragma unroll 1
        for (int j = 0; j < R::kStep / kRows; ++j) {
          const int r = lr + j * kRows;
          const bool ok = key0 + r < hi;
          const long off = ok ? (long)(key0 + r) * row_bytes + 16 * lc : 0;
          cp_async16(st + chunk_at<R::kRow>(r, lc), gk + off, ok);
          cp_async16(st + R::kTile + chunk_at<R::kRow>(r, lc), gv + off, ok);
        }
      }
      if constexpr (F8) {
        const int r = lane % R::kStep;
        const bool ok = key0 + r < hi;
        cp_async4(st + 2 * R::kTile + 4 * r, p.k_scale + sbase + (ok ? key0 + r : 0), ok);
        cp_async4(st + 2 * R::kTile + 4 * (R::kStep + r), p.v_scale + sbase + (ok ? key0 + r : 0), ok);
      }
    };
#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) {
      if (i < nblk) load(i);
      cp_async_commit();
    }

    // q as B fragments: column n = lane / 4 of block nb is query row 8 nb + n.  16-bit: k index =
    // d; E4M3: k pairs 2c and 2c + 8 of step j are d = 16 j + 4 c + {0, 1} and {2, 3}, c = lane & 3
    const uint16_t* gq = static_cast<const uint16_t*>(p.q) + ((long)b * p.Hq + (long)hk * G) * D;
    uint32_t qf[NB][D / 16][2];
    float cq[NB][2];  // scale log2(e) of rows 8 nb + 2 c + {0, 1}, without q's power of two
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = 8 * nb + (lane >> 2), c = lane & 3;
      float mul = 1.f, unmul = 1.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        qf[nb][j][0] = qf[nb][j][1] = 0u;
        if (row < G) {
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
        mul = pow2(14 - ex);
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
        cq[nb][e] = p.scale * kLog2e * __shfl_sync(0xffffffffu, unmul, (2 * c + e) * 4);
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

    for (int i = 0; i < nblk; ++i) {
      cp_async_wait<R::kStages - 2>();
      __syncwarp();  // block i is there, and every lane is done with block i - 1
      if (i + R::kStages - 1 < nblk) load(i + R::kStages - 1);
      cp_async_commit();
      const uint32_t st = ring + (i % R::kStages) * R::kStage;
      const int key0 = first + i * 4 * R::kStep;

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
      if (key0 + R::kStep > hi) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (key0 + 16 * mb + 8 * e + (lane >> 2) >= hi) {
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
      uint32_t pb[MB][NB][2];  // P^T as B fragments
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
            pb[mb][nb][e] = transpose8(Elem<M>::pack(F8 ? p0 * vf : p0, F8 ? p1 * vf : p1));
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
              for (int nb = 0; nb < NB; ++nb) mma16816<M>(acc[nb][k + h], a, pb[mb][nb][0], pb[mb][nb][1]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4];  // (keys, columns) halves in the order (0, 0), (0, 8), (8, 0), (8, 8)
            ldsm_x4_t(st + R::kTile + chunk_at<R::kRow>(16 * mb + (lane & 7) + 8 * (lane >> 4), 2 * k + ((lane >> 3) & 1)),
                      a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<M>(acc[nb][k], a, pb[mb][nb][0], pb[mb][nb][1]);
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();

    // merge the four warps through shared memory: O [4][8 NB][D], m and l [4][8 NB], fp32
    float* red_o = reinterpret_cast<float*>(smem);
    float* red_m = red_o + 4 * 8 * NB * D;
    float* red_l = red_m + 4 * 8 * NB;
    const float back = F8 ? pow2(ev - 8) : 1.f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = warp * 8 * NB + 8 * nb + 2 * (lane & 3) + e;
        const float ls = rows_sum(l[nb][e]);
        if (lane < 4) {
          red_m[row] = m[nb][e];
          red_l[row] = ls;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // MMA rows lane / 4 and lane / 4 + 8
          const int c0 = 16 * k + (F8 ? 2 * (lane >> 2) : (lane >> 2)), c1 = F8 ? c0 + 1 : c0 + 8;
          red_o[row * D + c0] = acc[nb][k][e] * back;
          red_o[row * D + c1] = acc[nb][k][2 + e] * back;
        }
      }
    __syncthreads();
    const long nparts = (long)p.B * p.Hq * S;
    const long part0 = ((long)b * p.Hq + (long)hk * G) * S + p.prefix_splits + s;
    for (int idx = tid; idx < G * D; idx += kThreads) {
      const int g = idx / D, col = idx % D;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, red_m[w * 8 * NB + g]);
      const float mu = mx == -INFINITY ? 0.f : mx;  // every score -inf (l = 0) or NaN (l NaN)
      float lt = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // a warp with no finite score has l and O of 0 or NaN in any unit
        const float f = red_m[w * 8 * NB + g] == -INFINITY ? 1.f : ex2(red_m[w * 8 * NB + g] - mu);
        lt += red_l[w * 8 * NB + g] * f;
        o += red_o[(w * 8 * NB + g) * D + col] * f;
      }
      const long oi = part0 + (long)g * S;
      if (FA_IN_BOUNDS(p.status, oi, nparts)) {
        p.o_part[oi * D + col] = lt == 0.f ? 0.f : o / lt;
        if (col == 0) p.lse_part[oi] = (mu - (mx == -INFINITY ? 0.f : kLift) + log2f(lt)) * kLn2;
      }
    }
  }
  // launched as a programmatic dependent of the prefix kernel: this grid must not end before that
  // one has, since the merge waits only for this one (without the launch attribute the wait
  // returns at once)
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Merge: WARPS warps per (h_q, b), each over its share of the live splits.  Every warp first takes
// all splits' LSE (a lane each, 32 at a time) to the shared maximum; the sums' loads then do not
// depend on one another.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(kThreads) cache_combine_kernel(CacheDecodeArgs p) {
  __shared__ float red[4][D];
  __shared__ float red_l[4];
  constexpr int kCols = D / 32;  // columns per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WARPS;
  const long row = (long)blockIdx.x * (4 / WARPS) + warp / WARPS;  // b Hq + h
  const long nrows = (long)p.B * p.Hq;
  const int S = p.prefix_splits + p.num_splits;
  int n = 0;
  if (row < nrows) n = p.seqlens[row / p.Hq];
  n = n < 0 ? 0 : (n > p.Nk_max ? p.Nk_max : n);
  int live = p.prefix_splits + (n + p.chunk - 1) / p.chunk;
  const long base = row * S;
  if (!(row < nrows && FA_IN_BOUNDS(p.status, base + S - 1, nrows * S))) live = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float mx = -INFINITY;
  for (int s = lane; s < live; s += 32) mx = fmaxf(mx, p.lse_part[base + s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float l = 0.f;
  float o[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) o[i] = 0.f;
#pragma unroll 8
  for (int s = part; s < live; s += WARPS) {
    const float w = ex2((p.lse_part[base + s] - mu) * kLog2e);
    const float* src = p.o_part + (base + s) * D + lane * kCols;
    float x[kCols];
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
    l += w;
#pragma unroll
    for (int i = 0; i < kCols; ++i) o[i] += w * x[i];
  }
  if constexpr (WARPS == 4) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) red[warp][lane * kCols + i] = o[i];
    if (lane == 0) red_l[warp] = l;
    __syncthreads();
    if (warp > 0) return;
    l = (red_l[0] + red_l[1]) + (red_l[2] + red_l[3]);
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int col = lane * kCols + i;
      o[i] = (red[0][col] + red[1][col]) + (red[2][col] + red[3][col]);
    }
  }
  if (row >= nrows) return;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < kCols; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;  // no key: O = 0, LSE = -inf
  uint32_t* go = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + lane * kCols);
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) go[i] = Elem<T>::pack(o[2 * i], o[2 * i + 1]);
  if (lane == 0) p.lse[row] = mu + logf(l);
}

template <typename T, int D, bool F8, int NB>
cudaError_t launch_part(const CacheDecodeArgs& a, int after_prefix, cudaStream_t s) {
  auto kern = cache_decode_kernel<T, D, F8, NB>;
  constexpr int smem = Smem<D, F8, NB>::kBytes;
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
  const bool wide = a.Hq / a.Hkv > 8;  // groups of 9 to 16 query heads take two column blocks
  if (a.k_scale) return wide ? launch_part<T, D, true, 2>(a, after_prefix, s) : launch_part<T, D, true, 1>(a, after_prefix, s);
  return wide ? launch_part<T, D, false, 2>(a, after_prefix, s) : launch_part<T, D, false, 1>(a, after_prefix, s);
}

template <typename T, int D>
cudaError_t launch_combine(const CacheDecodeArgs& a, cudaStream_t s) {
  const long rows = (long)a.B * a.Hq;
  // four warps a row for many splits or few rows
  const bool four = a.prefix_splits + a.num_splits > 8 || rows < 4l * device_sm_count();
  const long blocks = four ? rows : (rows + 3) / 4;
  if (blocks > 0x7fffffffL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, four ? cache_combine_kernel<T, D, 4> : cache_combine_kernel<T, D, 1>, a);
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
