// fp8_cache.cu -- rows of a key/value cache held as E4M3 codes: quantised as
// they are written, and read back as 16-bit values.
//
// A row is one head of one token (d values).  s = amax / 448 (1 for a row of
// zeros), code = E4M3(x / s) with IEEE fp32 divisions, round to nearest even:
// the rule of fp8_quant.cu with a block of one row, since rows that enter a
// cache one token at a time cannot share a scale without being rewritten.  A
// row that holds a NaN gets the scale NaN, one that holds an infinity the scale
// infinity, and both read back as NaN throughout.
//
// Codes [B, Nk_max, Hkv, d]; scales [B, Hkv, Nk_max], keys innermost, so that a
// decode CTA, which reads consecutive keys of one head, finds its scales in one
// stretch.
//
// Bound by HBM: 2 d bytes in and d + 4 out per appended row, d + 4 in and 2 d
// out per row read back.  A thread takes 16 values (two 16-byte loads, one
// 16-byte store of codes), so d / 16 threads hold a row and its maximum is
// log2(d / 16) shuffles.  Measured: 64000 tokens of 8 heads of 128 appended, 397
// MB, 66.5 us, 6.0 TB/s or 0.92 of a plain copy; 24003 tokens, a third of them
// past their counts, of 8 heads of 64, 50 MB, 10.5 us, 4.8 TB/s, where the issue
// slots that the exact quotients take weigh more; 65536 tokens of 8 heads of 128 read
// back, 407 MB, 62 to 69 us with where the buffers lie, 6.6 to 5.9 TB/s.
#include "common.cuh"
#include "kernels.h"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Maximum that a NaN in either argument turns into NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The same of pairs of 16-bit values, which are compared as they are.
template <typename T>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (Elem<T>::kBf16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Row r = (b n + i) Hkv + h of the 16-bit tensors.
struct Rows {
  uint32_t count;  // < 2^31
  FastDiv n, Hkv;
};
struct Row {
  uint32_t b, i, h;
};
__device__ __forceinline__ Row row_at(const Rows& rows, uint32_t r) {
  const uint32_t bi = rows.Hkv(r), b = rows.n(bi);
  return Row{b, bi - b * rows.n.d, r - bi * rows.Hkv.d};
}

// E4M3 codes of 16 values x / s, given as n = -x.  FAST, for 2^-90 <= s <= 2^90: a quotient is y = x r
// with r = RN(1 / s), corrected once by its own remainder, q = y - (y s - x) r, which is RN(x / s) as
// long as nothing leaves the normal range (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990).  Quotients small enough to leave it have the code +-0 either way,
// and taken in this order the remainder of an exact quotient is +0, so that -0 keeps its sign.
template <bool FAST>
__device__ __forceinline__ uint4 codes16(const float2 (&n)[8], float s) {
  const float r = __frcp_rn(s);
  uint32_t half[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 q;
    if constexpr (FAST) {
      const float2 y = __fmul2_rn(n[i], make_float2(-r, -r));
      const float2 rem = __ffma2_rn(y, make_float2(s, s), n[i]);
      q = __ffma2_rn(rem, make_float2(-r, -r), y);
    } else {
      q = make_float2(__fdiv_rn(-n[i].x, s), __fdiv_rn(-n[i].y, s));
    }
    half[i] = e4m3x2(q.x, q.y);
  }
  return make_uint4(half[0] | (half[1] << 16), half[2] | (half[3] << 16), half[4] | (half[5] << 16),
                    half[6] | (half[7] << 16));
}

// D / 16 consecutive threads hold a row.  TENSORS = 2: K's and V's, which share the arithmetic of its place;
// 1: one of them, by blockIdx.y.
template <typename T, int D, int TENSORS>
__global__ void __launch_bounds__(kThreads) append_kernel(Fp8CacheArgs p, Rows rows) {
  wait_for_earlier_grids();
  constexpr int kUnits = D / 16;
  const uint32_t r = blockIdx.x * (kThreads / kUnits) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  auto is_v = [&](int t) { return TENSORS == 2 ? t != 0 : blockIdx.y != 0; };
  long crow = -1, srow = 0;  // places of the codes and of the scale
  uint4 w[TENSORS][2] = {};
  if (r < rows.count) {
    const Row at = row_at(rows, r);
    const bool known = FA_IN_BOUNDS(p.status, at.b, p.B);
    const long dst = known ? (long)p.start[at.b] + at.i : -1;
    if (known && (int)at.i < (p.counts ? p.counts[at.b] : p.n) && dst >= 0 && dst < p.Nk_max) {
      const long c = ((long)at.b * p.Nk_max + dst) * p.Hkv + at.h;
      srow = ((long)at.b * p.Hkv + at.h) * p.Nk_max + dst;
      if (FA_IN_BOUNDS(p.status, c, (long)p.B * p.Nk_max * p.Hkv) &&
          FA_IN_BOUNDS(p.status, srow, (long)p.B * p.Nk_max * p.Hkv))
        crow = c;
#pragma unroll
      for (int t = 0; t < TENSORS; ++t) {
        const long bs = is_v(t) ? p.v_bs : p.k_bs, ts = is_v(t) ? p.v_ts : p.k_ts;
        const long in = at.b * bs + at.i * ts + (long)(at.h * D);
        if (FA_IN_BOUNDS(p.status, in + D - 1, (p.B - 1) * bs + (p.n - 1) * ts + (long)p.Hkv * D)) {
          const uint4* src =
              reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_v(t) ? p.v : p.k) + in) + 2 * unit;
          w[t][0] = src[0];
          w[t][1] = src[1];
        } else {
          crow = -1;
        }
      }
    }
  }
  // rows past their counts (a third of three prompts of up to 8001 tokens: 10.5 us with this, 10.8 without)
  if (!__any_sync(0xffffffffu, crow >= 0)) return;
#pragma unroll
  for (int t = 0; t < TENSORS; ++t) {
    const uint32_t u[8] = {w[t][0].x, w[t][0].y, w[t][0].z, w[t][0].w, w[t][1].x, w[t][1].y, w[t][1].z, w[t][1].w};
    uint32_t most = u[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) most = max2_nan<T>(most, u[i] & 0x7FFF7FFFu);
    const float2 both = Elem<T>::unpack(most);
    float amax = max_nan(both.x, both.y);
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f);
    float2 n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = Elem<T>::unpack(u[i] ^ 0x80008000u);
    if (crow >= 0) {
      reinterpret_cast<uint4*>((is_v(t) ? p.v8 : p.k8) + crow * D)[unit] =
          s >= 0x1p-90f && s <= 0x1p90f ? codes16<true>(n, s) : codes16<false>(n, s);
      if (unit == 0) (is_v(t) ? p.v_scale : p.k_scale)[srow] = s;
    }
  }
}

// 8 E4M3 codes times s, as a 16-byte vector of T.
template <typename T>
__device__ __forceinline__ uint4 decode8(const uint2 c, float s) {
  const uint32_t u[2] = {c.x, c.y};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(u[i >> 1] >> (16 * (i & 1)))));
    const float2 f = Elem<__half>::unpack(h2);
    w[i] = Elem<T>::pack(f.x * s, f.y * s);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// grid: (row groups, 2).  Rows at or past a sequence's length come out as zeros.  A thread takes 8 codes
// (so that a warp's 16-byte stores are one stretch) of ROWS rows, whose loads it issues together.
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kThreads) read_kernel(Fp8CacheArgs p, Rows rows) {
  wait_for_earlier_grids();
  constexpr int kUnits = D / 8, kPer = kThreads / kUnits;
  const bool isv = blockIdx.y != 0;
  const uint32_t r0 = blockIdx.x * (kPer * ROWS) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  uint2 c[ROWS];
  float s[ROWS];
  bool live[ROWS];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const uint32_t r = r0 + k * kPer;
    live[k] = false;
    if (r < rows.count) {
      const Row at = row_at(rows, r);
      if (FA_IN_BOUNDS(p.status, at.b, p.B) && (int)at.i < p.counts[at.b]) {
        const long crow = ((long)at.b * p.Nk_max + at.i) * p.Hkv + at.h;
        const long srow = ((long)at.b * p.Hkv + at.h) * p.Nk_max + at.i;
        if (FA_IN_BOUNDS(p.status, crow, (long)p.B * p.Nk_max * p.Hkv) &&
            FA_IN_BOUNDS(p.status, srow, (long)p.B * p.Nk_max * p.Hkv)) {
          live[k] = true;
          c[k] = reinterpret_cast<const uint2*>((isv ? p.v8 : p.k8) + crow * D)[unit];
          s[k] = (isv ? p.v_scale : p.k_scale)[srow];
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const uint32_t r = r0 + k * kPer;
    if (r < rows.count && FA_IN_BOUNDS(p.status, (long)r * D + 8 * unit + 7, (long)p.B * p.n * p.Hkv * D))
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(isv ? p.v_out : p.k_out) + (long)r * D)[unit] =
          live[k] ? decode8<T>(c[k], s[k]) : make_uint4(0u, 0u, 0u, 0u);
  }
}

Rows rows_of(const Fp8CacheArgs& a) { return Rows{(uint32_t)a.B * a.n * a.Hkv, FastDiv(a.n), FastDiv(a.Hkv)}; }

template <typename T, int D>
cudaError_t launch_append(const Fp8CacheArgs& a, cudaStream_t s) {
  const Rows rows = rows_of(a);
  const uint32_t per = kThreads / (D / 16), groups = (rows.count + per - 1) / per;
  // 64000 tokens of 8 heads of 128: 66.5 us with K and V in a thread, 75.6 apart; 2048: 3.9 and 3.6; 64: 2.1 and 1.7
  if (groups < 4u * device_sm_count())
    return launch_dependent(append_kernel<T, D, 1>, dim3(groups, 2), kThreads, 0, s, a, rows);
  return launch_dependent(append_kernel<T, D, 2>, dim3(groups), kThreads, 0, s, a, rows);
}
template <typename T, int D, int ROWS>
cudaError_t launch_read_rows(const Fp8CacheArgs& a, const Rows& rows, cudaStream_t s) {
  const uint32_t per = kThreads / (D / 8) * ROWS;
  return launch_dependent(read_kernel<T, D, ROWS>, dim3((rows.count + per - 1) / per, 2), kThreads, 0, s, a, rows);
}
template <typename T, int D>
cudaError_t launch_read(const Fp8CacheArgs& a, cudaStream_t s) {
  const Rows rows = rows_of(a);
  // 134 MB of codes: 61.9 us with four rows a thread, 81.5, 66.4 and 67.2 with one, two and eight; one where
  // four would leave SMs idle
  const bool few = (long)rows.count * (D / 8) < 4l * kThreads * device_sm_count();
  return few ? launch_read_rows<T, D, 1>(a, rows, s) : launch_read_rows<T, D, 4>(a, rows, s);
}

}  // namespace

cudaError_t launch_fp8_cache_append(const Fp8CacheArgs& a, cudaStream_t s) {
  if (a.bf16) return a.d == 128 ? launch_append<__nv_bfloat16, 128>(a, s) : launch_append<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_append<__half, 128>(a, s) : launch_append<__half, 64>(a, s);
}
cudaError_t launch_fp8_cache_read(const Fp8CacheArgs& a, cudaStream_t s) {
  if (a.bf16) return a.d == 128 ? launch_read<__nv_bfloat16, 128>(a, s) : launch_read<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_read<__half, 128>(a, s) : launch_read<__half, 64>(a, s);
}

}  // namespace fa
