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
// log2(d / 16) shuffles.
#include "common.cuh"
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

// E4M3 codes of 16 values x / s.  For 2^-90 <= s <= 2^90 a quotient is y = x r with r = RN(1 / s),
// corrected once by its own remainder: q = y + (x - y s) r, which is RN(x / s) as long as nothing
// leaves the normal range (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Quotients small enough to leave it have the code +-0 either way;
// -0 alone loses its sign in the correction and takes y's.  Other scales divide.
template <bool FAST>
__device__ __forceinline__ uint4 codes16(const float (&x)[16], float s) {
  const float r = __frcp_rn(s);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t half[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float2 v = make_float2(x[4 * i + 2 * k], x[4 * i + 2 * k + 1]);
      float2 q;
      if constexpr (FAST) {
        const float2 y = __fmul2_rn(v, make_float2(r, r));
        const float2 rem = __ffma2_rn(y, make_float2(-s, -s), v);
        q = __ffma2_rn(rem, make_float2(r, r), y);
        q.x = __uint_as_float(__float_as_uint(q.x) | (__float_as_uint(y.x) & 0x80000000u));
        q.y = __uint_as_float(__float_as_uint(q.y) | (__float_as_uint(y.y) & 0x80000000u));
      } else {
        q = make_float2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s));
      }
      half[k] = e4m3x2(q.x, q.y);
    }
    c[i] = half[0] | (half[1] << 16);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// grid: (row groups, 2); y = 0 appends K rows, 1 V rows.  D / 16 consecutive threads hold a row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(Fp8CacheArgs p, Rows rows) {
  wait_for_earlier_grids();
  constexpr int kUnits = D / 16;
  const bool isv = blockIdx.y != 0;
  const uint32_t r = blockIdx.x * (kThreads / kUnits) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  uint8_t* codes = nullptr;
  float* scale = nullptr;
  uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (r < rows.count) {
    const Row at = row_at(rows, r);
    const long dst = (long)p.start[at.b] + at.i;
    if ((int)at.i < (p.counts ? p.counts[at.b] : p.n) && dst >= 0 && dst < p.Nk_max) {
      const long bs = isv ? p.v_bs : p.k_bs, ts = isv ? p.v_ts : p.k_ts;
      const long in = at.b * bs + at.i * ts + (long)(at.h * D);
      const long crow = ((long)at.b * p.Nk_max + dst) * p.Hkv + at.h;
      const long srow = ((long)at.b * p.Hkv + at.h) * p.Nk_max + dst;
      if (FA_IN_BOUNDS(p.status, in + D - 1, (p.B - 1) * bs + (p.n - 1) * ts + (long)p.Hkv * D) &&
          FA_IN_BOUNDS(p.status, crow, (long)p.B * p.Nk_max * p.Hkv) &&
          FA_IN_BOUNDS(p.status, srow, (long)p.B * p.Nk_max * p.Hkv)) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(isv ? p.v : p.k) + in) + 2 * unit;
        w[0] = src[0];
        w[1] = src[1];
        codes = (isv ? p.v8 : p.k8) + crow * D;
        scale = (isv ? p.v_scale : p.k_scale) + srow;
      }
    }
  }
  const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  float x[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = Elem<T>::unpack(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(x[i]));
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = amax == 0.f ? 1.f : __fdiv_rn(amax, 448.f);
  if (codes) {
    *reinterpret_cast<uint4*>(codes + 16 * unit) =
        s >= 0x1p-90f && s <= 0x1p90f ? codes16<true>(x, s) : codes16<false>(x, s);
    if (unit == 0) *scale = s;
  }
}

// 16 E4M3 codes times s, as two 16-byte vectors of T.
template <typename T>
__device__ __forceinline__ void decode16(const uint4 c, float s, uint4 (&out)[2]) {
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(u[i] >> (16 * k))));
      const float2 f = Elem<__half>::unpack(h2);
      w[2 * i + k] = Elem<T>::pack(f.x * s, f.y * s);
    }
  }
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// grid: (row groups, 2).  Rows at or past a sequence's length come out as zeros.  A thread takes 16
// codes of kReadRows rows, whose loads it issues together.
constexpr int kReadRows = 2;
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Fp8CacheArgs p, Rows rows) {
  wait_for_earlier_grids();
  constexpr int kUnits = D / 16, kPer = kThreads / kUnits;
  const bool isv = blockIdx.y != 0;
  const uint32_t r0 = blockIdx.x * (kPer * kReadRows) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  uint4 c[kReadRows];
  float s[kReadRows];
  bool live[kReadRows];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    const uint32_t r = r0 + k * kPer;
    live[k] = false;
    if (r < rows.count) {
      const Row at = row_at(rows, r);
      if ((int)at.i < p.counts[at.b]) {
        const long crow = ((long)at.b * p.Nk_max + at.i) * p.Hkv + at.h;
        const long srow = ((long)at.b * p.Hkv + at.h) * p.Nk_max + at.i;
        if (FA_IN_BOUNDS(p.status, crow, (long)p.B * p.Nk_max * p.Hkv) &&
            FA_IN_BOUNDS(p.status, srow, (long)p.B * p.Nk_max * p.Hkv)) {
          live[k] = true;
          c[k] = reinterpret_cast<const uint4*>((isv ? p.v8 : p.k8) + crow * D)[unit];
          s[k] = (isv ? p.v_scale : p.k_scale)[srow];
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    const uint32_t r = r0 + k * kPer;
    if (r < rows.count && FA_IN_BOUNDS(p.status, r, rows.count)) {
      uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (live[k]) decode16<T>(c[k], s[k], w);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(isv ? p.v_out : p.k_out) + (long)r * D) + 2 * unit;
      dst[0] = w[0];
      dst[1] = w[1];
    }
  }
}

Rows rows_of(const Fp8CacheArgs& a) { return Rows{(uint32_t)a.B * a.n * a.Hkv, FastDiv(a.n), FastDiv(a.Hkv)}; }

template <typename T, int D>
cudaError_t launch_append(const Fp8CacheArgs& a, cudaStream_t s) {
  const Rows rows = rows_of(a);
  const uint32_t per = kThreads / (D / 16);
  return launch_dependent(append_kernel<T, D>, dim3((rows.count + per - 1) / per, 2), kThreads, 0, s, a, rows);
}
template <typename T, int D>
cudaError_t launch_read(const Fp8CacheArgs& a, cudaStream_t s) {
  const Rows rows = rows_of(a);
  const uint32_t per = kThreads / (D / 16) * kReadRows;
  return launch_dependent(read_kernel<T, D>, dim3((rows.count + per - 1) / per, 2), kThreads, 0, s, a, rows);
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
