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

// One row in D / 16 consecutive threads, 16 values each.
template <typename T, int D>
__device__ __forceinline__ void encode(const uint4 (&w)[2], uint8_t* codes, float* scale, int unit) {
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
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(__fdiv_rn(x[4 * i], s), __fdiv_rn(x[4 * i + 1], s)) |
           (e4m3x2(__fdiv_rn(x[4 * i + 2], s), __fdiv_rn(x[4 * i + 3], s)) << 16);
  if (codes) {
    *reinterpret_cast<uint4*>(codes + 16 * unit) = make_uint4(c[0], c[1], c[2], c[3]);
    if (unit == 0) *scale = s;
  }
}

// grid: (row groups, 2); y = 0 appends K rows, 1 V rows.  Row r = (b n + i) Hkv + h.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(Fp8CacheArgs p) {
  constexpr int kUnits = D / 16;
  const bool isv = blockIdx.y != 0;
  const long rows = (long)p.B * p.n * p.Hkv;
  const long r = (long)blockIdx.x * (kThreads / kUnits) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  uint8_t* codes = nullptr;
  float* scale = nullptr;
  uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (r < rows) {
    const int h = (int)(r % p.Hkv);
    const long bi = r / p.Hkv;
    const int i = (int)(bi % p.n), b = (int)(bi / p.n);
    const long dst = (long)p.start[b] + i;
    if (i < (p.counts ? p.counts[b] : p.n) && dst >= 0 && dst < p.Nk_max) {
      const long bs = isv ? p.v_bs : p.k_bs, ts = isv ? p.v_ts : p.k_ts;
      const long in = b * bs + i * ts + (long)h * D;
      const long crow = ((long)b * p.Nk_max + dst) * p.Hkv + h;
      const long srow = ((long)b * p.Hkv + h) * p.Nk_max + dst;
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
  encode<T, D>(w, codes, scale, unit);
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

// grid: (row groups, 2).  Rows at or past a sequence's length come out as zeros.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(Fp8CacheArgs p) {
  constexpr int kUnits = D / 16;
  const bool isv = blockIdx.y != 0;
  const long rows = (long)p.B * p.n * p.Hkv;
  const long r = (long)blockIdx.x * (kThreads / kUnits) + threadIdx.x / kUnits;
  const int unit = threadIdx.x % kUnits;
  if (r >= rows) return;
  const int h = (int)(r % p.Hkv);
  const long bi = r / p.Hkv;
  const int i = (int)(bi % p.n), b = (int)(bi / p.n);
  uint4 w[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (i < p.counts[b]) {
    const long crow = ((long)b * p.Nk_max + i) * p.Hkv + h;
    const long srow = ((long)b * p.Hkv + h) * p.Nk_max + i;
    if (FA_IN_BOUNDS(p.status, crow, (long)p.B * p.Nk_max * p.Hkv) &&
        FA_IN_BOUNDS(p.status, srow, (long)p.B * p.Nk_max * p.Hkv))
      decode16<T>(reinterpret_cast<const uint4*>((isv ? p.v8 : p.k8) + crow * D)[unit],
                  (isv ? p.v_scale : p.k_scale)[srow], w);
  }
  if (FA_IN_BOUNDS(p.status, r, rows)) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(isv ? p.v_out : p.k_out) + r * D) + 2 * unit;
    dst[0] = w[0];
    dst[1] = w[1];
  }
}

template <typename T, int D>
cudaError_t launch_append(const Fp8CacheArgs& a, cudaStream_t s) {
  const long rows = (long)a.B * a.n * a.Hkv, per = kThreads / (D / 16), groups = (rows + per - 1) / per;
  if (groups > 0x7fffffffL) return cudaErrorInvalidValue;
  append_kernel<T, D><<<dim3((unsigned)groups, 2), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_read(const Fp8CacheArgs& a, cudaStream_t s) {
  const long rows = (long)a.B * a.n * a.Hkv, per = kThreads / (D / 16), groups = (rows + per - 1) / per;
  if (groups > 0x7fffffffL) return cudaErrorInvalidValue;
  read_kernel<T, D><<<dim3((unsigned)groups, 2), kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
