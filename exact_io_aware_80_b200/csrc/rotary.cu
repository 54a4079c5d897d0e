// rotary.cu -- rotary position embedding of queries and keys, and its
// transpose for the backward pass.
//
// Each head's first `rot` values are pairs, (x[i], x[i + rot/2]) in the half
// layout or (x[2i], x[2i+1]) in the interleaved one, and pair i of a token at
// position p is turned by the angle p f_i and scaled by m:
//   y0 = m (x0 cos - x1 sin),  y1 = m (x1 cos + x0 sin);
// values past `rot` are copied.  The map is linear and orthogonal up to m, so
// the gradient with respect to x is the same map with the angle negated.
//
// The angle.  p f_i reaches 1e6 radians in long contexts, where an fp32 product
// is off by 0.06.  The caller's table holds u_i = f_i / (2 pi) turns per
// position as a 64-bit fraction of one turn, so p u_i mod 2^64 (one integer
// multiplication that wraps) is the phase with every whole turn removed, exact
// to |p| 2^-65 turns; its top 32 bits, signed, go to sincospif.
//
// Bound by HBM: every element is read and written once.  A thread takes 8
// pairs of one token (two 16-byte chunks: chunks j and j + rot/16 of the head
// in the half layout, 2j and 2j + 1 in the interleaved one), computes their
// sines once, and applies them to one head after another, kBatch heads' loads
// at a time.  Measured: 8192 tokens of 40 heads of 128, 168 MB, 28.0 us, 6.0 TB/s
// or 0.92 of a plain copy; 64 tokens, 2.3 us.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 128;

struct Params {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  const int* positions;
  const unsigned long long* turns;
  uint32_t tokens;  // B N < 2^31
  FastDiv N;
  int Hq, Hkv, rot;
  int per_y;  // heads per grid row
  long q_bs, q_ts, k_bs, k_ts, pos_stride;
  long q_len, k_len;  // elements from q (k) to the end of its last row
  long pos_len;       // positions
  float mag, sign;
  int* status;
};

template <typename T>
__device__ __forceinline__ void load8(float (&x)[8], const uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::unpack(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]), Elem<T>::pack(x[4], x[5]),
                    Elem<T>::pack(x[6], x[7]));
}

// The rotation of one thread's 8 pairs; cosines and sines as pairs of neighbouring j.
template <typename T, bool INTER>
__device__ __forceinline__ void turn(uint4& w0, uint4& w1, const float2 (&cs)[4], const float2 (&sn)[4]) {
  float x[8], y[8];
  load8<T>(x, w0);
  load8<T>(y, w1);
  float u[8], v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // pairs 2j and 2j + 1: (x[.], y[.]), or neighbours within the two chunks
    float2 a, c;
    if constexpr (INTER) {
      const float* z = j < 2 ? x : y;
      a = make_float2(z[4 * (j & 1)], z[4 * (j & 1) + 2]);
      c = make_float2(z[4 * (j & 1) + 1], z[4 * (j & 1) + 3]);
    } else {
      a = make_float2(x[2 * j], x[2 * j + 1]);
      c = make_float2(y[2 * j], y[2 * j + 1]);
    }
    const float2 ns = make_float2(-sn[j].x, -sn[j].y);
    const float2 r0 = __ffma2_rn(a, cs[j], __fmul2_rn(c, ns));
    const float2 r1 = __ffma2_rn(c, cs[j], __fmul2_rn(a, sn[j]));
    u[2 * j] = r0.x;
    u[2 * j + 1] = r0.y;
    v[2 * j] = r1.x;
    v[2 * j + 1] = r1.y;
  }
  if constexpr (INTER) {
    w0 = make_uint4(Elem<T>::pack(u[0], v[0]), Elem<T>::pack(u[1], v[1]), Elem<T>::pack(u[2], v[2]),
                    Elem<T>::pack(u[3], v[3]));
    w1 = make_uint4(Elem<T>::pack(u[4], v[4]), Elem<T>::pack(u[5], v[5]), Elem<T>::pack(u[6], v[6]),
                    Elem<T>::pack(u[7], v[7]));
  } else {
    w0 = pack8<T>(u);
    w1 = pack8<T>(v);
  }
}

// grid: (token groups, head groups); a warp covers 32 / (D / 16) heads of one token at a time.
template <typename T, int D, bool INTER, int BATCH>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Params p) {
  constexpr int kUnits = D / 16;     // threads per head, 16 values each
  constexpr int kRow = 32 / kUnits;  // heads per warp and step
  wait_for_earlier_grids();
  const int lane = threadIdx.x & 31;
  const uint32_t tok = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.tokens) return;
  const int unit = lane % kUnits;
  const int H = p.Hq + p.Hkv;
  const uint32_t b = p.N(tok), n = tok - b * p.N.d;
  const bool turned = unit < p.rot / 16;
  // first and second 8-value chunk of this thread within a head
  const int c0 = INTER || !turned ? 16 * unit : 8 * unit;
  const int c1 = INTER || !turned ? 16 * unit + 8 : p.rot / 2 + 8 * unit;
  const long q_in = b * p.q_bs + n * p.q_ts, k_in = b * p.k_bs + n * p.k_ts;
  const long q_out = (long)tok * p.Hq * D, k_out = (long)tok * p.Hkv * D;
  const int h_end = min(H, (int)(blockIdx.y + 1) * p.per_y);

  float2 cs[4], sn[4];
  bool have = false;
  for (int h0 = blockIdx.y * p.per_y + lane / kUnits; h0 < h_end; h0 += kRow * BATCH) {
    uint4 w0[BATCH], w1[BATCH];
    uint16_t* dst[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = h0 + i * kRow;
      const bool isq = h < p.Hq;
      const long in = isq ? q_in + h * D : k_in + (h - p.Hq) * D;
      const long out = isq ? q_out + h * D : k_out + (h - p.Hq) * D;
      const bool ok = h < h_end && FA_IN_BOUNDS(p.status, in + D - 1, isq ? p.q_len : p.k_len) &&
                      FA_IN_BOUNDS(p.status, out + D - 1, (long)p.tokens * (isq ? p.Hq : p.Hkv) * D);
      dst[i] = ok ? (isq ? p.qo : p.ko) + out : nullptr;
      if (ok) {
        const uint16_t* src = (isq ? p.q : p.k) + in;
        w0[i] = *reinterpret_cast<const uint4*>(src + c0);
        w1[i] = *reinterpret_cast<const uint4*>(src + c1);
      }
    }
    if (turned && !have) {  // while the first batch is in flight
      have = true;
      const long at = b * p.pos_stride + n;
      const long long pos = FA_IN_BOUNDS(p.status, at, p.pos_len) ? p.positions[at] : 0;
      auto angle = [&](int j, float* sine, float* cosine) {
        const unsigned long long phase = (unsigned long long)pos * p.turns[8 * unit + j];
        sincospif((float)(int)(phase >> 32) * 0x1p-31f, sine, cosine);  // half turns in [-1, 1]
        *sine *= p.sign * p.mag;
        *cosine *= p.mag;
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        angle(2 * j, &sn[j].x, &cs[j].x);
        angle(2 * j + 1, &sn[j].y, &cs[j].y);
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i)
      if (dst[i]) {
        if (turned) turn<T, INTER>(w0[i], w1[i], cs, sn);
        *reinterpret_cast<uint4*>(dst[i] + c0) = w0[i];
        *reinterpret_cast<uint4*>(dst[i] + c1) = w1[i];
      }
  }
}

template <typename T, int D, bool INTER>
cudaError_t launch(const RotaryArgs& a, Params p, cudaStream_t s) {
  // the half layout's 128-byte stretches gain from four heads in flight (8192 tokens, 40 heads: 28.0 us,
  // 29.9 with two), the interleaved layout does not (8192 tokens, 32 heads: 23.0, 22.4 with two)
  constexpr int kRow = 32 / (D / 16), kBatch = INTER ? 2 : 4;
  const unsigned groups = (p.tokens + kThreads / 32 - 1) / (kThreads / 32);
  const int H = a.Hq + a.Hkv;
  // a warp takes all heads of its token, or fewer where there are too few tokens to fill the SMs
  const int steps = (H + kRow * kBatch - 1) / (kRow * kBatch);
  const long want = 16l * device_sm_count();  // thread blocks
  const int rows = (int)std::min<long>(steps, std::max<long>(1, want / groups));
  p.per_y = (steps + rows - 1) / rows * (kRow * kBatch);
  const dim3 grid(groups, (H + p.per_y - 1) / p.per_y);
  return launch_dependent(rotary_kernel<T, D, INTER, kBatch>, grid, kThreads, 0, s, p);
}

template <typename T, int D>
cudaError_t launch_d(const RotaryArgs& a, const Params& p, cudaStream_t s) {
  return a.interleaved ? launch<T, D, true>(a, p, s) : launch<T, D, false>(a, p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  Params p{static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k), static_cast<uint16_t*>(a.q_out),
           static_cast<uint16_t*>(a.k_out), a.positions, a.turns, (uint32_t)a.B * a.N, FastDiv(a.N), a.Hq, a.Hkv, a.rot, 0,
           a.q_bs, a.q_ts, a.k_bs, a.k_ts, a.pos_stride,
           (a.B - 1) * a.q_bs + (a.N - 1) * a.q_ts + (long)a.Hq * a.d,
           (a.B - 1) * a.k_bs + (a.N - 1) * a.k_ts + (long)a.Hkv * a.d, (a.B - 1) * a.pos_stride + a.N, a.magnitude, a.inverse ? -1.f : 1.f, a.status};
  if (a.bf16) return a.d == 128 ? launch_d<__nv_bfloat16, 128>(a, p, s) : launch_d<__nv_bfloat16, 64>(a, p, s);
  return a.d == 128 ? launch_d<__half, 128>(a, p, s) : launch_d<__half, 64>(a, p, s);
}

}  // namespace fa
