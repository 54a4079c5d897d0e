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
// sines once, and applies them to up to kHeads heads, whose loads it issues
// together.
#include <math.h>

#include "common.cuh"
#include "serving.h"

namespace fa {
namespace {

constexpr int kThreads = 128;

struct Params {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  const int* positions;
  const unsigned long long* turns;
  long tokens;  // B N
  int N, Hq, Hkv, rot;
  long q_bs, q_ts, k_bs, k_ts, pos_stride;
  long q_len, k_len;  // elements from q (k) to the end of its last row
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

// grid: (token groups, head groups); a warp covers 32 / (D / 16) heads of one token at a time.
template <typename T, int D, bool INTER, int HEADS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Params p) {
  constexpr int kUnits = D / 16;         // threads per head, 16 values each
  constexpr int kRow = 32 / kUnits;      // heads per warp and step
  const int lane = threadIdx.x & 31;
  const long tok = (long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.tokens) return;
  const int unit = lane % kUnits;
  const int h0 = blockIdx.y * (kRow * HEADS) + lane / kUnits;
  const int H = p.Hq + p.Hkv;
  const long b = tok / p.N, n = tok % p.N;
  const int units_rot = p.rot / 16;
  const bool turned = unit < units_rot;
  // first and second 8-value chunk of this thread within a head
  const int c0 = INTER || !turned ? 16 * unit : 8 * unit;
  const int c1 = INTER || !turned ? 16 * unit + 8 : p.rot / 2 + 8 * unit;

  const uint16_t* src[HEADS];
  uint16_t* dst[HEADS];
  uint4 w0[HEADS], w1[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i * kRow;
    const bool isq = h < p.Hq;
    const long in = isq ? b * p.q_bs + n * p.q_ts + (long)h * D : b * p.k_bs + n * p.k_ts + (long)(h - p.Hq) * D;
    const long out = (isq ? tok * p.Hq + h : tok * p.Hkv + (h - p.Hq)) * D;
    bool ok = h < H;
    ok = ok && FA_IN_BOUNDS(p.status, in + D - 1, isq ? p.q_len : p.k_len) &&
         FA_IN_BOUNDS(p.status, out + D - 1, p.tokens * (isq ? p.Hq : p.Hkv) * D);
    src[i] = ok ? (isq ? p.q : p.k) + in : nullptr;
    dst[i] = (isq ? p.qo : p.ko) + out;
    if (src[i]) {
      w0[i] = *reinterpret_cast<const uint4*>(src[i] + c0);
      w1[i] = *reinterpret_cast<const uint4*>(src[i] + c1);
    }
  }
  if (!turned) {
#pragma unroll
    for (int i = 0; i < HEADS; ++i)
      if (src[i]) {
        *reinterpret_cast<uint4*>(dst[i] + c0) = w0[i];
        *reinterpret_cast<uint4*>(dst[i] + c1) = w1[i];
      }
    return;
  }
  const long long pos = p.positions[b * p.pos_stride + n];
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const unsigned long long phase = (unsigned long long)pos * p.turns[8 * unit + j];
    const float half_turns = (float)(int)(phase >> 32) * 0x1p-31f;  // in [-1, 1]
    sincospif(half_turns, &sn[j], &cs[j]);
    sn[j] *= p.sign * p.mag;
    cs[j] *= p.mag;
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i)
    if (src[i]) {
      float x[8], y[8], u[8], v[8];
      load8<T>(x, w0[i]);
      load8<T>(y, w1[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // pair j: (x[j], y[j]), or neighbours within the two chunks
        const float a = INTER ? (j < 4 ? x[(2 * j) & 7] : y[(2 * j) & 7]) : x[j];
        const float c = INTER ? (j < 4 ? x[(2 * j + 1) & 7] : y[(2 * j + 1) & 7]) : y[j];
        u[j] = fmaf(a, cs[j], -c * sn[j]);
        v[j] = fmaf(c, cs[j], a * sn[j]);
      }
      if constexpr (INTER) {
        *reinterpret_cast<uint4*>(dst[i] + c0) =
            make_uint4(Elem<T>::pack(u[0], v[0]), Elem<T>::pack(u[1], v[1]), Elem<T>::pack(u[2], v[2]),
                       Elem<T>::pack(u[3], v[3]));
        *reinterpret_cast<uint4*>(dst[i] + c1) =
            make_uint4(Elem<T>::pack(u[4], v[4]), Elem<T>::pack(u[5], v[5]), Elem<T>::pack(u[6], v[6]),
                       Elem<T>::pack(u[7], v[7]));
      } else {
        *reinterpret_cast<uint4*>(dst[i] + c0) = pack8<T>(u);
        *reinterpret_cast<uint4*>(dst[i] + c1) = pack8<T>(v);
      }
    }
}

template <typename T, int D, bool INTER, int HEADS>
cudaError_t launch(const Params& p, cudaStream_t s) {
  constexpr int kRow = 32 / (D / 16);
  const long groups = (p.tokens + kThreads / 32 - 1) / (kThreads / 32);
  if (groups > 0x7fffffffL) return cudaErrorInvalidValue;
  dim3 grid((unsigned)groups, (p.Hq + p.Hkv + kRow * HEADS - 1) / (kRow * HEADS));
  rotary_kernel<T, D, INTER, HEADS><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const RotaryArgs& a, const Params& p, cudaStream_t s) {
  return a.interleaved ? launch<T, D, true, 2>(p, s) : launch<T, D, false, 2>(p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  Params p{static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.k), static_cast<uint16_t*>(a.q_out),
           static_cast<uint16_t*>(a.k_out), a.positions, a.turns, (long)a.B * a.N, a.N, a.Hq, a.Hkv, a.rot,
           a.q_bs, a.q_ts, a.k_bs, a.k_ts, a.pos_stride,
           (a.B - 1) * a.q_bs + (a.N - 1) * a.q_ts + (long)a.Hq * a.d,
           (a.B - 1) * a.k_bs + (a.N - 1) * a.k_ts + (long)a.Hkv * a.d, a.magnitude, a.inverse ? -1.f : 1.f, a.status};
  if (a.bf16) return a.d == 128 ? launch_d<__nv_bfloat16, 128>(a, p, s) : launch_d<__nv_bfloat16, 64>(a, p, s);
  return a.d == 128 ? launch_d<__half, 128>(a, p, s) : launch_d<__half, 64>(a, p, s);
}

}  // namespace fa
