// serving.h -- host-side launchers of the rotary, E4M3-cache and cache-decode
// kernels (internal to libfa.so).  Arguments are validated in serving_api.cu
// before any launcher runs.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace fa {

// Device status word of the current device (fa_api.cu), nullptr if it cannot be found.
int* device_status_word();

// 4-D tensor map with 128-byte swizzle (tma.cu): dims innermost first, strides of dims 1..3 in
// bytes; the box's innermost extent must be 128 bytes.
constexpr int kMapF16 = 0, kMapBf16 = 1, kMapF32 = 2;
bool make_map_box(CUtensorMap* m, const void* base, int type, const uint64_t dims[4], const uint64_t strides[3],
                  const uint32_t box[4]);

// Division of n < 2^31 by a fixed d >= 1: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// floor(n / d) = (mulhi(n, m) + n) >> l (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994; the sum stays below 2^32 for these n).
struct FastDiv {
  uint32_t d, m, l;
  explicit FastDiv(uint32_t div = 1) : d(div), l(0) {
    while ((1ull << l) < d) ++l;
    m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, m) + n) >> l; }
#endif
};

// Launch as a programmatic dependent of whatever precedes on the stream: the grid may become
// resident before that has finished, and orders itself behind it (and behind all before it) with
// griddepcontrol.wait ahead of its first access to global memory.
template <typename... Params, typename... Args>
cudaError_t launch_dependent_clusters(void (*kern)(Params...), dim3 grid, int cluster, int threads, int smem,
                                      cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, Args&&... args) {
  return launch_dependent_clusters(kern, grid, 0, threads, smem, s, std::forward<Args>(args)...);
}
#ifdef __CUDACC__
// Behind every earlier grid, and then: the next one may become resident.
__device__ __forceinline__ void wait_for_earlier_grids() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

// Rotary positions of q [B,N,Hq,d] and k [B,N,Hkv,d] (rotary.cu).  Input strides in elements
// (heads are d apart); outputs contiguous, or the inputs themselves.
struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const int* positions;  // [B,N] (pos_stride = N) or [N] (pos_stride = 0)
  const unsigned long long* turns;  // [rot / 2]: turns per position, in units of 2^-64 turn
  int B, N, Hq, Hkv, d, rot;
  long q_bs, q_ts, k_bs, k_ts;  // batch and token strides of q and k
  long pos_stride;
  int interleaved, inverse;
  float magnitude;
  int bf16;
  int* status;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

// Rows of an E4M3 cache (fp8_cache.cu): codes [B,Nk_max,Hkv,d], scales [B,Hkv,Nk_max].
struct Fp8CacheArgs {
  const void *k, *v;  // append: [B,n,Hkv,d] 16-bit, batch and token strides below
  long k_bs, k_ts, v_bs, v_ts;
  uint8_t *k8, *v8;
  float *k_scale, *v_scale;
  const int* start;   // append: first cache row of each sequence
  const int* counts;  // append: rows of each sequence (nullptr: n); read: live rows
  void *k_out, *v_out;  // read: [B,n,Hkv,d] 16-bit
  int B, n, Hkv, Nk_max, d;
  int bf16;
  int* status;
};
cudaError_t launch_fp8_cache_append(const Fp8CacheArgs& a, cudaStream_t s);
cudaError_t launch_fp8_cache_read(const Fp8CacheArgs& a, cudaStream_t s);

// One-token attention over a cache (cache_decode.cu) and over a prefix that the whole batch
// shares (prefix_sm100.cu), both writing normalised fp32 partials that one kernel merges.  The
// prefix's: o_part [B,Hq,Sp,d], lse_part [B,Hq,Sp], Sp = prefix_splits.  The caches': one per CTA
// and sequence it reads keys of, o_cache [Hkv,slots,G,d], lse_cache [Hkv,slots,G] in slot
// b + CTA, slots = B + cache_ctas / Hkv, with the first and last CTA of every sequence that has
// keys in spans [B].
// CTAs of the cache kernel that an SM holds: 67 KB of shared memory each and up to 168 registers a
// thread, or 35 KB and 96 (128 for groups of 9 to 16 heads) with E4M3 rows of 64 values, which need
// more of them in flight.
constexpr int cache_ctas_per_sm(int d, bool fp8, bool wide) { return d == 64 && fp8 ? (wide ? 4 : 5) : 3; }
constexpr int kMaxCacheCtas = 1024;
struct CacheDecodeArgs {
  const void* q;  // [B,1,Hq,d]
  const void *kp, *vp;  // prefix [Np,Hkv,d] (prefix_splits > 0)
  const void *k, *v;    // cache [B,Nk_max,Hkv,d]: 16-bit, or E4M3 codes with scales [B,Hkv,Nk_max]
  const float *k_scale, *v_scale;
  const int* seqlens;
  float *o_part, *lse_part, *o_cache, *lse_cache;
  int2* spans;
  void* o;
  float* lse;
  int B, Hq, Hkv, Np, Nk_max, d;
  int prefix_splits, prefix_chunk;  // keys per prefix split, a multiple of 128
  int after_prefix;                 // the launch before the cache kernel's is the prefix kernel's
  int prefix_ctas;                  // CTAs that take the prefix's work in turn
  int solo;                         // > 0: CTAs of a cluster per sequence and KV head, which merge alone
  int cache_ctas;                   // a multiple of Hkv, at most max(kMaxCacheCtas, Hkv)
  float scale;
  int bf16;
  int* status;
};
cudaError_t launch_prefix_sm100(const CacheDecodeArgs& a, cudaStream_t s);
// The caches' partials.
cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t s);
// The merge; always launched right after launch_cache_decode, on the same stream.
cudaError_t launch_cache_combine(const CacheDecodeArgs& a, cudaStream_t s);

}  // namespace fa
