// serving_api.cu -- C ABI of the rotary, E4M3-cache and cache-decode operators
// (declared in include/fa.h): argument validation, split heuristics and
// dispatch.  Validation happens before anything is launched; the library
// allocates no device memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "fa.h"
#include "kernels.h"
#include "serving.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Half-open byte range of a strided [B, N, H, d] 16-bit tensor.
struct Range {
  uintptr_t lo, hi;
};
Range range_of(const void* p, long long bs, long long ts, int B, int N, int H, int d) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + 2ull * ((unsigned long long)(B - 1) * bs + (unsigned long long)(N - 1) * ts + (unsigned long long)H * d)};
}
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Element strides of the token and batch dimensions: whole 16-byte chunks, and far below the
// point where an address computation could leave 64 bits.
bool strides_ok(long long bs, long long ts) {
  const long long most = 1ll << 40;
  return bs >= 0 && ts >= 0 && bs <= most && ts <= most;
}
bool strides_aligned(long long bs, long long ts) { return bs % 8 == 0 && ts % 8 == 0; }

int sm_count(int num_sms) { return num_sms > 0 ? num_sms : fa::device_sm_count(); }

fa_status check_decode(int B, int Hq, int Hkv, int Nk_max, int d, float scale, fa_dtype dt) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nk_max < 1) return FA_ERR_INVALID;
  if (Hq % Hkv != 0) return FA_ERR_INVALID;
  if (!(scale >= 0.f) || std::isinf(scale)) return FA_ERR_INVALID;
  if (dt != FA_FP16 && dt != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 16) return FA_ERR_UNSUPPORTED;  // one CTA holds a GQA group of at most 16 query heads
  if (B > 65535 || Hkv > 65535 || Hq > 65535 || Nk_max > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// CTAs of a cluster per sequence and KV head for a batch small enough to go without a separate merge
// (0: too large): as many as 128 keys each leave, all resident at once, at most 1024 keys each and 8 of a
// prefix's partials a row.  64 sequences of up to 500 E4M3 keys, 8 KV heads of 64 (512 clusters of one, 740
// resident): 9.3 us, with a merge of its own 13.2; heads of 128 (444 resident): 18.0 and 17.1.  Resident on the
// 148 SMs of a B200, whatever device is current: the workspace, which a cluster does without, has to be the
// same wherever its bytes are asked for.
int solo_of(int B, int Hq, int Hkv, int Nk_max, int prefix_splits, int d, bool fp8) {
  const long long units = (long long)B * Hkv, most = 148ll * fa::cache_ctas_per_sm(d, fp8, Hq / Hkv > 8);
  if (units > most || prefix_splits > 8) return 0;
  int n = 8;
  while (n > 1 && (units * n > most || 128ll * (n / 2) >= Nk_max)) n /= 2;
  return Nk_max <= 1024 * n ? n : 0;
}

// Bytes of the partials, and where each kind lies: O of the prefix and of the caches, then the LSEs, then the spans.
struct Workspace {
  size_t o_cache, lse_part, lse_cache, spans, bytes;
};
Workspace workspace_of(int B, int Hq, int Hkv, int prefix_splits, int d) {
  const size_t rows = (size_t)B * Hq * prefix_splits;
  const size_t slots = ((size_t)B * Hkv + std::max(fa::kMaxCacheCtas, Hkv)) * (Hq / Hkv);
  Workspace w;
  w.o_cache = rows * d * 4;
  w.lse_part = w.o_cache + slots * d * 4;
  w.lse_cache = w.lse_part + rows * 4;
  w.spans = (w.lse_cache + slots * 4 + 15) / 16 * 16;
  w.bytes = w.spans + ((size_t)B * 8 + 255) / 256 * 256;
  return w;
}

void place(fa::CacheDecodeArgs& a, void* workspace, const Workspace& w) {
  unsigned char* base = static_cast<unsigned char*>(workspace);
  a.o_part = reinterpret_cast<float*>(base);
  a.o_cache = reinterpret_cast<float*>(base + w.o_cache);
  a.lse_part = reinterpret_cast<float*>(base + w.lse_part);
  a.lse_cache = reinterpret_cast<float*>(base + w.lse_cache);
  a.spans = reinterpret_cast<int2*>(base + w.spans);
}

// CTAs of the cache kernel: the SMs that a prefix running beside it leaves (all of them once they are
// few), two blocks of keys a CTA at least.
int cache_ctas_of(int B, int Hkv, int Nk_max, int d, int G, bool fp8, int sms, long long prefix_ctas) {
  const long long left = sms - prefix_ctas >= sms / 4 ? sms - prefix_ctas : sms;
  const long long blocks = (long long)B * ((Nk_max + 127) / 128);
  const long long most = std::min<long long>(fa::cache_ctas_per_sm(d, fp8, G > 8) * left, fa::kMaxCacheCtas) / Hkv;  // per KV head
  return (int)(Hkv * std::max<long long>(1, std::min(most, blocks / 2)));
}

// Row blocks of the prefix kernel: 128 / G sequences to a query tile, one or two tiles to a block.
long long prefix_row_blocks(int B, int G) {
  const int seqs = 128 / G;
  return B <= seqs ? 1 : (B + 2 * seqs - 1) / (2 * seqs);
}

// CTAs of the prefix kernel for a number of splits, and an estimate of the call's time in microseconds.
// As measured: a K/V tile takes 2 with two query tiles, 1.6 with one, a work 4 more in its turn and the
// kernel 5 to start and end (heads of 128; the same is taken for 64); beside it an SM streams 60 KB of a 16-bit
// cache, 40 KB of an E4M3 one.  The lengths are on the device, so four fifths of a cache's room are taken to be
// in use, and caches that hold far less leave the prefix too few SMs: 64 sequences of 100 E4M3 keys behind 8192
// take 23 us in caches of 128 rows, 31 of 1024, 69 of 4096, 482 of 32768.  The cache kernel fills the SMs that the
// prefix leaves, if they are a quarter at least, or follows it, which costs 8 and a third of its time more.  64
// sequences behind 32768 keys, 1024 of their own: 80 CTAs 65 us, 144 79; 250 behind 8192, 512: 64 CTAs 73 us, 128 87.
struct PrefixPlan {
  int ctas;
  double cost;
};
PrefixPlan plan_prefix(int B, int G, int Hkv, int Np, int Nk_max, int d, bool fp8, int splits, int sms) {
  const long long work = prefix_row_blocks(B, G) * Hkv * splits;
  const int per = ((Np + 127) / 128 + splits - 1) / splits;  // K/V tiles of a work
  const double tile = B > 128 / G ? 2.0 : 1.6;
  const double kb = 0.8 * 2.0 * B * Nk_max * Hkv * (fp8 ? d + 4 : 2 * d) / 1e3;
  const double cache = kb / (fp8 ? 40 : 60);  // SM microseconds
  const double hbm = (kb + 4.0 * Np * Hkv * d / 1e3) / 6500.0;
  PrefixPlan best{0, 0};
  for (int rounds = 1; rounds <= 8; ++rounds) {
    const long long ctas = (work + rounds - 1) / rounds;
    if (ctas > sms) continue;
    const double prefix = rounds * (per * tile + 4.0) + 5.0, left = (double)(sms - ctas);
    const double cost = std::max(hbm, left >= sms / 4 ? std::max(prefix, cache / left) : prefix + 1.3 * cache / sms + 8.0);
    if (best.ctas == 0 || cost < best.cost) best = PrefixPlan{(int)ctas, cost};
  }
  if (best.ctas == 0) {
    const long long rounds = (work + sms - 1) / sms;
    best = PrefixPlan{sms, std::max(hbm, rounds * (per * tile + 4.0) + 5.0 + 1.3 * cache / sms + 8.0)};
  }
  return best;
}

}  // namespace

extern "C" {

fa_status fa_rotary(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
                    const unsigned long long* turns, int B, int N, int Hq, int Hkv, int d, int rot_dim,
                    int interleaved, int inverse, float magnitude, long long q_batch_stride, long long q_token_stride,
                    long long k_batch_stride, long long k_token_stride, long long position_batch_stride, fa_dtype dt,
                    fa_stream_t stream) {
  if (!q || !q_out || !positions || !turns || (Hkv > 0 && (!k || !k_out))) return FA_ERR_INVALID;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 0) return FA_ERR_INVALID;
  if (rot_dim < 2 || rot_dim > d) return FA_ERR_INVALID;
  if (!std::isfinite(magnitude)) return FA_ERR_INVALID;
  if (position_batch_stride != 0 && position_batch_stride < N) return FA_ERR_INVALID;
  if (!strides_ok(q_batch_stride, q_token_stride) || (Hkv > 0 && !strides_ok(k_batch_stride, k_token_stride)))
    return FA_ERR_INVALID;
  if (dt != FA_FP16 && dt != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hq > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if ((long long)B * N > (1ll << 31) - 1) return FA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(positions, 4) || !aligned(turns, 8) ||
      !strides_aligned(q_batch_stride, q_token_stride))
    return FA_ERR_ALIGN;
  if (Hkv > 0 && (!aligned(k, 16) || !aligned(k_out, 16) || !strides_aligned(k_batch_stride, k_token_stride)))
    return FA_ERR_ALIGN;
  // an output is its own input, element for element, or apart from both inputs and the other output
  const long long qt = (long long)Hq * d, kt = (long long)Hkv * d;
  const Range qi = range_of(q, q_batch_stride, q_token_stride, B, N, Hq, d), qo = range_of(q_out, N * qt, qt, B, N, Hq, d);
  if (q_out == q ? !((N == 1 || q_token_stride == qt) && (B == 1 || q_batch_stride == N * qt)) : overlap(qo, qi))
    return FA_ERR_INVALID;
  if (Hkv > 0) {
    const Range ki = range_of(k, k_batch_stride, k_token_stride, B, N, Hkv, d), ko = range_of(k_out, N * kt, kt, B, N, Hkv, d);
    if (k_out == k ? !((N == 1 || k_token_stride == kt) && (B == 1 || k_batch_stride == N * kt)) : overlap(ko, ki))
      return FA_ERR_INVALID;
    if (overlap(qo, ko) || overlap(qo, ki) || overlap(ko, qi)) return FA_ERR_INVALID;
  }
  fa::RotaryArgs a{q, k, q_out, k_out, positions, turns, B, N, Hq, Hkv, d, rot_dim, q_batch_stride, q_token_stride,
                   k_batch_stride, k_token_stride, position_batch_stride, interleaved ? 1 : 0, inverse ? 1 : 0,
                   magnitude, dt == FA_BF16 ? 1 : 0, fa::device_status_word()};
  if (!a.status) return FA_ERR_CUDA;
  return from_cuda(fa::launch_rotary(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_fp8_cache_append(const void* k, const void* v, void* k8, void* v8, float* k_scale, float* v_scale,
                              const int* start, const int* counts, int B, int n, int Hkv, int Nk_max, int d,
                              long long k_batch_stride, long long k_token_stride, long long v_batch_stride,
                              long long v_token_stride, fa_dtype dt, fa_stream_t stream) {
  if (!k || !v || !k8 || !v8 || !k_scale || !v_scale || !start) return FA_ERR_INVALID;
  if (B < 1 || n < 1 || Hkv < 1 || Nk_max < 1) return FA_ERR_INVALID;
  if (!strides_ok(k_batch_stride, k_token_stride) || !strides_ok(v_batch_stride, v_token_stride)) return FA_ERR_INVALID;
  if (dt != FA_FP16 && dt != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || Nk_max > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)B * n * Hkv > (1ll << 31) - 1) return FA_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(start, 4) || (counts && !aligned(counts, 4)) ||
      !strides_aligned(k_batch_stride, k_token_stride) || !strides_aligned(v_batch_stride, v_token_stride))
    return FA_ERR_ALIGN;
  fa::Fp8CacheArgs a{};
  a.k = k;
  a.v = v;
  a.k_bs = k_batch_stride;
  a.k_ts = k_token_stride;
  a.v_bs = v_batch_stride;
  a.v_ts = v_token_stride;
  a.k8 = static_cast<uint8_t*>(k8);
  a.v8 = static_cast<uint8_t*>(v8);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.start = start;
  a.counts = counts;
  a.B = B;
  a.n = n;
  a.Hkv = Hkv;
  a.Nk_max = Nk_max;
  a.d = d;
  a.bf16 = dt == FA_BF16 ? 1 : 0;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  return from_cuda(fa::launch_fp8_cache_append(a, static_cast<cudaStream_t>(stream)));
}

fa_status fa_fp8_cache_read(const void* k8, const void* v8, const float* k_scale, const float* v_scale,
                            const int* seqlens_k, void* k, void* v, int B, int Nk, int Hkv, int Nk_max, int d,
                            fa_dtype dt, fa_stream_t stream) {
  if (!k8 || !v8 || !k_scale || !v_scale || !seqlens_k || !k || !v) return FA_ERR_INVALID;
  if (B < 1 || Nk < 1 || Hkv < 1 || Nk_max < Nk) return FA_ERR_INVALID;
  if (dt != FA_FP16 && dt != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || Nk_max > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)B * Nk * Hkv > (1ll << 31) - 1) return FA_ERR_UNSUPPORTED;
  if (!aligned(k8, 16) || !aligned(v8, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(seqlens_k, 4))
    return FA_ERR_ALIGN;
  fa::Fp8CacheArgs a{};
  a.k8 = static_cast<uint8_t*>(const_cast<void*>(k8));
  a.v8 = static_cast<uint8_t*>(const_cast<void*>(v8));
  a.k_scale = const_cast<float*>(k_scale);
  a.v_scale = const_cast<float*>(v_scale);
  a.counts = seqlens_k;
  a.k_out = k;
  a.v_out = v;
  a.B = B;
  a.n = Nk;
  a.Hkv = Hkv;
  a.Nk_max = Nk_max;
  a.d = d;
  a.bf16 = dt == FA_BF16 ? 1 : 0;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  return from_cuda(fa::launch_fp8_cache_read(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_decode_fp8_workspace_bytes(int B, int Hq, int Hkv, int Nk_max, int prefix_splits, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Nk_max < 1 || Hq % Hkv != 0 || prefix_splits < 0 || d < 1) return 0;
  if (prefix_splits == 0 && solo_of(B, Hq, Hkv, Nk_max, 0, d, true) > 0) return 0;
  return workspace_of(B, Hq, Hkv, prefix_splits, d).bytes;
}

fa_status fa_decode_fp8(const void* q, const void* k8, const void* v8, const float* k_scale, const float* v_scale,
                        const int* seqlens_k, void* o, float* lse, void* workspace, int B, int Hq, int Hkv, int Nk_max,
                        int d, float scale, fa_dtype dt, fa_stream_t stream) {
  if (!q || !k8 || !v8 || !k_scale || !v_scale || !seqlens_k || !o || !lse) return FA_ERR_INVALID;
  const fa_status st = check_decode(B, Hq, Hkv, Nk_max, d, scale, dt);
  if (st != FA_OK) return st;
  const int solo = solo_of(B, Hq, Hkv, Nk_max, 0, d, true);
  if (!workspace && !solo) return FA_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k8, 16) || !aligned(v8, 16) || !aligned(o, 16) || !aligned(workspace, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(seqlens_k, 4) || !aligned(lse, 4))
    return FA_ERR_ALIGN;
  fa::CacheDecodeArgs a{};
  a.q = q;
  a.k = k8;
  a.v = v8;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.seqlens = seqlens_k;
  place(a, workspace, workspace_of(B, Hq, Hkv, 0, d));
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.Nk_max = Nk_max;
  a.d = d;
  a.solo = solo;
  a.cache_ctas = cache_ctas_of(B, Hkv, Nk_max, d, Hq / Hkv, true, fa::device_sm_count(), 0);
  a.scale = scale;
  a.bf16 = dt == FA_BF16 ? 1 : 0;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_cache_decode(a, s);
  if (e == cudaSuccess && !a.solo) e = fa::launch_cache_combine(a, s);
  return from_cuda(e);
}

// Keys per prefix split: ceil(Np / splits) rounded up to a 128-key tile.
static int prefix_chunk(int Np, int splits) { return ((Np + splits - 1) / splits + 127) / 128 * 128; }

int fa_decode_prefix_splits(int B, int Hq, int Hkv, int Np, int Nk_max, int d, int fp8_cache, int num_sms) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Np < 1 || Nk_max < 0 || d < 1 || Hq % Hkv != 0 || Hq / Hkv > 128) return 1;
  const int tiles = (Np + 127) / 128;
  int best = 1;
  double least = -1;
  for (int s = 1; s <= std::min(tiles, 256); ++s) {
    const int per = (tiles + s - 1) / s;
    if ((tiles + per - 1) / per != s) continue;  // the same lengths with fewer splits
    const double cost = plan_prefix(B, Hq / Hkv, Hkv, Np, Nk_max, d, fp8_cache != 0, s, sm_count(num_sms)).cost + 0.1 * s;
    if (least < 0 || cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

fa_status fa_decode_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k_cache,
                                  const void* v_cache, const float* k_scale, const float* v_scale,
                                  const int* seqlens_k, void* o, float* lse, void* workspace, int B, int Hq, int Hkv,
                                  int Np, int Nk_max, int d, float scale, int prefix_splits,
                                  fa_dtype dt, fa_stream_t stream) {
  if (!q || !k_prefix || !v_prefix || !k_cache || !v_cache || !seqlens_k || !o || !lse || !workspace)
    return FA_ERR_INVALID;
  if ((k_scale == nullptr) != (v_scale == nullptr)) return FA_ERR_INVALID;
  const fa_status st = check_decode(B, Hq, Hkv, Nk_max, d, scale, dt);
  if (st != FA_OK) return st;
  if (Np < 1 || prefix_splits < 1) return FA_ERR_INVALID;
  if (Np > (1 << 30) || prefix_splits > 65535) return FA_ERR_UNSUPPORTED;
  if (prefix_splits > (Np + 127) / 128) return FA_ERR_INVALID;
  const int pchunk = prefix_chunk(Np, prefix_splits);
  if ((long long)(prefix_splits - 1) * pchunk >= Np) return FA_ERR_INVALID;  // the last split would be empty
  if (!aligned(q, 16) || !aligned(k_prefix, 16) || !aligned(v_prefix, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(workspace, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(seqlens_k, 4) || !aligned(lse, 4))
    return FA_ERR_ALIGN;
  if (!fa::tma_available()) return FA_ERR_CUDA;  // the driver lacks the tensor-map encoder
  fa::CacheDecodeArgs a{};
  a.q = q;
  a.kp = k_prefix;
  a.vp = v_prefix;
  a.k = k_cache;
  a.v = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.seqlens = seqlens_k;
  place(a, workspace, workspace_of(B, Hq, Hkv, prefix_splits, d));
  a.o = o;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.Np = Np;
  a.Nk_max = Nk_max;
  a.d = d;
  a.prefix_splits = prefix_splits;
  a.after_prefix = 1;
  a.prefix_chunk = pchunk;
  a.solo = solo_of(B, Hq, Hkv, Nk_max, prefix_splits, d, k_scale != nullptr);
  const int sms = fa::device_sm_count();
  a.prefix_ctas = plan_prefix(B, Hq / Hkv, Hkv, Np, Nk_max, d, k_scale != nullptr, prefix_splits, sms).ctas;
  a.cache_ctas = cache_ctas_of(B, Hkv, Nk_max, d, Hq / Hkv, k_scale != nullptr, sms, a.prefix_ctas);
  a.scale = scale;
  a.bf16 = dt == FA_BF16 ? 1 : 0;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_prefix_sm100(a, s);
  if (e == cudaSuccess) e = fa::launch_cache_decode(a, s);
  if (e == cudaSuccess && !a.solo) e = fa::launch_cache_combine(a, s);
  return from_cuda(e);
}

}  // extern "C"
