// append.cu -- new keys (rotated) and values into a paged cache, queries
// rotated (kv_append).
//
// Pair u of a head, (a, b), at a position with (c_u, s_u) becomes
// (a c - b s, b c + a s) in fp32, rounded once.  A copy with an address per
// token: bound by bytes, or by the launch for a few tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kAppThreads = 256;

__device__ __forceinline__ float ld_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld_f(const float *p) { return *p; }
__device__ __forceinline__ void st_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void st_f(float *p, float x) { *p = x; }

// the last request i with cu[i] <= t: one warp, 32 probes a round
__device__ __forceinline__ int32_t find_request(const int32_t *cu, int32_t N, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = N;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) / 32;
    const int32_t at = lo + lane * step;
    const bool le = (lane * step < n) && (__ldg(cu + at) <= t);
    const unsigned b = __ballot_sync(0xffffffffu, le);
    const int k = b ? 31 - __clz(b) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// one CTA per new token
template <typename T>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(AppendArgs a) {
  const int64_t t = blockIdx.x;
  const int32_t i = find_request(a.cu, a.N, t);
  const int32_t c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
  const int64_t place = static_cast<int64_t>(__ldg(a.kv_len + i)) - c1 + t;
  const bool owned = (c0 >= 0 && c0 <= t && t < c1);  // some request's token
  bool write = (owned && place >= 0 && place / a.page_size < a.max_pages);
  int64_t page = 0;
  if (write) {
    page = __ldg(a.table + i * a.table_stride + place / a.page_size);
    write = (page >= 0 && page < a.n_pages);
  }
  const int64_t pos = a.positions ? __ldg(a.positions + t) : (owned ? place : -1);
  const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
  if ((!write || !pos_ok) && threadIdx.x == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  write = write && pos_ok;
  const int64_t row = write ? place % a.page_size : 0;
  const int D = a.D, half = a.rot / 2;
  const float *cs = a.cos_sin + (pos_ok ? pos : 0) * a.rot;
  const int heads = a.Hq + 2 * a.Hkv;
  for (int e = threadIdx.x; e < heads * D; e += kAppThreads) {
    const int h = e / D, x = e % D;
    const T *src;
    T *dst;
    bool rotate = a.rot > 0 && x < a.rot;
    if (h < a.Hkv) {
      if (!write) continue;
      src = reinterpret_cast<const T *>(a.k) + t * a.k_ts + h * a.k_hs;
      dst = reinterpret_cast<T *>(a.k_cache) + page * a.kc[0] + h * a.kc[1] + row * a.kc[2];
    } else if (h < 2 * a.Hkv) {
      if (!write) continue;
      const int hh = h - a.Hkv;
      src = reinterpret_cast<const T *>(a.v) + t * a.v_ts + hh * a.v_hs;
      dst = reinterpret_cast<T *>(a.v_cache) + page * a.vc[0] + hh * a.vc[1] + row * a.vc[2];
      rotate = false;
    } else {
      const int hh = h - 2 * a.Hkv;
      src = reinterpret_cast<const T *>(a.q) + t * a.q_ts + hh * a.q_hs;
      dst = reinterpret_cast<T *>(a.q_out) + (t * a.Hq + hh) * D;
    }
    if (!rotate) {
      dst[x] = src[x];
      continue;
    }
    // the thread of a pair's first element does the pair (q_out may be q)
    const int u = a.interleaved ? x / 2 : x;
    if (a.interleaved ? (x & 1) : (x >= half)) continue;
    const int x2 = a.interleaved ? x + 1 : x + half;
    float c = __int_as_float(0x7fffffff), s = c;
    if (pos_ok) {
      c = __ldg(cs + u);
      s = __ldg(cs + half + u);
    }
    const float p = ld_f(src + x), r = ld_f(src + x2);
    st_f(dst + x, __fsub_rn(__fmul_rn(p, c), __fmul_rn(r, s)));
    st_f(dst + x2, __fadd_rn(__fmul_rn(r, c), __fmul_rn(p, s)));
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t st) {
  void *tm = timer_before("kv_append", st);
  if (dtype == SVW_BF16)
    kv_append_kernel<__nv_bfloat16><<<static_cast<unsigned>(a.T), kAppThreads, 0, st>>>(a);
  else
    kv_append_kernel<float><<<static_cast<unsigned>(a.T), kAppThreads, 0, st>>>(a);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
