// gather.cu -- cached keys and values of many requests read back, packed
// (kv_gather): out = code x scale of the head in fp32, rounded once.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "append_device.cuh"
#include "e4m3.cuh"
#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kThreads = 256;

// where a token lies: page -1 if nowhere
struct Where {
  int32_t page, row;
};
// The token's request is the last one i with cu[i] <= t.
__device__ __forceinline__ Where find(const GatherArgs &a, int64_t t) {
  int32_t lo = 0, hi = a.N;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (__ldg(a.cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int32_t c0 = __ldg(a.cu + lo), c1 = __ldg(a.cu + lo + 1);
  Where w = {-1, 0};
  if (!(c0 >= 0 && c0 <= t && t < c1 && c1 <= a.T)) return w;
  const int64_t first = a.first ? __ldg(a.first + lo) : 0;
  if (first < 0) return w;
  const int64_t place = first + (t - c0);
  const int64_t at = place / a.page_size;
  if (at >= a.max_pages) return w;
  w.row = static_cast<int32_t>(place - at * a.page_size);
  const int32_t page = __ldg(a.table + lo * a.table_stride + at);
  if (page >= 0 && page < a.n_pages) w.page = page;
  return w;
}

__device__ __forceinline__ float entry(const uint8_t *p) { return e4m3x2_f2(*p).x; }
__device__ __forceinline__ float entry(const __nv_bfloat16 *p) { return ld_f(p); }
__device__ __forceinline__ float entry(const float *p) { return *p; }

// one CTA per token, entry by entry
template <typename C, typename O>
__global__ void __launch_bounds__(kThreads) gather_any(const __grid_constant__ GatherArgs a) {
  const int64_t t = blockIdx.x;
  const Where w = find(a, t);
  if (w.page < 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  const int each = a.Hkv * a.D;
  for (int e = threadIdx.x; e < 2 * each; e += kThreads) {
    const bool is_v = e >= each;
    O *out = static_cast<O *>(is_v ? a.v_out : a.k_out);
    if (!out) continue;
    const int i = is_v ? e - each : e, h = i / a.D;
    float x = __uint_as_float(kNaNs);
    if (w.page >= 0) {
      const int64_t (&st)[3] = is_v ? a.vc : a.kc;
      x = entry(static_cast<const C *>(is_v ? a.v_cache : a.k_cache) + w.page * st[0] + h * st[1] + w.row * st[2] +
                (i - h * a.D));
      if (sizeof(C) == 1) x = __fmul_rn(x, head_scale(is_v ? a.v_scale : a.k_scale, h, a.status));
    }
    st_f(out + t * each + i, x);
  }
}

template <typename C, typename O>
void launch(const GatherArgs &a, cudaStream_t st) {
  gather_any<C, O><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
}
template <typename C>
void launch(const GatherArgs &a, int out_dtype, cudaStream_t st) {
  out_dtype == SVW_BF16 ? launch<C, __nv_bfloat16>(a, st) : launch<C, float>(a, st);
}

}  // namespace

cudaError_t launch_gather(const GatherArgs &a, int cache_dtype, int out_dtype, cudaStream_t st) {
  void *tm = timer_before("kv_gather", st);
  if (cache_dtype == SVW_E4M3)
    launch<uint8_t>(a, out_dtype, st);
  else if (cache_dtype == SVW_BF16)
    launch<__nv_bfloat16>(a, out_dtype, st);
  else
    launch<float>(a, out_dtype, st);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
