// attention.cu -- attention of a chunk of new tokens over a paged cache
// (paged_attention).
//
// New token t of request i and query head h see keys j in [lo, hi):
//   hi = causal ? min(kv_len, p + 1) : kv_len,  lo = window ? max(0, p + 1 - window) : 0,
// p = kv_len - n_i + t its place;  out = sum_j softmax_j(scale q . k_j) v_j,
// lse = log sum_j exp(scale q . k_j).  One pass over the keys with a running
// maximum m and sum l: when m grows to m', l and the accumulated output are
// multiplied by exp(m - m').
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kAttThreads = 128;

// one warp per (new token, query head); lane l holds elements l, l + 32, ...
template <int D>
__global__ void __launch_bounds__(kAttThreads) paged_attention_simple(AttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kAttThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / a.Hq;
  const int h = static_cast<int>(w % a.Hq);
  if (t >= a.T) return;
  int32_t i = 0, top = a.N;  // the last request with cu[i] <= t
  while (top - i > 1) {
    const int32_t mid = (i + top) / 2;
    if (__ldg(a.cu + mid) <= t)
      i = mid;
    else
      top = mid;
  }
  const int32_t c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
  if (!(c0 >= 0 && c0 <= t && t < c1 && c1 <= a.T)) {
    if (lane == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
    return;
  }
  const int32_t kv = __ldg(a.kv_len + i);
  const int64_t p = static_cast<int64_t>(kv) - c1 + t;
  const int64_t hi = a.causal ? min(static_cast<int64_t>(kv), p + 1) : kv;
  const int64_t lo = a.window > 0 ? max(static_cast<int64_t>(0), p + 1 - a.window) : 0;
  bool bad = kv < 0 || static_cast<int64_t>(kv) > static_cast<int64_t>(a.max_pages) * a.page_size;
  const int hk = h / (a.Hq / a.Hkv);
  const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q) + t * a.q_ts + h * a.q_hs;
  const float k2 = a.scale * kLog2e;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[lane + 32 * e]);
    o[e] = 0.f;
  }
  for (int64_t j = lo; j < hi && !bad; ++j) {
    const int64_t page = __ldg(a.table + i * a.table_stride + j / a.page_size);
    if (page < 0 || page >= a.n_pages) {
      bad = true;
      break;
    }
    const int64_t row = j % a.page_size;
    const __nv_bfloat16 *kp = reinterpret_cast<const __nv_bfloat16 *>(a.k_cache) + page * a.kc[0] + hk * a.kc[1] + row * a.kc[2];
    const __nv_bfloat16 *vp = reinterpret_cast<const __nv_bfloat16 *>(a.v_cache) + page * a.vc[0] + hk * a.vc[1] + row * a.vc[2];
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], __bfloat162float(kp[lane + 32 * e]), s);
    s = warp_sum(s) * k2;
    const float mn = fmaxf(m, s);
    const float f = (m == -INFINITY) ? 0.f : ex2(m - mn), pr = (s == -INFINITY) ? 0.f : ex2(s - mn);
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(pr, __bfloat162float(vp[lane + 32 * e]), o[e] * f);
  }
  const float nan = __int_as_float(0x7fffffff);
  if (bad && lane == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  const float inv = bad ? nan : (l == 0.f ? 0.f : 1.f / l);
  __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + (t * a.Hq + h) * D;
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 32 * e] = __float2bfloat16_rn(o[e] * inv);
  if (a.lse && lane == 0) a.lse[t * a.Hq + h] = bad ? nan : (l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2);
}

}  // namespace

size_t attention_workspace(int64_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  (void)T, (void)Hq, (void)Hkv, (void)D;
  return 256;
}

cudaError_t launch_attention(const AttendArgs &a, cudaStream_t st) {
  const int64_t warps = a.T * a.Hq;
  const int64_t grid = (warps + kAttThreads / 32 - 1) / (kAttThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  void *tm = timer_before("paged_attention", st);
  if (a.D == 128)
    paged_attention_simple<128><<<static_cast<unsigned>(grid), kAttThreads, 0, st>>>(a);
  else
    paged_attention_simple<64><<<static_cast<unsigned>(grid), kAttThreads, 0, st>>>(a);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
