// attention_fp8.cu -- attention of new tokens over a paged cache of e4m3 codes
// (paged_attention_fp8):
//   s_j = scale k_scale q . K_j,  out = v_scale sum_j softmax_j(s) V_j,
//   lse = log sum_j exp(s_j).
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
constexpr int kMany = 8;  // keys under way

// a warp per token and query head: the keys one by one, a running maximum and sum
template <int D>
__global__ void __launch_bounds__(kThreads) attention_fp8_any(const __grid_constant__ AttendArgs a) {
  constexpr int E = D / 32;
  const int64_t orow = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (orow >= a.T * a.Hq) return;
  const int64_t t = orow / a.Hq;
  const int h = static_cast<int>(orow - t * a.Hq), hk = h / (a.Hq / a.Hkv);
  int32_t lo = 0, up = a.N;
  while (up - lo > 1) {
    const int32_t mid = lo + (up - lo) / 2;
    if (__ldg(a.cu + mid) <= t)
      lo = mid;
    else
      up = mid;
  }
  const int32_t c0 = __ldg(a.cu + lo), c1 = __ldg(a.cu + lo + 1);
  int32_t kv = __ldg(a.kv_len + lo);
  auto report = [&] {
    if (lane == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  };
  if (!(c0 >= 0 && c0 <= t && t < c1 && c1 <= a.T)) {
    report();
    return;
  }
  bool bad = kv < 0 || kv > a.max_pages * a.page_size;
  if (bad) kv = 0;
  const int32_t pos = kv - (c1 - c0) + static_cast<int32_t>(t - c0);
  const int32_t end = a.causal ? min(kv, pos + 1) : kv;
  const int32_t begin = a.window > 0 ? max(0, pos + 1 - min(a.window, max(pos + 1, 1))) : 0;
  float q[E], acc[E];
  for (int e = 0; e < E; ++e) {
    q[e] = ld_f(static_cast<const __nv_bfloat16 *>(a.q) + t * a.q_ts + h * a.q_hs + lane * E + e);
    acc[e] = 0.f;
  }
  const float k2 = a.scale * kLog2e * head_scale(a.k_scale, hk, a.status), vs = head_scale(a.v_scale, hk, a.status);
  float M = -INFINITY, l = 0.f;
  for (int32_t j0 = begin; j0 < end; j0 += kMany) {
    float s[kMany], v[kMany][E];
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      const int32_t j = min(j0 + u, end - 1);
      const int32_t page = __ldg(a.table + lo * a.table_stride + j / a.page_size);
      const bool ok = page >= 0 && page < a.n_pages;
      bad |= !ok;
      const int32_t row = j % a.page_size;
      const uint8_t *kp = static_cast<const uint8_t *>(a.k_cache) + (ok ? page : 0) * a.kc[0] + hk * a.kc[1] + row * a.kc[2];
      const uint8_t *vp = static_cast<const uint8_t *>(a.v_cache) + (ok ? page : 0) * a.vc[0] + hk * a.vc[1] + row * a.vc[2];
      s[u] = 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 k = e4m3x2_f2(*reinterpret_cast<const uint16_t *>(kp + lane * E + e));
        const float2 w = e4m3x2_f2(*reinterpret_cast<const uint16_t *>(vp + lane * E + e));
        s[u] = fmaf(q[e + 1], k.y, fmaf(q[e], k.x, s[u]));
        v[u][e] = w.x;
        v[u][e + 1] = w.y;
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      s[u] = warp_sum(s[u]) * k2;
      if (j0 + u < end) top = fmaxf(top, s[u]);
    }
    const float f = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
    for (int u = 0; u < kMany; ++u) {
      if (j0 + u >= end) break;
      const float p = ex2(s[u] - M);
      l += p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(p, v[u][e], acc[e]);
    }
  }
  if (bad) {
    report();
    l = __uint_as_float(kNaNs);
  }
  const float inv = l == 0.f ? 0.f : vs / l;
  for (int e = 0; e < E; ++e)
    st_f(static_cast<__nv_bfloat16 *>(a.out) + orow * D + lane * E + e, acc[e] * inv);
  if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_attention_fp8(const AttendArgs &a, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((a.T * a.Hq + kThreads / 32 - 1) / (kThreads / 32));
  void *tm = timer_before("paged_attention_fp8", st);
  a.D == 128 ? attention_fp8_any<128><<<blocks, kThreads, 0, st>>>(a) : attention_fp8_any<64><<<blocks, kThreads, 0, st>>>(a);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
