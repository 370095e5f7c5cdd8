// append_norm.cu -- new keys (normed per head, rotated) and values into a paged
// cache of their own type or of e4m3 codes, queries normed and rotated
// (kv_append_norm).
//
//   y_e = x_e w_e / sqrt(mean_e x_e^2 + eps);  pairs (a, b) of y become
//   (a c - b s, b c + a s);  code = e4m3(y / scale of the head)
// in fp32, rounded once.
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

// any sizes, strides and alignments: one CTA per new token, a warp per head
template <typename T, bool kCodes>
__global__ void __launch_bounds__(kThreads) append_norm_any(const __grid_constant__ AppendNormArgs a) {
  const int64_t t = blockIdx.x;
  const Place p = find_place(a, t);
  const int lane = threadIdx.x & 31, D = a.D, half = a.rot / 2;
  for (int h = threadIdx.x >> 5; h < a.Hq + 2 * a.Hkv; h += kThreads / 32) {
    const bool is_q = h >= 2 * a.Hkv, is_v = h >= a.Hkv && !is_q;
    const int hh = is_q ? h - 2 * a.Hkv : (is_v ? h - a.Hkv : h);
    if (!is_q && !p.write) continue;
    const T *src;
    head_rows<T>(a, t, h, src);
    const float *weight = is_q ? a.q_weight : (is_v ? nullptr : a.k_weight);
    float r = 1.f, inv = 1.f;
    if (weight) {
      float ss = 0.f;
      for (int e = lane; e < D; e += 32) ss = fmaf(ld_f(src + e), ld_f(src + e), ss);
      r = rsqrtf(warp_sum(ss) / static_cast<float>(D) + a.eps);
    }
    if (kCodes && !is_q) inv = __frcp_rn(head_scale(is_v ? a.v_scale : a.k_scale, hh, a.status));
    auto get = [&](int e) { return weight ? __fmul_rn(__fmul_rn(ld_f(src + e), r), __ldg(weight + e)) : ld_f(src + e); };
    T *q_out = reinterpret_cast<T *>(a.q_out) + (t * a.Hq + hh) * D;
    const int64_t at = is_v ? p.page * a.vc[0] + hh * a.vc[1] + p.row * a.vc[2]
                            : p.page * a.kc[0] + hh * a.kc[1] + p.row * a.kc[2];
    void *cache = is_v ? a.v_cache : a.k_cache;
    auto put = [&](int e, float y) {
      if (is_q)
        st_f(q_out + e, y);
      else if (kCodes)
        static_cast<uint8_t *>(cache)[at + e] = static_cast<uint8_t>(e4m3x2(__fmul_rn(y, inv), 0.f));
      else
        st_f(static_cast<T *>(cache) + at + e, y);
    };
    const int turned = is_v ? 0 : half;
    if (is_q && !p.pos_ok) {  // nothing to rotate it by
      for (int e = lane; e < D; e += 32) st_f(q_out + e, __uint_as_float(kNaNs));
      continue;
    }
    for (int u = lane; u < turned; u += 32) {
      const int x = a.interleaved ? 2 * u : u, y = a.interleaved ? x + 1 : u + half;
      float f = get(x), g = get(y);
      turn(f, g, __ldg(p.cs + u), __ldg(p.cs + half + u));
      put(x, f);
      put(y, g);
    }
    for (int e = 2 * turned + lane; e < D; e += 32) put(e, get(e));
  }
}

template <typename T, bool kCodes>
void launch(const AppendNormArgs &a, cudaStream_t st) {
  append_norm_any<T, kCodes><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_append_norm(const AppendNormArgs &a, int dtype, cudaStream_t st) {
  void *tm = timer_before("kv_append_norm", st);
  if (dtype == SVW_BF16)
    a.codes ? launch<__nv_bfloat16, true>(a, st) : launch<__nv_bfloat16, false>(a, st);
  else
    a.codes ? launch<float, true>(a, st) : launch<float, false>(a, st);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
