// append_device.cuh -- what the calls that write the paged cache share (kv_append,
// kv_append_norm): a token's place and position, its rotation.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

constexpr uint32_t kNaNs = 0x7fff7fffu;  // a NaN in fp32, two in bf16

__device__ __forceinline__ float ld_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld_f(const float *p) { return *p; }
__device__ __forceinline__ void st_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void st_f(float *p, float x) { *p = x; }

// where a token goes, and what it is rotated by
struct Place {
  bool write;    // it has a place in the cache
  bool pos_ok;   // its position has a row of cosines
  int64_t page;
  int32_t row;
  const float *cs;  // the first row's if not
};

// By one warp: the token's request is the last one i with cu[i] <= t (32 probes
// a round; the last round brings the lengths along), then its place.
__device__ __forceinline__ Place find_place(const AppendArgs &a, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = a.N;  // the answer lies in [lo, lo + n)
  while (n > 32) {
    const int32_t step = (n + 31) / 32;
    const bool le = (lane * step < n) && (__ldg(a.cu + lo + lane * step) <= t);
    const unsigned b = __ballot_sync(0xffffffffu, le);
    const int k = b ? 31 - __clz(b) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  int32_t first = INT32_MAX, after = 0, len = 0;
  if (lane < n) {
    first = __ldg(a.cu + lo + lane);
    after = __ldg(a.cu + lo + lane + 1);
    len = __ldg(a.kv_len + lo + lane);
  }
  const unsigned b = __ballot_sync(0xffffffffu, lane < n && first <= t);
  const int k = b ? 31 - __clz(b) : 0;
  const int32_t i = lo + k;
  first = __shfl_sync(0xffffffffu, first, k);
  after = __shfl_sync(0xffffffffu, after, k);
  len = __shfl_sync(0xffffffffu, len, k);
  Place p;
  const bool owned = (first >= 0 && first <= t && t < after && after <= a.T);  // some request's token
  const int64_t place = static_cast<int64_t>(len) - after + t;
  const int64_t pos = a.positions ? __ldg(a.positions + t) : (owned ? place : -1);
  p.pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
  p.cs = a.cos_sin + (p.pos_ok ? pos : 0) * a.rot;
  p.write = owned && p.pos_ok && place >= 0;
  p.page = 0;
  p.row = 0;
  if (p.write) {  // place < 2^31
    const int32_t at = static_cast<int32_t>(place) / a.page_size;
    p.row = static_cast<int32_t>(place) - at * a.page_size;
    p.write = at < a.max_pages;
    if (p.write) p.page = __ldg(a.table + i * a.table_stride + at);
    p.write = p.write && p.page >= 0 && p.page < a.n_pages;
  }
  if (!(p.write && p.pos_ok) && lane == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  return p;
}

// By one warp: of each lane's token t the last request i with cu[i] <= t.  The
// tokens follow one another from the first lane's on; those behind `last` count
// as it does.
__device__ __forceinline__ int32_t request_of(const int32_t *cu, int32_t N, int64_t t, int64_t last) {
  const int lane = threadIdx.x & 31;
  auto search = [&](int32_t lo, int64_t x) {  // in [lo, N), 32 probes a round
    int32_t n = N - lo;
    while (n > 1) {
      const int32_t step = (n + 31) / 32;
      const bool le = (lane * step < n) && (__ldg(cu + lo + lane * step) <= x);
      const unsigned b = __ballot_sync(0xffffffffu, le);
      const int k = b ? 31 - __clz(b) : 0;
      n = min(step, n - k * step);
      lo += k * step;
    }
    return lo;
  };
  int32_t lo = search(0, __shfl_sync(0xffffffffu, t, 0));
  int32_t hi = __ldg(cu + lo + 1) > last ? lo : search(lo, last);  // often the same request
  if (t > last) t = last;
  while (hi > lo) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (__ldg(cu + mid) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// source of head h of the token (keys, then values, then queries)
template <typename T>
__device__ __forceinline__ void head_rows(const AppendArgs &a, int64_t t, int h, const T *&src) {
  if (h < a.Hkv)
    src = reinterpret_cast<const T *>(a.k) + t * a.k_ts + h * a.k_hs;
  else if (h < 2 * a.Hkv)
    src = reinterpret_cast<const T *>(a.v) + t * a.v_ts + (h - a.Hkv) * a.v_hs;
  else
    src = reinterpret_cast<const T *>(a.q) + t * a.q_ts + (h - 2 * a.Hkv) * a.q_hs;
}

// entries 4 q .. 4 q + 3 of a 16-byte vector as floats, and back
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static uint32_t two(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static float4 get(const uint4 &w, int q) {
    const float2 a = bf16x2_f2(q ? w.z : w.x), b = bf16x2_f2(q ? w.w : w.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
  __device__ static void put(uint4 &w, int q, const float4 &f) {
    (q ? w.z : w.x) = two(f.x, f.y);
    (q ? w.w : w.y) = two(f.z, f.w);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static float4 get(const uint4 &w, int) {
    return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ static void put(uint4 &w, int, const float4 &f) {
    w = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
  }
};

__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
  const float p = x, r = y;
  x = __fsub_rn(__fmul_rn(p, c), __fmul_rn(r, s));
  y = __fadd_rn(__fmul_rn(r, c), __fmul_rn(p, s));
}

// The cosines and sines of a slot's pairs: of the elements x .. x + N - 1 with
// half a rotation further (halves), or of the N pairs of neighbours from x on.
template <typename T>
struct Turns {
  static constexpr int N = Vec<T>::N;
  float4 c[N / 4], s[N / 4];
  __device__ void load(const Place &p, bool halves, int x, int half) {
    const float *cs = p.cs + (halves ? x : x / 2);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      c[q] = __ldg(reinterpret_cast<const float4 *>(cs + 4 * q));
      s[q] = __ldg(reinterpret_cast<const float4 *>(cs + half + 4 * q));
    }
  }
  // the slot's two vectors rotated
  __device__ void apply(bool halves, uint4 &u, uint4 &w) const {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      if (halves) {
        float4 f = Vec<T>::get(u, q), g = Vec<T>::get(w, q);
        turn(f.x, g.x, c[q].x, s[q].x);
        turn(f.y, g.y, c[q].y, s[q].y);
        turn(f.z, g.z, c[q].z, s[q].z);
        turn(f.w, g.w, c[q].w, s[q].w);
        Vec<T>::put(u, q, f);
        Vec<T>::put(w, q, g);
      } else {  // four pairs: a vector of eight, or two of four
        uint4 &m = (N == 8 && q == 1) ? w : u, &n = (N == 8) ? m : w;
        float4 f = Vec<T>::get(m, 0), g = Vec<T>::get(n, N == 8 ? 1 : 0);
        turn(f.x, f.y, c[q].x, s[q].x);
        turn(f.z, f.w, c[q].y, s[q].y);
        turn(g.x, g.y, c[q].z, s[q].z);
        turn(g.z, g.w, c[q].w, s[q].w);
        Vec<T>::put(m, 0, f);
        Vec<T>::put(n, N == 8 ? 1 : 0, g);
      }
    }
  }
};

inline bool at16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace svw
