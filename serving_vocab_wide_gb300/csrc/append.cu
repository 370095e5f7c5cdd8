// append.cu -- new keys (rotated) and values into a paged cache, queries
// rotated (kv_append).
//
// Pair u of a head, (a, b), at a position with (c_u, s_u) becomes
// (a c - b s, b c + a s) in fp32, rounded once to the cache's type.
//
// A copy with an address per token: bound by bytes for many tokens, by its
// chain of dependent loads (offsets and lengths -> block table, cosines ->
// stores) for a few.  Threads of a row of the block belong to one token; each
// takes one or more pairs of 16-byte vectors (both halves of its rotated
// pairs, so that queries may be rotated in place), whose loads are under way
// before the token's request has been found.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kAppThreads = 256;
constexpr int kAppMaxRow = 512;  // threads of a token at most

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
  const float *cs;
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
  const bool owned = (first >= 0 && first <= t && t < after);  // some request's token
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

// source and destination of head h of the token (keys, then values, then queries)
template <typename T>
__device__ __forceinline__ void head_rows(const AppendArgs &a, int64_t t, int h, const T *&src) {
  if (h < a.Hkv)
    src = reinterpret_cast<const T *>(a.k) + t * a.k_ts + h * a.k_hs;
  else if (h < 2 * a.Hkv)
    src = reinterpret_cast<const T *>(a.v) + t * a.v_ts + (h - a.Hkv) * a.v_hs;
  else
    src = reinterpret_cast<const T *>(a.q) + t * a.q_ts + (h - 2 * a.Hkv) * a.q_hs;
}
template <typename T>
__device__ __forceinline__ T *head_out(const AppendArgs &a, const Place &p, int64_t t, int h) {
  if (h < a.Hkv) return reinterpret_cast<T *>(a.k_cache) + p.page * a.kc[0] + h * a.kc[1] + p.row * a.kc[2];
  if (h < 2 * a.Hkv)
    return reinterpret_cast<T *>(a.v_cache) + p.page * a.vc[0] + (h - a.Hkv) * a.vc[1] + p.row * a.vc[2];
  return reinterpret_cast<T *>(a.q_out) + (t * a.Hq + (h - 2 * a.Hkv)) * a.D;
}

// a 16-byte vector as floats and back
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void get(const uint4 &w, float *f) { Elem<1>::unpack(w, f); }
  __device__ static uint32_t two(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static uint4 put(const float *f) {
    return make_uint4(two(f[0], f[1]), two(f[2], f[3]), two(f[4], f[5]), two(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void get(const uint4 &w, float *f) { Elem<0>::unpack(w, f); }
  __device__ static uint4 put(const float *f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ void turn(float &x, float &y, float c, float s) {
  const float p = x, r = y;
  x = __fsub_rn(__fmul_rn(p, c), __fmul_rn(r, s));
  y = __fadd_rn(__fmul_rn(r, c), __fmul_rn(p, s));
}

// Rows of the block: tokens.  Heads and rotated parts in multiples of two
// vectors, everything 16-byte aligned.
template <typename T>
__global__ void kv_append_vec(AppendArgs a) {
  constexpr int N = Vec<T>::N;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int slots = a.D / (2 * N), items = (a.Hq + 2 * a.Hkv) * slots;
  const int half = a.rot / 2;
  Place p;
  bool found = false;
  for (int m = threadIdx.x; m - static_cast<int>(threadIdx.x & 31) < items; m += blockDim.x) {
    const bool mine = m < items;
    const int h = mine ? m / slots : 0, sl = mine ? m % slots : 0;
    const bool rotates = h < a.Hkv || h >= 2 * a.Hkv;
    // the slot's two vectors: both halves of rotated pairs, or neighbours
    const bool halves = !a.interleaved && rotates && sl * N < half;
    const int x = halves ? sl * N : 2 * sl * N;
    const int y = halves ? half + sl * N : x + N;
    const T *src;
    head_rows<T>(a, t, h, src);
    uint4 u, w;
    if (mine) {
      u = *reinterpret_cast<const uint4 *>(src + x);
      w = *reinterpret_cast<const uint4 *>(src + y);
    }
    if (!found) {
      p = find_place(a, t);
      found = true;
    }
    if (!mine) continue;
    if (h < 2 * a.Hkv && !p.write) continue;
    if (rotates && x < a.rot) {
      if (!p.pos_ok) {
        float f[N];
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = __int_as_float(0x7fffffff);
        u = w = Vec<T>::put(f);
      } else {
        float f[N], g[N];
        Vec<T>::get(u, f);
        Vec<T>::get(w, g);
        if (halves) {
          float c[N], s[N];
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            *reinterpret_cast<float4 *>(c + e) = __ldg(reinterpret_cast<const float4 *>(p.cs + x + e));
            *reinterpret_cast<float4 *>(s + e) = __ldg(reinterpret_cast<const float4 *>(p.cs + half + x + e));
          }
#pragma unroll
          for (int e = 0; e < N; ++e) turn(f[e], g[e], c[e], s[e]);
        } else {
          // neighbours are pairs: N / 2 of each vector, N in a row of the table
          float c[N], s[N];
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            *reinterpret_cast<float4 *>(c + e) = __ldg(reinterpret_cast<const float4 *>(p.cs + x / 2 + e));
            *reinterpret_cast<float4 *>(s + e) = __ldg(reinterpret_cast<const float4 *>(p.cs + half + x / 2 + e));
          }
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            turn(f[2 * e], f[2 * e + 1], c[e], s[e]);
            turn(g[2 * e], g[2 * e + 1], c[N / 2 + e], s[N / 2 + e]);
          }
        }
        u = Vec<T>::put(f);
        w = Vec<T>::put(g);
      }
    }
    T *dst = head_out<T>(a, p, t, h);
    *reinterpret_cast<uint4 *>(dst + x) = u;
    *reinterpret_cast<uint4 *>(dst + y) = w;
  }
}

// any sizes, strides and alignments: one CTA per new token, entry by entry
template <typename T>
__global__ void __launch_bounds__(kAppThreads) kv_append_any(AppendArgs a) {
  const int64_t t = blockIdx.x;
  const Place p = find_place(a, t);
  const int D = a.D, half = a.rot / 2;
  const int heads = a.Hq + 2 * a.Hkv;
  for (int e = threadIdx.x; e < heads * D; e += kAppThreads) {
    const int h = e / D, x = e % D;
    const bool rotate = (h < a.Hkv || h >= 2 * a.Hkv) && x < a.rot;
    if (h < 2 * a.Hkv && !p.write) continue;
    const T *src;
    head_rows<T>(a, t, h, src);
    T *dst = head_out<T>(a, p, t, h);
    if (!rotate) {
      dst[x] = src[x];
      continue;
    }
    // the thread of a pair's first element does the pair (queries in place)
    const int u = a.interleaved ? x / 2 : x;
    if (a.interleaved ? (x & 1) : (x >= half)) continue;
    const int x2 = a.interleaved ? x + 1 : x + half;
    float f = ld_f(src + x), g = ld_f(src + x2);
    if (p.pos_ok)
      turn(f, g, __ldg(p.cs + u), __ldg(p.cs + half + u));
    else
      f = g = __int_as_float(0x7fffffff);
    st_f(dst + x, f);
    st_f(dst + x2, g);
  }
}

bool at16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
void launch(const AppendArgs &a, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  int64_t odd = a.k_ts | a.k_hs | a.v_ts | a.v_hs | a.q_ts | a.q_hs;
  for (int d = 0; d < 3; ++d) odd |= a.kc[d] | a.vc[d];
  const bool vec = at16(a.k) && at16(a.v) && at16(a.q) && at16(a.q_out) && at16(a.k_cache) && at16(a.v_cache) &&
                   at16(a.cos_sin) && odd % N == 0 && a.D % (2 * N) == 0 && a.rot % (2 * N) == 0;
  if (!vec) {
    kv_append_any<T><<<static_cast<unsigned>(a.T), kAppThreads, 0, st>>>(a);
    return;
  }
  // one slot per thread where a row of kAppMaxRow threads allows it; small
  // tokens share a block
  const int items = (a.Hq + 2 * a.Hkv) * (a.D / (2 * N));
  const int x = items >= kAppMaxRow ? kAppMaxRow : (items + 31) / 32 * 32;
  int y = kAppThreads / x < 1 ? 1 : kAppThreads / x;
  while (y > 1 && (a.T + y - 1) / y < 2 * 152) y /= 2;  // rather more blocks than fuller ones
  kv_append_vec<T><<<static_cast<unsigned>((a.T + y - 1) / y), dim3(x, y), 0, st>>>(a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t st) {
  void *tm = timer_before("kv_append", st);
  if (dtype == SVW_BF16)
    launch<__nv_bfloat16>(a, st);
  else
    launch<float>(a, st);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
