// append.cu -- new keys (rotated) and values into a paged cache, queries
// rotated (kv_append).
//
// Pair u of a head, (a, b), at a position with (c_u, s_u) becomes
// (a c - b s, b c + a s) in fp32, rounded once to the cache's type.
//
// A copy with an address per token: bound by bytes for many tokens, by its
// chain of dependent loads (offsets and lengths -> block table, cosines ->
// stores) for a few.  Threads of a row of the block belong to one token; each
// takes slots of two 16-byte vectors (both halves of its rotated pairs, so that
// queries may be rotated in place), whose loads are under way before the
// token's request has been found.  Two tokens a row, to search once for both,
// were slower (18 us against 16 where a slot a thread was), and a torch copy of
// 27 MB takes 9.9 us where rotating and scattering them takes 12.1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kAppThreads = 256;  // of a block of many tokens' rows
constexpr int kAppRow = 512;      // of a row when tokens are few
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

// Rows of the block: tokens.  A thread has one slot, two vectors (both halves
// of its pairs), of every blockDim.x / slots-th head, kItems heads under way:
// its cosines and sines are read once.  (Read again for each head, with the
// head found by a division: 12.8 us where this takes 12.1 on 2220 tokens of 48
// heads of 128, 34.7 where it takes 33.1 on 14 k tokens of 48 heads of 64; 56%
// of the issue slots were busy.)  Heads and rotated parts in multiples of two
// vectors, everything 16-byte aligned.
template <typename T, int kItems>
__global__ void __launch_bounds__(kItems == 1 ? kAppRow : kAppThreads, kItems == 1 ? 3 : 4) kv_append_vec(const __grid_constant__ AppendArgs a) {
  constexpr int N = Vec<T>::N;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= a.T) return;
  const int slots = a.D / (2 * N), heads = a.Hq + 2 * a.Hkv, step = blockDim.x / slots;
  const int half = a.rot / 2, h0 = threadIdx.x / slots, sl = threadIdx.x - h0 * slots;
  const bool halves = !a.interleaved && sl * N < half;
  const int x = halves ? sl * N : 2 * sl * N, y = halves ? half + sl * N : x + N;
  const bool turns = x < a.rot;
  Place p;
  Turns<T> cs;
  bool found = false;
  for (int h = h0; h - h0 < heads; h += kItems * step) {  // the whole warp as often
    uint4 u[kItems], w[kItems];
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
      if (h + q * step < heads) {
        const T *src;
        head_rows<T>(a, t, h + q * step, src);
        u[q] = *reinterpret_cast<const uint4 *>(src + x);
        w[q] = *reinterpret_cast<const uint4 *>(src + y);
      }
    }
    if (!found) {
      p = find_place(a, t);
      if (turns) cs.load(p, halves, x, half);
      found = true;
    }
#pragma unroll
    for (int q = 0; q < kItems; ++q) {
      const int hq = h + q * step;
      if (hq >= heads || (hq < 2 * a.Hkv && !p.write)) continue;
      if (turns && (hq < a.Hkv || hq >= 2 * a.Hkv)) cs.apply(halves, u[q], w[q]);
      T *dst = head_out<T>(a, p, t, hq);
      *reinterpret_cast<uint4 *>(dst + x) = u[q];
      *reinterpret_cast<uint4 *>(dst + y) = w[q];
    }
  }
  // queries that nothing is there to rotate by, once more (looked for inside the loop: 12.6 -> 13.0 us)
  if (!p.pos_ok) {
    for (int h = h0; h < heads; h += step) {
      if (h < 2 * a.Hkv) continue;
      T *dst = head_out<T>(a, p, t, h);
      *reinterpret_cast<uint4 *>(dst + x) = *reinterpret_cast<uint4 *>(dst + y) = make_uint4(kNaNs, kNaNs, kNaNs, kNaNs);
    }
  }
}

// any sizes, strides and alignments: one CTA per new token, entry by entry
template <typename T>
__global__ void __launch_bounds__(kAppThreads) kv_append_any(const __grid_constant__ AppendArgs a) {
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
    if (!p.pos_ok) {  // a query: nothing to rotate it by
      st_f(dst + x, __uint_as_float(kNaNs));
      continue;
    }
    if (!rotate) {
      dst[x] = src[x];
      continue;
    }
    // the thread of a pair's first element does the pair (queries in place)
    const int u = a.interleaved ? x / 2 : x;
    if (a.interleaved ? (x & 1) : (x >= half)) continue;
    const int x2 = a.interleaved ? x + 1 : x + half;
    float f = ld_f(src + x), g = ld_f(src + x2);
    turn(f, g, __ldg(p.cs + u), __ldg(p.cs + half + u));
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
  // threads of a row: whole warps, and as many for each slot
  const int slots = vec ? a.D / (2 * N) : 1;
  int unit = 32;
  while (unit % slots != 0) unit += 32;
  if (!vec || unit > kAppThreads) {
    kv_append_any<T><<<static_cast<unsigned>(a.T), kAppThreads, 0, st>>>(a);
    return;
  }
  // Many tokens: about six heads a thread, in two rounds of three (the second
  // round's loads run beside the first one's stores): 12.1 and 33.1 us on the
  // two batches above; three in one round 13.2 and 36.1, in rounds of two 12.7
  // and 34.2, of four 13.4 and 39.0.  Few: one, the shortest way through.
  const int items = (a.Hq + 2 * a.Hkv) * slots;
  const bool few = a.T < 2 * 152;
  const int share = few ? items : (items + 5) / 6;
  const int most = (few ? kAppRow : kAppThreads) / unit * unit;
  const int x = share >= most ? most : (share + unit - 1) / unit * unit;
  int y = kAppThreads / x < 1 ? 1 : kAppThreads / x;
  while (y > 1 && (a.T + y - 1) / y < 2 * 152) y /= 2;  // rather more blocks than fuller ones
  const dim3 grid(static_cast<unsigned>((a.T + y - 1) / y)), block(x, y);
  if (few)
    kv_append_vec<T, 1><<<grid, block, 0, st>>>(a);
  else
    kv_append_vec<T, 3><<<grid, block, 0, st>>>(a);
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
