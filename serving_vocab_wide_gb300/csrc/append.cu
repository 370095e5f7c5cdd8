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

#include "append_device.cuh"
#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kAppThreads = 256;  // of a block of many tokens' rows
constexpr int kAppRow = 512;      // of a row when tokens are few

// destination of head h of the token
template <typename T>
__device__ __forceinline__ T *head_out(const AppendArgs &a, const Place &p, int64_t t, int h) {
  if (h < a.Hkv) return reinterpret_cast<T *>(a.k_cache) + p.page * a.kc[0] + h * a.kc[1] + p.row * a.kc[2];
  if (h < 2 * a.Hkv)
    return reinterpret_cast<T *>(a.v_cache) + p.page * a.vc[0] + (h - a.Hkv) * a.vc[1] + p.row * a.vc[2];
  return reinterpret_cast<T *>(a.q_out) + (t * a.Hq + (h - 2 * a.Hkv)) * a.D;
}

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

cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t st, const char *name) {
  void *tm = timer_before(name, st);
  if (dtype == SVW_BF16)
    launch<__nv_bfloat16>(a, st);
  else
    launch<float>(a, st);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
