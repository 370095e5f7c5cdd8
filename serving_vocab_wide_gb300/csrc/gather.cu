// gather.cu -- cached keys and values of many requests read back, packed
// (kv_gather): out = code x scale of the head in fp32, rounded once.
//
// A copy, bound by DRAM for many tokens: 333 k tokens of 8 heads of 128, codes to
// bf16, 2.04 GB, in 345 us (5.9 TB/s of 6.8; a third of it is read, two thirds
// written), 777 tokens in 3.9.  (A block per token, entry by entry: 2520.)
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
constexpr int kTile = 32;  // tokens of a block, at most: one warp finds them

// where a token lies: page -1 if nowhere
struct Where {
  int32_t page, row;
};
// By one warp: where its lanes' tokens lie, which follow one another up to `last`.
__device__ __forceinline__ Where find(const GatherArgs &a, int64_t t, int64_t last) {
  const int32_t i = request_of(a.cu, a.N, t, last);
  const int32_t c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
  Where w = {-1, 0};
  if (t > last) return w;
  if (c0 >= 0 && c0 <= t && t < c1 && c1 <= a.T) {
    const int64_t first = a.first ? __ldg(a.first + i) : 0, place = first + (t - c0);
    const int32_t at = first < 0 || place > INT32_MAX ? a.max_pages : static_cast<int32_t>(place) / a.page_size;
    if (at < a.max_pages) {
      w.row = static_cast<int32_t>(place) - at * a.page_size;
      const int32_t page = __ldg(a.table + i * a.table_stride + at);
      if (page >= 0 && page < a.n_pages) w.page = page;
    }
  }
  if (w.page < 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  return w;
}

__device__ __forceinline__ float entry(const uint8_t *p) { return e4m3x2_f2(*p).x; }
__device__ __forceinline__ float entry(const __nv_bfloat16 *p) { return ld_f(p); }
__device__ __forceinline__ float entry(const float *p) { return *p; }

// the elements of a 16-byte vector of a cache, as floats
__device__ __forceinline__ void open(const uint4 &w, float (&f)[16]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 g = e4m3x2_f2((i & 1) ? in[i / 2] >> 16 : in[i / 2]);
    f[2 * i] = g.x, f[2 * i + 1] = g.y;
  }
}
__device__ __forceinline__ void open(const uint4 &w, float (&f)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 g = bf16x2_f2(in[i]);
    f[2 * i] = g.x, f[2 * i + 1] = g.y;
  }
}
__device__ __forceinline__ void open(const uint4 &w, float (&f)[4]) {
  f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
}
template <int E>
__device__ __forceinline__ void put(__nv_bfloat16 *dst, const float (&f)[E]) {
  if constexpr (E == 4) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(Vec<__nv_bfloat16>::two(f[0], f[1]), Vec<__nv_bfloat16>::two(f[2], f[3]));
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 8)
      *reinterpret_cast<uint4 *>(dst + e) =
          make_uint4(Vec<__nv_bfloat16>::two(f[e], f[e + 1]), Vec<__nv_bfloat16>::two(f[e + 2], f[e + 3]),
                     Vec<__nv_bfloat16>::two(f[e + 4], f[e + 5]), Vec<__nv_bfloat16>::two(f[e + 6], f[e + 7]));
  }
}
template <int E>
__device__ __forceinline__ void put(float *dst, const float (&f)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 4) *reinterpret_cast<float4 *>(dst + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
}

// A block has a tile of tokens: its first warp finds them, then a thread has one
// 16-byte vector of keys or values (or every blockDim.x-th) of every
// blockDim.y-th token, kItems of them under way (two: 345 us, four 355, eight
// 367).  Everything 16-byte aligned.
template <typename C, typename O, int kItems>
__global__ void __launch_bounds__(kThreads) gather_vec(const __grid_constant__ GatherArgs a) {
  constexpr int E = 16 / sizeof(C);
  __shared__ int64_t at[2][kTile];  // of keys and values, in elements; -1: nowhere
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tile), a.T - t0));
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  if (tid < 32) {
    const Where w = find(a, t0 + tid, t0 + tokens - 1);
    if (tid < tokens) {
      at[0][tid] = w.page < 0 ? -1 : w.page * a.kc[0] + w.row * a.kc[2];
      at[1][tid] = w.page < 0 ? -1 : w.page * a.vc[0] + w.row * a.vc[2];
    }
  }
  __syncthreads();
  const int of_head = a.D / E, of_side = a.Hkv * of_head;
  for (int s = threadIdx.x; s < 2 * of_side; s += blockDim.x) {
    const int side = s >= of_side, i = s - side * of_side, h = i / of_head;
    O *out = static_cast<O *>(side ? a.v_out : a.k_out);
    if (!out) continue;
    const float scale = sizeof(C) == 1 ? head_scale(side ? a.v_scale : a.k_scale, h, a.status) : 1.f;
    const C *in = static_cast<const C *>(side ? a.v_cache : a.k_cache) + h * (side ? a.vc[1] : a.kc[1]) + (i - h * of_head) * E;
    out += t0 * (of_side * E) + i * E;
    for (int t = threadIdx.y; t < tokens; t += kItems * blockDim.y) {
      uint4 w[kItems];
      bool ok[kItems];
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int tq = t + q * blockDim.y;
        const int64_t from = tq < tokens ? at[side][tq] : -1;
        ok[q] = from >= 0;
        if (ok[q]) w[q] = ld_stream(in + from);
      }
#pragma unroll
      for (int q = 0; q < kItems; ++q) {
        const int tq = t + q * blockDim.y;
        if (tq >= tokens) break;
        float f[E];
        open(w[q], f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = !ok[q] ? __uint_as_float(kNaNs) : sizeof(C) == 1 ? __fmul_rn(f[e], scale) : f[e];
        put<E>(out + static_cast<int64_t>(tq) * (of_side * E), f);
      }
    }
  }
}

// any sizes, strides and alignments: one CTA per token, entry by entry
template <typename C, typename O>
__global__ void __launch_bounds__(kThreads) gather_any(const __grid_constant__ GatherArgs a) {
  __shared__ Where found;
  const int64_t t = blockIdx.x;
  if (threadIdx.x < 32) {
    const Where w = find(a, t + threadIdx.x, t);
    if (threadIdx.x == 0) found = w;
  }
  __syncthreads();
  const Where w = found;
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
void launch(GatherArgs a, cudaStream_t st) {
  constexpr int E = 16 / sizeof(C), kItems = 2;
  int64_t odd = a.D;
  for (int d = 0; d < 3; ++d) odd |= a.kc[d] | a.vc[d];
  if (!at16(a.k_cache) || !at16(a.v_cache) || !at16(a.k_out) || !at16(a.v_out) || odd % E != 0) {
    gather_any<C, O><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    return;
  }
  const int vectors = 2 * a.Hkv * (a.D / E);
  const int x = vectors >= kThreads ? kThreads : (vectors + 31) / 32 * 32, y = kThreads / x;
  // tokens of a block: no fewer blocks than four for each SM, where there are so many
  const int64_t share = a.T / (4 * 152);
  a.tile = static_cast<int32_t>(share < y ? y : share > kTile ? kTile : share);
  gather_vec<C, O, kItems><<<static_cast<unsigned>((a.T + a.tile - 1) / a.tile), dim3(x, y), 0, st>>>(a);
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
