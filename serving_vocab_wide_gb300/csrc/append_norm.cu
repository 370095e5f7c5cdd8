// append_norm.cu -- new keys (normed per head, rotated) and values into a paged
// cache of their own type or of e4m3 codes, queries normed and rotated
// (kv_append_norm).
//
//   y_e = x_e w_e / sqrt(mean_e x_e^2 + eps);  pairs (a, b) of y become
//   (a c - b s, b c + a s);  code = e4m3(y / scale of the head)
// in fp32, the quotient too, rounded once.
//
// Bound by instructions and by its chain of dependent loads (offsets and lengths
// -> block table, cosines -> stores) rather than by its bytes.  A kernel like
// kv_append's, whose threads take slots of heads of all classes one after
// another, executed 460 instructions for each warp's round of heads (22.5 us on
// 2196 tokens of 32 query and 8 key heads of 128, 50.6 MB into codes); warps of
// one class, which form the products of weights, cosines and sines once, take
// 197 (18 us), and finding the tokens once a block instead of once a warp does
// the rest.  Device time: 14.8 us there (3.4 TB/s), 30.6 on 14 k tokens of 48
// heads of 64 (4.7 TB/s), 14.8 on 1742 tokens of 40 and 8 heads into bf16, 3.3 for
// one token.  Rounds in fours 16.0 and 40, one at a time 16.4 and 34; two blocks
// an SM 17.5 and 34, four 15.6 and 32; loads staged through shared memory two
// tasks ahead 14.6 and 39.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "append_device.cuh"
#include "e4m3.cuh"
#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSms = 152;
constexpr int kTokens = 32;  // of a block, at most: one warp finds them

// The N values of pairs' first and second elements: the two vectors (kApart), or
// the neighbours of their 2N elements.  (What is not turned may lie either way.)
template <typename T, bool kApart>
__device__ __forceinline__ void open(const uint4 &u, const uint4 &w, float *f, float *g) {
  constexpr int N = Vec<T>::N;
  float x[2 * N];
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const float4 m = Vec<T>::get(u, q), n = Vec<T>::get(w, q);
    x[4 * q] = m.x, x[4 * q + 1] = m.y, x[4 * q + 2] = m.z, x[4 * q + 3] = m.w;
    x[N + 4 * q] = n.x, x[N + 4 * q + 1] = n.y, x[N + 4 * q + 2] = n.z, x[N + 4 * q + 3] = n.w;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    f[e] = kApart ? x[e] : x[2 * e];
    g[e] = kApart ? x[N + e] : x[2 * e + 1];
  }
}
// back into the order of the two vectors
template <int N, bool kApart>
__device__ __forceinline__ void shut(const float *f, const float *g, float *x) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    x[e] = kApart ? f[e] : (e & 1) ? g[e / 2] : f[e / 2];
    x[N + e] = kApart ? g[e] : (e & 1) ? g[(N + e) / 2] : f[(N + e) / 2];
  }
}
template <typename T>
__device__ __forceinline__ void put(T *dst, const float *f) {
  uint4 u;
#pragma unroll
  for (int q = 0; q < Vec<T>::N / 4; ++q) Vec<T>::put(u, q, make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]));
  *reinterpret_cast<uint4 *>(dst) = u;
}
__device__ __forceinline__ float2 at2(const float *f, int e) { return make_float2(f[e], f[e + 1]); }
__device__ __forceinline__ void to2(float *f, int e, const float2 &v) { f[e] = v.x, f[e + 1] = v.y; }

// The four codes nearest to quotients in fp32, of any size.
__device__ __noinline__ uint32_t codes_of_quotients(float a, float b, float c, float d, float s) {
  return e4m3x4(__fdiv_rn(a, s), __fdiv_rn(b, s), __fdiv_rn(c, s), __fdiv_rn(d, s));
}
// The codes nearest to x / s, that quotient in fp32, of E numbers.  A product
// with a rounded 1 / s is off by an ulp or two, which at a tie is another code (19
// of 1920 bf16 numbers under 7 / 512), so 1 / s comes as two numbers, 47 bits.
// Neither is zero or negative: an infinity stays one, and a zero keeps its sign.
// (Beside a product with the rounded one: 14.5 and 30.5 us instead of 14.8 and 30.6
// on the two cases above; the product corrected by its remainder 15.1 and 32.1.)
template <int E>
__device__ __forceinline__ void codes(const float *x, float s, uint32_t *c) {
  if (s >= 0x1p-60f && s <= 0x1p60f) {
    const float inv = __frcp_rd(s), rest = fmaxf(fmaf(-s, inv, 1.f) * inv, inv * 0x1p-40f);
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      float2 m[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 y = at2(x, 4 * q + 2 * i);
        m[i] = __ffma2_rn(y, make_float2(inv, inv), __fmul2_rn(y, make_float2(rest, rest)));
      }
      c[q] = e4m3x4(m[0].x, m[0].y, m[1].x, m[1].y);
    }
  } else {  // a scale near the ends of fp32's range, or none
#pragma unroll
    for (int q = 0; q < E / 4; ++q) c[q] = codes_of_quotients(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3], s);
  }
}

// where a token goes
struct Spot {
  int64_t k, v;  // elements of the caches to its row; k -1: nowhere
  int32_t pos;   // the row of cosines, -1: none
};
// By one warp: those of its lanes' tokens, which follow one another.
__device__ __forceinline__ Spot find_spot(const AppendNormArgs &a, int64_t t, int64_t last) {
  const int32_t i = request_of(a.cu, a.N, t, last);
  Spot s = {-1, 0, -1};
  if (t > last) return s;
  const int32_t first = __ldg(a.cu + i), after = __ldg(a.cu + i + 1), len = __ldg(a.kv_len + i);
  const bool owned = first >= 0 && first <= t && t < after && after <= a.T;  // some request's token
  const int64_t place = static_cast<int64_t>(len) - after + t;
  const int64_t pos = a.positions ? __ldg(a.positions + t) : (owned ? place : -1);
  const bool pos_ok = a.rot == 0 || (pos >= 0 && pos < a.max_pos);
  if (pos_ok) s.pos = a.rot == 0 ? 0 : static_cast<int32_t>(pos);
  if (owned && pos_ok && place >= 0) {  // place < 2^31
    const int32_t at = static_cast<int32_t>(place) / a.page_size, row = static_cast<int32_t>(place) - at * a.page_size;
    const int32_t page = at < a.max_pages ? __ldg(a.table + i * a.table_stride + at) : -1;
    if (page >= 0 && page < a.n_pages) {
      s.k = page * a.kc[0] + row * a.kc[2];
      s.v = page * a.vc[0] + row * a.vc[2];
    }
  }
  if (s.k < 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  return s;
}

enum { kKeysOf, kValuesOf, kQueriesOf };

// A warp's task: kItems rounds of a token's heads of one class; of round 0 head
// h0, and slot sl of it, are the lane's.
template <typename T, bool kCodes, bool kApart, int kItems, int kClass>
__device__ __forceinline__ void form(const AppendNormArgs &a, const Spot &p, uint32_t t, int h0, int sl,
                                     const uint4 (&u)[kItems], const uint4 (&w)[kItems]) {
  constexpr int N = Vec<T>::N;
  constexpr bool kCode = kCodes && kClass != kQueriesOf;
  using Out = std::conditional_t<kCode, uint8_t, T>;
  const int lane = threadIdx.x & 31, heads_round = 32 >> a.lane_bits, half = a.rot / 2;
  const int heads = kClass == kQueriesOf ? a.Hq : a.Hkv;
  const bool apart = kApart && sl * N < half;
  const int x = apart ? sl * N : 2 * sl * N, y = apart ? half + sl * N : x + N;
  const bool mine = x < a.D, turns = x < a.rot && kClass != kValuesOf;
  const float *weight = kClass == kQueriesOf ? a.q_weight : kClass == kKeysOf ? a.k_weight : nullptr;
  // where head h0's slot goes, and how much further a round's is
  Out *dst;
  int64_t next;
  if (kClass == kQueriesOf) {
    dst = static_cast<Out *>(a.q_out) + (static_cast<int64_t>(t) * a.Hq + h0) * a.D;
    next = heads_round * a.D;
  } else {
    const int64_t hs = kClass == kKeysOf ? a.kc[1] : a.vc[1];
    dst = static_cast<Out *>(kClass == kKeysOf ? a.k_cache : a.v_cache) + (kClass == kKeysOf ? p.k : p.v) + h0 * hs;
    next = heads_round * hs;
    if (p.k < 0) return;
  }
  float ca[N], cb[N], sa[N], sb[N];  // sb: negative (not turned: ca and cb the weights)
  if (kClass != kValuesOf) {
    float c[N], s[N];
#pragma unroll
    for (int e = 0; e < N; ++e) c[e] = 1.f, s[e] = 0.f;
    if (turns && p.pos >= 0) {
      const float *cs = a.cos_sin + static_cast<int64_t>(p.pos) * a.rot + (apart ? x : x / 2);
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        *reinterpret_cast<float4 *>(c + e) = __ldg(reinterpret_cast<const float4 *>(cs + e));
        *reinterpret_cast<float4 *>(s + e) = __ldg(reinterpret_cast<const float4 *>(cs + half + e));
      }
    }
    float v[2 * N];
#pragma unroll
    for (int e = 0; e < 2 * N; ++e) v[e] = 1.f;
    if (weight && mine) {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        *reinterpret_cast<float4 *>(v + e) = __ldg(reinterpret_cast<const float4 *>(weight + x + e));
        *reinterpret_cast<float4 *>(v + N + e) = __ldg(reinterpret_cast<const float4 *>(weight + y + e));
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float f = kApart ? v[e] : v[2 * e], g = kApart ? v[N + e] : v[2 * e + 1];
      ca[e] = __fmul_rn(f, c[e]), sa[e] = __fmul_rn(f, s[e]);
      cb[e] = __fmul_rn(g, c[e]), sb[e] = __fmul_rn(g, -s[e]);
    }
  }
#pragma unroll
  for (int q = 0; q < kItems; ++q, dst += next) {
    const int h = h0 + q * heads_round;
    if (q > 0 && h - (lane >> a.lane_bits) >= heads) break;  // the whole warp
    float f[N], g[N];
    open<T, kApart>(u[q], w[q], f, g);
    float r = 1.f;
    if (kClass != kValuesOf && weight) {
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < N; e += 2) s2 = __ffma2_rn(at2(f, e), at2(f, e), __ffma2_rn(at2(g, e), at2(g, e), s2));
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = 0; o < 5; ++o)
        if (o < a.lane_bits) ss += __shfl_xor_sync(0xffffffffu, ss, 1 << o);
      r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
    }
    if (h >= heads || !mine) continue;
    if (kClass == kQueriesOf && p.pos < 0) {  // nothing to rotate it by
      *reinterpret_cast<uint4 *>(dst + x) = *reinterpret_cast<uint4 *>(dst + y) = make_uint4(kNaNs, kNaNs, kNaNs, kNaNs);
      continue;
    }
    if (!kCode && !turns && (kClass == kValuesOf || !weight)) {  // as it is, NaN bits too
      *reinterpret_cast<uint4 *>(dst + x) = u[q];
      *reinterpret_cast<uint4 *>(dst + y) = w[q];
      continue;
    }
    if (turns) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 fe = at2(f, e), ge = at2(g, e);
        to2(f, e, __ffma2_rn(ge, at2(sb, e), __fmul2_rn(fe, at2(ca, e))));
        to2(g, e, __ffma2_rn(fe, at2(sa, e), __fmul2_rn(ge, at2(cb, e))));
      }
    } else if (kClass != kValuesOf) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        to2(f, e, __fmul2_rn(at2(f, e), at2(ca, e)));
        to2(g, e, __fmul2_rn(at2(g, e), at2(cb, e)));
      }
    }
    if (kClass != kValuesOf) {  // (no norm: by 1, which is faster than a branch)
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        to2(f, e, __fmul2_rn(at2(f, e), make_float2(r, r)));
        to2(g, e, __fmul2_rn(at2(g, e), make_float2(r, r)));
      }
    }
    float o[2 * N];
    shut<N, kApart>(f, g, o);
    if constexpr (kCode) {
      uint32_t c[N / 2];
      codes<2 * N>(o, head_scale(kClass == kKeysOf ? a.k_scale : a.v_scale, h, a.status), c);
      if constexpr (N == 8) {
        *reinterpret_cast<uint2 *>(dst + x) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2 *>(dst + y) = make_uint2(c[2], c[3]);
      } else {
        *reinterpret_cast<uint32_t *>(dst + x) = c[0];
        *reinterpret_cast<uint32_t *>(dst + y) = c[1];
      }
    } else {
      put<T>(dst + x, o);
      put<T>(dst + y, o + N);
    }
  }
}

// A block has a stretch of the line of all tokens' tasks, a.share of them, a warp
// one after another; its first warp finds the tokens' spots, once for all their
// tasks, while the warps' first loads are under way.  2^lane_bits lanes share a
// head; each has one slot of it, two vectors (both halves of its pairs), and adds
// the squares up by exchange.  What is the same for all heads of a class, the
// weights times cosines and sines, is formed once a task:
//   a' = r (a (w_a c) - b (w_b s)),  b' = r (b (w_b c) + a (w_a s)).
// Heads and rotated parts in multiples of two
// vectors, everything 16-byte aligned.
template <typename T, bool kCodes, bool kApart, int kItems>
__global__ void __launch_bounds__(kThreads, 3) append_norm_vec(const __grid_constant__ AppendNormArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Spot spots[kTokens];
  const uint32_t begin = blockIdx.x * a.share, end = min(begin + a.share, a.line);
  const uint32_t t0 = begin / a.tasks;
  const int lane = threadIdx.x & 31, heads_round = 32 >> a.lane_bits, half = a.rot / 2;
  const int sl = lane & ((1 << a.lane_bits) - 1);
  const bool apart = kApart && sl * N < half;
  const int x = apart ? sl * N : 2 * sl * N, y = apart ? half + sl * N : x + N;
  const bool mine = x < a.D;
  uint32_t at = begin + (threadIdx.x >> 5), t = 0;
  int kind = 0, h0 = 0;
  uint4 u[kItems], w[kItems];
  auto load = [&] {
    t = at / a.tasks;
    int task = static_cast<int>(at - t * a.tasks);
    kind = task < a.kv_tasks ? kKeysOf : task < 2 * a.kv_tasks ? kValuesOf : kQueriesOf;
    task -= kind * a.kv_tasks;
    h0 = task * kItems * heads_round + (lane >> a.lane_bits);
    const int heads = kind == kQueriesOf ? a.Hq : a.Hkv;
    const void *base = kind == kQueriesOf ? a.q : kind == kValuesOf ? a.v : a.k;
    const int64_t ts = kind == kQueriesOf ? a.q_ts : kind == kValuesOf ? a.v_ts : a.k_ts;
    const int64_t hs = kind == kQueriesOf ? a.q_hs : kind == kValuesOf ? a.v_hs : a.k_hs;
    const T *src = static_cast<const T *>(base) + t * ts + h0 * hs;
#pragma unroll
    for (int q = 0; q < kItems; ++q, src += heads_round * hs) {
      u[q] = w[q] = make_uint4(0, 0, 0, 0);
      if (h0 + q * heads_round < heads && mine) {
        u[q] = *reinterpret_cast<const uint4 *>(src + x);
        w[q] = *reinterpret_cast<const uint4 *>(src + y);
      }
    }
  };
  if (at < end) load();
  if (threadIdx.x < 32) {
    const uint32_t last = (end - 1) / a.tasks;
    const Spot s = find_spot(a, static_cast<int64_t>(t0) + lane, last);
    if (t0 + lane <= last) spots[lane] = s;
  }
  __syncthreads();
  while (at < end) {
    const Spot &p = spots[t - t0];
    if (kind == kQueriesOf)
      form<T, kCodes, kApart, kItems, kQueriesOf>(a, p, t, h0, sl, u, w);
    else if (kind == kKeysOf)
      form<T, kCodes, kApart, kItems, kKeysOf>(a, p, t, h0, sl, u, w);
    else
      form<T, kCodes, kApart, kItems, kValuesOf>(a, p, t, h0, sl, u, w);
    at += kWarps;
    if (at < end) load();
  }
}

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
    float r = 1.f, scale = 1.f;
    if (weight) {
      float ss = 0.f;
      for (int e = lane; e < D; e += 32) ss = fmaf(ld_f(src + e), ld_f(src + e), ss);
      r = rsqrtf(fmaf(warp_sum(ss), a.inv_dim, a.eps));
    }
    if (kCodes && !is_q) scale = head_scale(is_v ? a.v_scale : a.k_scale, hh, a.status);
    auto get = [&](int e) { return weight ? __fmul_rn(__fmul_rn(ld_f(src + e), r), __ldg(weight + e)) : ld_f(src + e); };
    T *q_out = reinterpret_cast<T *>(a.q_out) + (t * a.Hq + hh) * D;
    const int64_t at = is_v ? p.page * a.vc[0] + hh * a.vc[1] + p.row * a.vc[2]
                            : p.page * a.kc[0] + hh * a.kc[1] + p.row * a.kc[2];
    void *cache = is_v ? a.v_cache : a.k_cache;
    auto put = [&](int e, float y) {
      if (is_q)
        st_f(q_out + e, y);
      else if (kCodes)
        static_cast<uint8_t *>(cache)[at + e] = static_cast<uint8_t>(e4m3x2(__fdiv_rn(y, scale), 0.f));
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
void launch(AppendNormArgs a, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  int64_t odd = a.k_ts | a.k_hs | a.v_ts | a.v_hs | a.q_ts | a.q_hs;
  for (int d = 0; d < 3; ++d) odd |= a.kc[d] | a.vc[d];
  const bool vec = at16(a.k) && at16(a.v) && at16(a.q) && at16(a.q_out) && at16(a.k_cache) && at16(a.v_cache) &&
                   at16(a.cos_sin) && at16(a.k_weight) && at16(a.q_weight) && odd % N == 0 && a.D % (2 * N) == 0 &&
                   a.rot % (2 * N) == 0;
  a.inv_dim = 1.f / static_cast<float>(a.D);
  const int slots = vec ? a.D / (2 * N) : 64;
  while ((1 << a.lane_bits) < slots) ++a.lane_bits;
  // As long as all tasks of one round fit the SMs at once (three blocks each), a round a task is the shortest way
  // through: of 48 heads of 128, 1 token 3.3 us (rounds in twos 3.8), 300 tokens 4.5 (4.6), 400 5.4 (4.7).
  const int round = 32 >> a.lane_bits;
  const int items = a.T * (a.Hq + 2 * a.Hkv) < 3 * kSms * kWarps * round ? 1 : 2;
  const int each = items * std::max(round, 1);
  a.kv_tasks = (a.Hkv + each - 1) / each;
  a.tasks = 2 * a.kv_tasks + (a.Hq + each - 1) / each;
  if (slots > 32 || a.T * a.tasks > INT32_MAX) {
    append_norm_any<T, kCodes><<<static_cast<unsigned>(a.T), kThreads, 0, st>>>(a);
    return;
  }
  a.line = static_cast<uint32_t>(a.T * a.tasks);
  // three blocks an SM at once, of a task a warp at least and of kTokens tokens at most
  const uint32_t even = (a.line + 3 * kSms - 1) / (3 * kSms);
  a.share = std::min(std::max<uint32_t>(even, kWarps), (kTokens - 1) * a.tasks);
  const unsigned grid = (a.line + a.share - 1) / a.share;
  auto go = [&](auto apart) {
    constexpr bool kApart = decltype(apart)::value;
    if (items == 1)
      append_norm_vec<T, kCodes, kApart, 1><<<grid, kThreads, 0, st>>>(a);
    else
      append_norm_vec<T, kCodes, kApart, 2><<<grid, kThreads, 0, st>>>(a);
  };
  a.interleaved ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace

cudaError_t launch_append_norm(const AppendNormArgs &a, int dtype, cudaStream_t st) {
  if (!a.codes && !a.k_weight && !a.q_weight) return launch_append(a, dtype, st, "kv_append_norm");
  void *tm = timer_before("kv_append_norm", st);
  if (dtype == SVW_BF16)
    a.codes ? launch<__nv_bfloat16, true>(a, st) : launch<__nv_bfloat16, false>(a, st);
  else
    a.codes ? launch<float, true>(a, st) : launch<float, false>(a, st);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
