// adjust.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of drafted positions (logits_adjust).
//
// Row j of request i has seen the request's history and its drafted tokens
// x_0 .. x_{j-1}; with n(v) the occurrences of v after the prompt part,
//   y = logits[row, v];  seen: y = y > 0 ? y / rep : y rep;
//   n > 0: y -= freq n + pres;  y += bias(v);  mask bit 0: y = -inf.
//
// Bound by bytes: a row is read and written once, and few of its entries
// change.  One CTA owns a chunk of the vocabulary of one request: it counts
// the history's tokens that fall into its chunk in shared memory (32-bit
// integer atomics: the order does not matter) and lists them, the biased and
// the drafted ones, each once.  It walks the request's rows over that chunk
// twice: all entries in 16-byte vectors, copied with the mask applied by
// selection (a vector that is all masked is written without being read; in
// place, one that is all allowed is left alone), and, once the history is
// counted, the listed entries one by one.  A thread keeps four vectors under
// way, of several rows where the chunk is short.  (Looking at listed entries inside the first walk
// cost more: some lane of nearly every warp has one, and 929 us against the
// two walks' time on the benchmark batch.)  The drafted prefix differs from
// row to row and is not counted: the chunk's drafted tokens (at most
// SVW_MAX_LEN) are kept as a list and compared by the listed entries.  Every
// chunk of a request reads the whole history (from L2): at 8192 tokens that is
// 32 KB beside the ~140 KB of logits that a chunk of 4096 entries moves for
// nine bf16 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjBatch = 4;  // vectors of a thread under way
constexpr int kAhead = 8;     // history tokens of a thread under way
constexpr uint32_t kNothing = 0x100;  // no vector to write
constexpr int32_t kPromptBit = static_cast<int32_t>(0x80000000u);

// what a CTA knows of its request and chunk
struct AdjChunk {
  const int32_t *cnt;   // [chunk] occurrences after the prompt part | kPromptBit
  const int32_t *bidx;  // [chunk] 1 + the last place in the bias list that names the token (0: none)
  const float *bias_values;
  int32_t nd;           // the chunk's drafted tokens (in shared memory: token, position)
  const int32_t *dtok, *dpos;
  float rep, freq, pres;
};

// the entry's value after penalties and bias; false: it stays as it is
__device__ __forceinline__ bool adjust_entry(const AdjChunk &c, int u, int j, float &y) {
  const int32_t w = c.cnt[u];
  int32_t n = w & ~kPromptBit;
  for (int d = 0; d < c.nd; ++d) n += (c.dtok[d] == u && c.dpos[d] < j) ? 1 : 0;
  const bool seen = (w != 0) || (n > 0);
  const int32_t b = c.bidx ? c.bidx[u] : 0;
  if (!seen && b == 0) return false;
  if (seen) y = (y > 0.f) ? __fdiv_rn(y, c.rep) : __fmul_rn(y, c.rep);
  if (n > 0) y = __fsub_rn(__fsub_rn(y, __fmul_rn(c.freq, static_cast<float>(n))), c.pres);
  if (b != 0) y = __fadd_rn(y, __ldg(c.bias_values + b - 1));
  return true;
}

// one entry in the bits of its type
template <int DT>
struct Bits;
template <>
struct Bits<1> {
  using T = uint16_t;
  static constexpr uint32_t kNegInf = 0xff80u, kNaN = 0x7fffu;
  // word w of a vector (entries 2 w, 2 w + 1) with the entries whose bit of ok is 0 made -inf
  __device__ static uint32_t hide(uint32_t x, uint32_t ok, int w) {
    const uint32_t keep = ((ok >> (2 * w)) & 1u) * 0xffffu + ((ok >> (2 * w + 1)) & 1u) * 0xffff0000u;
    return (x & keep) | (0xff80ff80u & ~keep);
  }
  __device__ static float value(uint32_t b) { return __uint_as_float(b << 16); }
  __device__ static uint32_t bits(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
template <>
struct Bits<0> {
  using T = uint32_t;
  static constexpr uint32_t kNegInf = 0xff800000u, kNaN = 0x7fffffffu;
  __device__ static uint32_t hide(uint32_t x, uint32_t ok, int w) { return ((ok >> w) & 1u) ? x : kNegInf; }
  __device__ static float value(uint32_t b) { return __uint_as_float(b); }
  __device__ static uint32_t bits(float x) { return __float_as_uint(x); }
};

// `count` bits of a bitmap from bit `at` on (words: how many it has)
__device__ __forceinline__ uint32_t bits_at(const uint32_t *map, int64_t words, int64_t at, uint32_t count) {
  const int64_t w = at >> 5;
  const uint32_t lo = map[w], hi = (w + 1 < words) ? map[w + 1] : 0u;
  return __funnelshift_r(lo, hi, static_cast<uint32_t>(at & 31)) & ((1u << count) - 1u);
}

// kRowVecs: vectors of a chunk's row per thread; 0: the input and output rows
// do not lie equally far from a 16-byte boundary, entry by entry
template <int DT, int kRowVecs>
__global__ void __launch_bounds__(kAdjThreads, 4) logits_adjust_kernel(AdjustArgs a) {
  constexpr bool VEC = kRowVecs > 0;
  using B = Bits<DT>;
  using T = typename B::T;
  constexpr int EPV = 16 / sizeof(T);
  constexpr uint32_t kAll = (1u << EPV) - 1u;
  extern __shared__ int32_t dyn[];
  __shared__ int32_t dtok[SVW_MAX_LEN], dpos[SVW_MAX_LEN], nd, nlist;
  __shared__ int32_t mask_of[SVW_MAX_LEN + 1];  // mask row of each of this CTA's rows; -1: none, -2: a bad row
  const int tid = threadIdx.x;
  const unsigned item = blockIdx.x / static_cast<unsigned>(a.groups);
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.groups));
  const int32_t i = static_cast<int32_t>(item / static_cast<unsigned>(a.chunks));
  const int32_t v0 = static_cast<int32_t>(item % static_cast<unsigned>(a.chunks)) * a.chunk_len;
  const int32_t len = min(a.chunk_len, a.V - v0);
  // counts | bias places (if any) | bitmap of the listed entries | their list
  int32_t *cnt = dyn, *bidx = dyn + a.chunk_len;
  uint32_t *mark = reinterpret_cast<uint32_t *>(dyn + a.chunk_len * (a.cu_bias ? 2 : 1));
  const int mark_words = a.chunk_len / 32;
  uint16_t *list = reinterpret_cast<uint16_t *>(mark + mark_words);

  // the request's offsets and factors, all under way at once
  const int32_t d0 = __ldg(a.cu + i), d1 = __ldg(a.cu + i + 1);
  int32_t h0 = 0, h1 = 0, pl = 0, b0 = 0, b1 = 0;
  if (a.cu_history) {
    h0 = __ldg(a.cu_history + i);
    h1 = __ldg(a.cu_history + i + 1);
    pl = a.prompt_len ? __ldg(a.prompt_len + i) : 0;
  }
  if (a.cu_bias) {
    b0 = __ldg(a.cu_bias + i);
    b1 = __ldg(a.cu_bias + i + 1);
  }
  AdjChunk ch;
  ch.rep = a.repetition ? __ldg(a.repetition + i) : 1.f;
  ch.freq = a.frequency ? __ldg(a.frequency + i) : 0.f;
  ch.pres = a.presence ? __ldg(a.presence + i) : 0.f;
  for (int u = tid * 4; u < a.chunk_len * (a.cu_bias ? 2 : 1) + mark_words; u += kAdjThreads * 4)
    *reinterpret_cast<int4 *>(dyn + u) = make_int4(0, 0, 0, 0);
  if (tid == 0) nd = nlist = 0;
  const int64_t L = static_cast<int64_t>(d1) - d0;
  const bool range_ok = d0 >= 0 && L >= 0 && d1 <= a.R && L <= SVW_MAX_LEN;
  if (tid == 0 && a.status && (!range_ok || (i == 0 && d0 != 0) || (i == a.N - 1 && d1 != a.R)))
    atomicOr(a.status, SVW_DEV_BAD_INPUT);
  if (!range_ok) return;
  // this CTA's rows: group, group + groups, ... of the request's
  const int rows = (static_cast<int>(L) + a.bonus - group + a.groups - 1) / a.groups;
  const int64_t row0 = static_cast<int64_t>(d0) + (a.bonus ? i : 0) + group;
  if (tid < rows) {
    const int64_t r = row0 + static_cast<int64_t>(tid) * a.groups;
    const int32_t m = a.mask ? (a.mask_row ? __ldg(a.mask_row + r) : static_cast<int32_t>(r)) : -1;
    const bool row_bad = m < -1 || (m >= 0 && m >= a.mask_rows);
    mask_of[tid] = row_bad ? -2 : m;
    if (row_bad && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  }
  bool bad = !(ch.rep > 0.f && ch.rep < INFINITY && fabsf(ch.freq) < INFINITY && fabsf(ch.pres) < INFINITY);
  bad |= h0 < 0 || h1 < h0 || h1 > a.total_history || pl < 0 || pl > h1 - h0;
  bad |= b0 < 0 || b1 < b0 || b1 > a.total_bias;
  if (bad) h1 = h0, b1 = b0;
  const int32_t *hist = a.history + h0;
  const int32_t hn = h1 - h0;
  __syncthreads();

  // ---- every entry: copied, masked ----

  const bool in_place = (a.out == a.logits);
  const T *in = reinterpret_cast<const T *>(a.logits) + row0 * a.in_stride + v0;
  T *out = reinterpret_cast<T *>(a.out) + row0 * a.out_stride + v0;
  const int64_t in_step = a.in_stride * a.groups, out_step = a.out_stride * a.groups;
  auto words_of = [&](int32_t m) { return a.mask + static_cast<int64_t>(m) * a.mask_words; };
  auto allowed = [&](int32_t m, int32_t v) { return m < 0 || ((__ldg(words_of(m) + (v >> 5)) >> (v & 31)) & 1u); };
  auto single = [&](int q, int u) {
    const bool ok = allowed(mask_of[q], v0 + u);
    if (!(in_place && ok)) out[q * out_step + u] = ok ? in[q * in_step + u] : static_cast<T>(B::kNegInf);
  };
  // entries of row q before its first 16-byte boundary
  auto head_of = [&](int q) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(in + q * in_step) & 15u;
    return min(len, static_cast<int>(((16u - at) & 15u) / sizeof(T)));
  };
  if (!VEC) {
    for (int q = 0; q < rows; ++q)
      for (int u = tid; u < len; u += kAdjThreads) single(q, u);
  } else {
    // kRowVecs vectors of a row per thread, kAdjBatch / kRowVecs rows at a time
    constexpr int kPerRow = VEC ? kRowVecs : 1, kRowsAtOnce = kAdjBatch / kPerRow;
    for (int q0 = 0; q0 < rows; q0 += kRowsAtOnce) {
      uint32_t ok[kAdjBatch];
      uint4 x[kAdjBatch];
#pragma unroll
      for (int b = 0; b < kAdjBatch; ++b) {
        const int q = q0 + b / kPerRow, k = tid + (b % kPerRow) * kAdjThreads;
        ok[b] = kNothing;
        if (q < rows) {
          const int head = head_of(q), v = v0 + head + k * EPV;
          if (head + (k + 1) * EPV <= len) {
            const int32_t m = mask_of[q];
            ok[b] = kAll;
            if (m >= 0)
              ok[b] = (head == 0) ? (__ldg(words_of(m) + (v >> 5)) >> (v & 31)) & kAll
                                  : bits_at(words_of(m), a.mask_words, v, EPV);
            if (in_place && ok[b] == kAll) ok[b] = kNothing;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kAdjBatch; ++b) {
        const int q = q0 + b / kPerRow, k = tid + (b % kPerRow) * kAdjThreads;
        if (ok[b] != 0 && ok[b] != kNothing) x[b] = *(reinterpret_cast<const uint4 *>(in + q * in_step + head_of(q)) + k);
      }
#pragma unroll
      for (int b = 0; b < kAdjBatch; ++b) {
        const int q = q0 + b / kPerRow, k = tid + (b % kPerRow) * kAdjThreads;
        if (ok[b] == kNothing) continue;
        if (ok[b] != kAll) {
          x[b].x = B::hide(x[b].x, ok[b], 0);
          x[b].y = B::hide(x[b].y, ok[b], 1);
          x[b].z = B::hide(x[b].z, ok[b], 2);
          x[b].w = B::hide(x[b].w, ok[b], 3);
        }
        *(reinterpret_cast<uint4 *>(out + q * out_step + head_of(q)) + k) = x[b];
      }
    }
    // what lies before the first and after the last boundary of each row
    for (int m = tid; m < rows * 2 * EPV; m += kAdjThreads) {
      const int r = m / (2 * EPV), e = m % (2 * EPV), head = head_of(r);
      const int tail = head + (len - head) / EPV * EPV;
      if (e < EPV ? e < head : tail + e - EPV < len) single(r, e < EPV ? e : tail + e - EPV);
    }
  }

  // ---- what the request has seen of the chunk ----

  auto look_at = [&](int32_t u) {
    const uint32_t bit = 1u << (u & 31);
    if (!(atomicOr(mark + (u >> 5), bit) & bit)) list[atomicAdd(&nlist, 1)] = static_cast<uint16_t>(u);
  };
  {
    auto count = [&](int32_t v, int32_t p) {
      const int32_t u = v - v0;
      if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(a.V))
        bad = true;
      else if (u >= 0 && u < len) {
        if (p < pl)
          atomicOr(cnt + u, kPromptBit);
        else
          atomicAdd(cnt + u, 1);
        look_at(u);
      }
    };
    for (int32_t p0 = tid; p0 < hn; p0 += kAhead * kAdjThreads) {
      int32_t ahead[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) ahead[q] = (p0 + q * kAdjThreads < hn) ? __ldg(hist + p0 + q * kAdjThreads) : 0;
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (p0 + q * kAdjThreads < hn) count(ahead[q], p0 + q * kAdjThreads);
    }
  }
  for (int32_t p = b0 + tid; p < b1; p += kAdjThreads) {
    const int32_t bias_v = __ldg(a.bias_tokens + p);
    const float bias_x = __ldg(a.bias_values + p);
    const int32_t u = bias_v - v0;
    if (static_cast<uint32_t>(bias_v) >= static_cast<uint32_t>(a.V) || !(bias_x < INFINITY))
      bad = true;
    else if (u >= 0 && u < len) {
      atomicMax(bidx + u, p + 1);
      look_at(u);
    }
  }
  if (tid < static_cast<int>(L)) {
    const int32_t draft = __ldg(a.tokens + d0 + tid);
    const int32_t u = draft - v0;
    if (static_cast<uint32_t>(draft) >= static_cast<uint32_t>(a.V))
      bad = true;
    else if (u >= 0 && u < len) {
      const int s = atomicAdd(&nd, 1);
      dtok[s] = u;
      dpos[s] = tid;
      look_at(u);
    }
  }
  bad = __syncthreads_or(bad);  // also: every vector is written
  if (bad && tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);

  // ---- the listed entries again, or a bad request's or row's NaN ----
  for (int q = 0; q < rows; ++q)
    if (bad || mask_of[q] == -2)
      for (int u = tid; u < len; u += kAdjThreads) out[q * out_step + u] = static_cast<T>(B::kNaN);
  if (bad) return;
  ch.cnt = cnt;
  ch.bidx = a.cu_bias ? bidx : nullptr;
  ch.bias_values = a.bias_values;
  ch.nd = nd;
  ch.dtok = dtok;
  ch.dpos = dpos;
  const int n = nlist;
  constexpr int kMany = 4;
  for (int m0 = tid; m0 < n * rows; m0 += kMany * kAdjThreads) {
    uint32_t x[kMany];
    int qs[kMany], us[kMany];
#pragma unroll
    for (int b = 0; b < kMany; ++b) {
      const int m = m0 + b * kAdjThreads;
      qs[b] = -1;
      if (m < n * rows) {
        const int q = m / n, u = list[m - q * n];
        if (mask_of[q] != -2 && allowed(mask_of[q], v0 + u)) {
          qs[b] = q;
          us[b] = u;
          x[b] = in[q * in_step + u];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kMany; ++b) {
      if (qs[b] < 0) continue;
      float y = B::value(x[b]);
      if (adjust_entry(ch, us[b], group + qs[b] * a.groups, y)) out[qs[b] * out_step + us[b]] = static_cast<T>(B::bits(y));
    }
  }
}

}  // namespace

cudaError_t launch_adjust(const AdjustArgs &args, int dtype, cudaStream_t st) {
  AdjustArgs a = args;
  const int es = dtype == SVW_BF16 ? 2 : 4;
  // 4096 entries a chunk (41 KB of shared memory with biases: five CTAs per SM);
  // fewer where the batch would leave SMs without work, then the rows of a
  // request are shared out too
  constexpr int64_t kFull = 2 * 152;
  a.chunk_len = 4096;
  while (a.chunk_len > 1024 && a.N * ((a.V + a.chunk_len - 1) / static_cast<int64_t>(a.chunk_len)) < kFull) a.chunk_len /= 2;
  a.chunks = (a.V + a.chunk_len - 1) / a.chunk_len;
  const int64_t rows = a.R / a.N + (a.bonus ? 1 : 0);  // of a request, on average
  const int64_t want = kFull / (a.N * static_cast<int64_t>(a.chunks));
  a.groups = static_cast<int32_t>(want < 1 ? 1 : (want > rows ? (rows < 1 ? 1 : rows) : want));
  const int64_t grid = static_cast<int64_t>(a.N) * a.chunks * a.groups;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(a.chunk_len) * (4 * (a.cu_bias ? 2 : 1) + 2) + a.chunk_len / 8;
  const uintptr_t apart = reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out);
  const bool vec = (apart & 15u) == 0 && ((a.in_stride - a.out_stride) * es) % 16 == 0;
  void *tm = timer_before("logits_adjust", st);
  const dim3 g(static_cast<unsigned>(grid)), b(kAdjThreads);
  const int row_vecs = vec ? (a.chunk_len * es / 16 + kAdjThreads - 1) / kAdjThreads : 0;  // 0, 1, 2 or 4
#define SVW_ADJUST(DT, RV) logits_adjust_kernel<DT, RV><<<g, b, smem, st>>>(a)
  if (dtype == SVW_BF16) {
    if (row_vecs == 0)
      SVW_ADJUST(1, 0);
    else if (row_vecs == 1)
      SVW_ADJUST(1, 1);
    else
      SVW_ADJUST(1, 2);
  } else {
    if (row_vecs == 0)
      SVW_ADJUST(0, 0);
    else if (row_vecs == 1)
      SVW_ADJUST(0, 1);
    else if (row_vecs == 2)
      SVW_ADJUST(0, 2);
    else
      SVW_ADJUST(0, 4);
  }
#undef SVW_ADJUST
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
