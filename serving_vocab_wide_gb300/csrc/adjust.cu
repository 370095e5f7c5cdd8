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
// the drafted ones, each once.  Then it walks the request's rows over that
// chunk twice: all entries in 16-byte vectors, copied with the mask applied by
// selection (a vector that is all masked is written without being read; in
// place, one that is all allowed is left alone), and after a barrier the
// listed entries one by one.  (Looking at listed entries inside the first walk
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
constexpr int kAdjBatch = 4;  // vectors of a thread in flight
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

// VEC: the two rows of every row pair lie equally far from a 16-byte boundary
template <int DT, bool VEC>
__global__ void __launch_bounds__(kAdjThreads) logits_adjust_kernel(AdjustArgs a) {
  using B = Bits<DT>;
  using T = typename B::T;
  constexpr int EPV = 16 / sizeof(T);
  constexpr uint32_t kAll = (1u << EPV) - 1u;
  extern __shared__ int32_t dyn[];
  __shared__ int32_t dtok[SVW_MAX_LEN], dpos[SVW_MAX_LEN], nd, nlist;
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
  const int rows = static_cast<int>(L) + a.bonus;
  const int64_t row0 = static_cast<int64_t>(d0) + (a.bonus ? i : 0);
  bool bad = !(ch.rep > 0.f && ch.rep < INFINITY && fabsf(ch.freq) < INFINITY && fabsf(ch.pres) < INFINITY);
  bad |= h0 < 0 || h1 < h0 || h1 > a.total_history || pl < 0 || pl > h1 - h0;
  bad |= b0 < 0 || b1 < b0 || b1 > a.total_bias;
  if (bad) h1 = h0, b1 = b0;
  __syncthreads();
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
    const int32_t *hist = a.history + h0;
    const int32_t n = h1 - h0;
    int32_t p = tid;
    for (; p + 3 * kAdjThreads < n; p += 4 * kAdjThreads) {
      int32_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __ldg(hist + p + q * kAdjThreads);
#pragma unroll
      for (int q = 0; q < 4; ++q) count(v[q], p + q * kAdjThreads);
    }
    for (; p < n; p += kAdjThreads) count(__ldg(hist + p), p);
  }
  for (int32_t p = b0 + tid; p < b1; p += kAdjThreads) {
    const int32_t v = __ldg(a.bias_tokens + p);
    const int32_t u = v - v0;
    if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(a.V) || !(__ldg(a.bias_values + p) < INFINITY))
      bad = true;
    else if (u >= 0 && u < len) {
      atomicMax(bidx + u, p + 1);
      look_at(u);
    }
  }
  if (tid < static_cast<int>(L)) {
    const int32_t v = __ldg(a.tokens + d0 + tid);
    const int32_t u = v - v0;
    if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(a.V))
      bad = true;
    else if (u >= 0 && u < len) {
      const int s = atomicAdd(&nd, 1);
      dtok[s] = u;
      dpos[s] = tid;
      look_at(u);
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  ch.cnt = cnt;
  ch.bidx = a.cu_bias ? bidx : nullptr;
  ch.bias_values = a.bias_values;
  ch.nd = nd;
  ch.dtok = dtok;
  ch.dpos = dpos;

  const bool in_place = (a.out == a.logits);
  for (int j = group; j < rows; j += a.groups) {
    const int64_t r = row0 + j;
    const T *in = reinterpret_cast<const T *>(a.logits) + r * a.in_stride + v0;
    T *out = reinterpret_cast<T *>(a.out) + r * a.out_stride + v0;
    const int32_t mr = a.mask ? (a.mask_row ? __ldg(a.mask_row + r) : static_cast<int32_t>(r)) : -1;
    const bool row_bad = mr < -1 || (mr >= 0 && mr >= a.mask_rows);
    if (row_bad && tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
    if (bad || row_bad) {
      for (int u = tid; u < len; u += kAdjThreads) out[u] = static_cast<T>(B::kNaN);
      continue;
    }
    const uint32_t *mw = (mr >= 0) ? a.mask + static_cast<int64_t>(mr) * a.mask_words : nullptr;
    auto single = [&](int u) {
      const bool ok = !mw || ((__ldg(mw + ((v0 + u) >> 5)) >> ((v0 + u) & 31)) & 1u);
      if (!(in_place && ok)) out[u] = ok ? in[u] : static_cast<T>(B::kNegInf);
    };
    if (!VEC) {
      for (int u = tid; u < len; u += kAdjThreads) single(u);
      continue;
    }
    // the row's entries before its first 16-byte boundary and after its last
    const int head = min(len, static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(in) & 15u)) & 15u) / sizeof(T)));
    const int nvec = (len - head) / EPV;
    if (tid < head) single(tid);
    if (tid < len - head - nvec * EPV) single(head + nvec * EPV + tid);
    const uint4 *vin = reinterpret_cast<const uint4 *>(in + head);
    uint4 *vout = reinterpret_cast<uint4 *>(out + head);
    for (int k0 = tid; k0 < nvec; k0 += kAdjThreads * kAdjBatch) {
      uint32_t ok[kAdjBatch];
      uint4 x[kAdjBatch];
#pragma unroll
      for (int q = 0; q < kAdjBatch; ++q) {
        const int k = k0 + q * kAdjThreads, v = v0 + head + k * EPV;
        ok[q] = kAll;
        if (mw && k < nvec)
          ok[q] = (head == 0) ? (__ldg(mw + (v >> 5)) >> (v & 31)) & kAll : bits_at(mw, a.mask_words, v, EPV);
      }
#pragma unroll
      for (int q = 0; q < kAdjBatch; ++q) {
        const int k = k0 + q * kAdjThreads;
        if (k < nvec && ok[q] != 0 && !(in_place && ok[q] == kAll)) x[q] = __ldcs(vin + k);
      }
#pragma unroll
      for (int q = 0; q < kAdjBatch; ++q) {
        const int k = k0 + q * kAdjThreads;
        if (k >= nvec || (in_place && ok[q] == kAll)) continue;
        if (ok[q] != kAll) {
          x[q].x = B::hide(x[q].x, ok[q], 0);
          x[q].y = B::hide(x[q].y, ok[q], 1);
          x[q].z = B::hide(x[q].z, ok[q], 2);
          x[q].w = B::hide(x[q].w, ok[q], 3);
        }
        __stcs(vout + k, x[q]);
      }
    }
  }
  if (bad || nlist == 0) return;
  __syncthreads();  // the listed entries are written again after their vectors
  const int n = nlist, mine = (rows - group + a.groups - 1) / a.groups;  // this CTA's rows
  for (int m = tid; m < n * mine; m += kAdjThreads) {
    const int q = m / n, u = list[m - q * n], j = group + q * a.groups;
    const int64_t r = row0 + j;
    const int32_t mr = a.mask ? (a.mask_row ? __ldg(a.mask_row + r) : static_cast<int32_t>(r)) : -1;
    if (mr < -1 || (mr >= 0 && mr >= a.mask_rows)) continue;  // a bad row: NaN
    if (mr >= 0 && !((__ldg(a.mask + static_cast<int64_t>(mr) * a.mask_words + ((v0 + u) >> 5)) >> ((v0 + u) & 31)) & 1u))
      continue;  // masked: -inf
    float y = B::value((reinterpret_cast<const T *>(a.logits) + r * a.in_stride + v0)[u]);
    if (adjust_entry(ch, u, j, y))
      (reinterpret_cast<T *>(a.out) + r * a.out_stride + v0)[u] = static_cast<T>(B::bits(y));
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
  if (dtype == SVW_BF16) {
    if (vec)
      logits_adjust_kernel<1, true><<<g, b, smem, st>>>(a);
    else
      logits_adjust_kernel<1, false><<<g, b, smem, st>>>(a);
  } else {
    if (vec)
      logits_adjust_kernel<0, true><<<g, b, smem, st>>>(a);
    else
      logits_adjust_kernel<0, false><<<g, b, smem, st>>>(a);
  }
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
