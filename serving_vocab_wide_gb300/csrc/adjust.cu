// adjust.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of drafted positions (logits_adjust).
//
// Row j of request i has seen the request's history and its drafted tokens
// x_0 .. x_{j-1}; with n(v) the occurrences of v after the prompt part,
//   y = logits[row, v];  seen: y = y > 0 ? y / rep : y rep;
//   n > 0: y -= freq n + pres;  y += bias(v);  mask bit 0: y = -inf.
//
// One CTA owns a chunk of the vocabulary of one request: it counts the
// history's tokens that fall into its chunk in shared memory (32-bit integer
// atomics: the order does not matter), then walks the request's rows over that
// chunk.  The drafted prefix differs from row to row and is not counted: the
// chunk's drafted tokens (at most SVW_MAX_LEN) are kept as a list and
// compared by the entries that hold one of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kAdjThreads = 256;
constexpr int32_t kPromptBit = static_cast<int32_t>(0x80000000u);

__device__ __forceinline__ float elem_f(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float elem_f(float x) { return x; }
__device__ __forceinline__ void elem_store(uint16_t &o, float x) { o = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void elem_store(float &o, float x) { o = x; }

template <int DT>
struct Store;
template <>
struct Store<1> {
  using T = uint16_t;
};
template <>
struct Store<0> {
  using T = float;
};

// what a CTA knows of its request and chunk
struct AdjChunk {
  int32_t *cnt;    // [CH] occurrences after the prompt part | kPromptBit
  int32_t *bidx;   // [CH] 1 + the last place in the bias list that names the token (0: none)
  int32_t dtok[SVW_MAX_LEN], dpos[SVW_MAX_LEN];  // the chunk's drafted tokens and their positions
  int32_t nd;
  float rep, freq, pres;
};

// the entry's value after penalties and bias; false: it stays as it is
__device__ __forceinline__ bool adjust_entry(const AdjChunk &c, const AdjustArgs &a, int u, int j, float &y) {
  const int32_t w = c.cnt[u];
  int32_t n = w & ~kPromptBit;
  for (int d = 0; d < c.nd; ++d) n += (c.dtok[d] == u && c.dpos[d] < j) ? 1 : 0;
  const bool seen = (w != 0) || (n > 0);
  const int32_t b = a.cu_bias ? c.bidx[u] : 0;
  if (!seen && b == 0) return false;
  if (seen) y = (y > 0.f) ? __fdiv_rn(y, c.rep) : __fmul_rn(y, c.rep);
  if (n > 0) y = __fsub_rn(__fsub_rn(y, __fmul_rn(c.freq, static_cast<float>(n))), c.pres);
  if (b != 0) y = __fadd_rn(y, __ldg(a.bias_values + b - 1));
  return true;
}

template <int DT>
__global__ void __launch_bounds__(kAdjThreads) logits_adjust_kernel(AdjustArgs a) {
  using T = typename Store<DT>::T;
  extern __shared__ int32_t dyn[];
  __shared__ AdjChunk ch;
  const int tid = threadIdx.x;
  const int64_t item = blockIdx.x / a.groups;
  const int group = static_cast<int>(blockIdx.x % a.groups);
  const int32_t i = static_cast<int32_t>(item / a.chunks);
  const int32_t v0 = static_cast<int32_t>(item % a.chunks) * a.chunk_len;
  const int32_t len = min(a.chunk_len, a.V - v0);

  const int32_t d0 = __ldg(a.cu + i), d1 = __ldg(a.cu + i + 1);
  const int64_t L = static_cast<int64_t>(d1) - d0;
  if ((i == 0 && d0 != 0) || (i == a.N - 1 && d1 != a.R) || d0 < 0 || L < 0 || d1 > a.R || L > SVW_MAX_LEN) {
    if (tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
    if (d0 < 0 || L < 0 || d1 > a.R || L > SVW_MAX_LEN) return;
  }
  const int rows = static_cast<int>(L) + a.bonus;
  const int64_t row0 = static_cast<int64_t>(d0) + (a.bonus ? i : 0);

  for (int u = tid; u < len; u += kAdjThreads) {
    dyn[u] = 0;
    if (a.cu_bias) dyn[a.chunk_len + u] = 0;
  }
  bool bad = false;
  if (tid == 0) {
    ch.cnt = dyn;
    ch.bidx = dyn + a.chunk_len;
    ch.nd = 0;
    ch.rep = a.repetition ? __ldg(a.repetition + i) : 1.f;
    ch.freq = a.frequency ? __ldg(a.frequency + i) : 0.f;
    ch.pres = a.presence ? __ldg(a.presence + i) : 0.f;
    bad = !(ch.rep > 0.f && ch.rep < INFINITY && fabsf(ch.freq) < INFINITY && fabsf(ch.pres) < INFINITY);
  }
  __syncthreads();
  if (a.cu_history) {
    const int32_t h0 = __ldg(a.cu_history + i), h1 = __ldg(a.cu_history + i + 1);
    const int32_t pl = a.prompt_len ? __ldg(a.prompt_len + i) : 0;
    if (h0 < 0 || h1 < h0 || h1 > a.total_history || pl < 0 || pl > h1 - h0) {
      bad = true;
    } else {
      for (int32_t p = tid; p < h1 - h0; p += kAdjThreads) {
        const int32_t v = __ldg(a.history + h0 + p);
        const int32_t u = v - v0;
        if (v < 0 || v >= a.V)
          bad = true;
        else if (u >= 0 && u < len) {
          if (p < pl)
            atomicOr(dyn + u, kPromptBit);
          else
            atomicAdd(dyn + u, 1);
        }
      }
    }
  }
  if (a.cu_bias) {
    const int32_t b0 = __ldg(a.cu_bias + i), b1 = __ldg(a.cu_bias + i + 1);
    if (b0 < 0 || b1 < b0 || b1 > a.total_bias) {
      bad = true;
    } else {
      for (int32_t p = b0 + tid; p < b1; p += kAdjThreads) {
        const int32_t v = __ldg(a.bias_tokens + p);
        const int32_t u = v - v0;
        if (v < 0 || v >= a.V || !(__ldg(a.bias_values + p) < INFINITY))
          bad = true;
        else if (u >= 0 && u < len)
          atomicMax(dyn + a.chunk_len + u, p + 1);
      }
    }
  }
  if (tid < static_cast<int>(L)) {
    const int32_t v = __ldg(a.tokens + d0 + tid);
    const int32_t u = v - v0;
    if (v < 0 || v >= a.V)
      bad = true;
    else if (u >= 0 && u < len) {
      const int s = atomicAdd(&ch.nd, 1);
      ch.dtok[s] = u;
      ch.dpos[s] = tid;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);

  for (int j = group; j < rows; j += a.groups) {
    const int64_t r = row0 + j;
    const T *in = reinterpret_cast<const T *>(a.logits) + r * a.in_stride + v0;
    T *out = reinterpret_cast<T *>(a.out) + r * a.out_stride + v0;
    const int32_t mr = a.mask ? (a.mask_row ? __ldg(a.mask_row + r) : static_cast<int32_t>(r)) : -1;
    const bool row_bad = mr < -1 || (mr >= 0 && mr >= a.mask_rows);
    if (row_bad && tid == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
    if (bad || row_bad) {
      for (int u = tid; u < len; u += kAdjThreads) elem_store(out[u], __int_as_float(0x7fffffff));
      continue;
    }
    const uint32_t *mw = a.mask + static_cast<int64_t>(max(mr, 0)) * a.mask_words;
    for (int u = tid; u < len; u += kAdjThreads) {
      const int32_t v = v0 + u;
      T x = in[u];
      if (mr >= 0 && !((__ldg(mw + (v >> 5)) >> (v & 31)) & 1u)) {
        elem_store(x, -INFINITY);
      } else {
        float y = elem_f(x);
        if (adjust_entry(ch, a, u, j, y)) elem_store(x, y);
      }
      out[u] = x;
    }
  }
}

}  // namespace

cudaError_t launch_adjust(const AdjustArgs &args, int dtype, cudaStream_t st) {
  AdjustArgs a = args;
  a.chunk_len = 4096;
  a.chunks = (a.V + a.chunk_len - 1) / a.chunk_len;
  a.groups = 1;
  const int64_t grid = static_cast<int64_t>(a.N) * a.chunks * a.groups;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(a.chunk_len) * 4 * (a.cu_bias ? 2 : 1);
  void *tm = timer_before("logits_adjust", st);
  if (dtype == SVW_BF16)
    logits_adjust_kernel<1><<<static_cast<unsigned>(grid), kAdjThreads, smem, st>>>(a);
  else
    logits_adjust_kernel<0><<<static_cast<unsigned>(grid), kAdjThreads, smem, st>>>(a);
  timer_after(tm, st);
  return cudaGetLastError();
}

}  // namespace svw
