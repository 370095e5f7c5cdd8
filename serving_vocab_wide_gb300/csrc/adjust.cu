// adjust.cu -- penalties for repeated tokens, biases and grammar masks on the
// logits of drafted positions (logits_adjust).
//
// Row j of request i has seen the request's history and its drafted tokens
// x_0 .. x_{j-1}; with n(v) the occurrences of v after the prompt part,
//   y = logits[row, v];  seen: y = y > 0 ? y / rep : y rep;
//   n > 0: y -= freq n + pres;  y += bias(v);  mask bit 0: y = -inf.
//
// Bound by bytes: a row is read and written once, and few of its entries
// change.  Those that the history, the biases or the drafts name are listed and
// written apart from the stream of vectors.  (Looking at them inside the stream
// took 929 us on the benchmark batch, 256 requests, 2220 bf16 rows of 151936,
// histories of 128 to 8192 tokens, 1356 MB: some lane of nearly every warp has
// one.  The batch's floor is 200 us; a plain copy of it takes 200.)  Counts are
// 32-bit integers, so the order of the atomics that add them up does not
// matter.  The drafted prefix differs from row to row and is not counted: a
// listed entry that is drafted looks through the request's drafts (at most
// SVW_MAX_LEN).
//
// Large batches (given a workspace), 225 us on the benchmark batch (6.0 TB/s):
//   adjust_lists   a CTA per request lists its distinct tokens, ascending, with
//                  their counts (15 to 17 us by itself where the longest
//                  history has 8192, partly beside the rows' first loads);
//   adjust_staged  a CTA per chunk of 8 KB of a request's rows: they pass
//                  through shared memory by bulk copies, masked and adjusted on
//                  the way; seven CTAs of three 8 KB stages per SM (four stages
//                  and five CTAs: 240 us; the rows in registers and the listed
//                  entries by a second trip to memory: 329);
//   adjust_rows    in place, 92 us without masks and 258 with (only what
//                  changes is written; a vector's load waits for its mask
//                  word), or rows that do not lie alike.
// Small batches, one launch: adjust_chunks, a CTA counts the tokens of its chunk
// itself by reading the whole history (4.1 us for one row of 32000; on the
// benchmark batch: 329, each of 38 chunks of a request waits for its loads.
// Counting beside staged rows' loads was slower than the lists for all but few
// requests: 43 us where the lists took 39 on 544 fp32 rows of 32003, now 34.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjBatch = 4;  // vectors of a thread under way
constexpr int kAhead = 8;     // history tokens of a thread under way
constexpr int kChunk = 4096;  // entries of a chunk, unless the batch is small
// of the lists, and of rows that are staged: 8 KB (with 16 KB of fp32 there
// are four CTAs of three stages per SM instead of seven: 544 masked rows of
// 32003 took 33.1 us instead of 30.4; in place, through registers, the larger
// chunks are the faster ones, 34 against 42)
__host__ __device__ constexpr int list_shift(int es) { return es == 2 ? 12 : 11; }
__host__ __device__ constexpr int list_chunk(int es) { return 1 << list_shift(es); }
static_assert(list_chunk(2) == kChunk && list_chunk(4) * 2 == kChunk, "a chunk is one or two of the lists'");
constexpr uint32_t kNothing = 0x100;  // no vector to write
constexpr int32_t kPromptBit = static_cast<int32_t>(0x80000000u);
constexpr int32_t kDraftBit = 0x40000000;  // lists: the token is drafted too

// a request's factors
struct Factors {
  float rep, freq, pres;
  __device__ bool fine() const {
    return rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY;
  }
};
__device__ __forceinline__ Factors factors_of(const AdjustArgs &a, int32_t i) {
  Factors f;
  f.rep = a.repetition ? __ldg(a.repetition + i) : 1.f;
  f.freq = a.frequency ? __ldg(a.frequency + i) : 0.f;
  f.pres = a.presence ? __ldg(a.presence + i) : 0.f;
  return f;
}
// an entry's value after penalties and bias: n occurrences after the prompt
// part, `seen` there or in it; false: it stays as it is
__device__ __forceinline__ bool adjust_entry(const Factors &f, int32_t n, bool seen, bool biased, float bias, float &y) {
  if (!seen && !biased) return false;
  if (seen) y = (y > 0.f) ? __fdiv_rn(y, f.rep) : __fmul_rn(y, f.rep);
  if (n > 0) y = __fsub_rn(__fsub_rn(y, __fmul_rn(f.freq, static_cast<float>(n))), f.pres);
  if (biased) y = __fadd_rn(y, bias);
  return true;
}

// One more, for each of the lanes that come here together: one addition of a
// warp instead of one a lane (4.5 thousand additions to one address of shared
// memory took 45 us).  Returns the lane's number.
__device__ __forceinline__ int32_t one_more(int32_t *counter) {
  const uint32_t here = __activemask();
  const int lane = threadIdx.x & 31, first = __ffs(here) - 1;
  int32_t at = 0;
  if (lane == first) at = atomicAdd(counter, __popc(here));
  return __shfl_sync(here, at, first) + __popc(here & ((1u << lane) - 1u));
}

// a request's slices of the three lists; false: they are inconsistent
struct Slices {
  int32_t d0, d1, h0, h1, pl, b0, b1;
};
__device__ __forceinline__ Slices slices_of(const AdjustArgs &a, int32_t i) {
  Slices s = {__ldg(a.cu + i), __ldg(a.cu + i + 1), 0, 0, 0, 0, 0};
  if (a.cu_history) {
    s.h0 = __ldg(a.cu_history + i);
    s.h1 = __ldg(a.cu_history + i + 1);
    s.pl = a.prompt_len ? __ldg(a.prompt_len + i) : 0;
  }
  if (a.cu_bias) {
    s.b0 = __ldg(a.cu_bias + i);
    s.b1 = __ldg(a.cu_bias + i + 1);
  }
  return s;
}
__device__ __forceinline__ bool rows_fine(const AdjustArgs &a, const Slices &s) {
  return s.d0 >= 0 && s.d1 >= s.d0 && s.d1 <= a.R && s.d1 - s.d0 <= SVW_MAX_LEN;
}
__device__ __forceinline__ bool lists_fine(const AdjustArgs &a, const Slices &s) {
  return s.h0 >= 0 && s.h1 >= s.h0 && s.h1 <= a.total_history && s.pl >= 0 && s.pl <= s.h1 - s.h0 && s.b0 >= 0 &&
         s.b1 >= s.b0 && s.b1 <= a.total_bias;
}
__device__ __forceinline__ void report(const AdjustArgs &a) {
  if (a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
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

// A CTA's rows over its chunk [v0, v0 + len): row q of `rows` at in + q *
// in_step, mask row mask_of[q] (-1: none, -2: a bad row)
template <int DT>
struct Rows {
  using B = Bits<DT>;
  using T = typename B::T;
  const T *in;
  T *out;
  int64_t in_step, out_step;
  int rows, len;
  int32_t v0;
  const uint32_t *mask;
  int64_t mask_words;
  const int32_t *mask_of;
  __device__ const uint32_t *words(int32_t m) const { return mask + static_cast<int64_t>(m) * mask_words; }
  __device__ bool allowed(int32_t m, int32_t v) const {
    return m < 0 || ((__ldg(words(m) + (v >> 5)) >> (v & 31)) & 1u);
  }
  __device__ bool in_place() const { return out == in; }
  // entries of row q before its first 16-byte boundary
  __device__ int head(int q) const {
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(in + q * in_step)) & 15u;
    return min(len, static_cast<int>(((16u - at) & 15u) / sizeof(T)));
  }
  __device__ void single(int q, int u) const {
    const bool ok = allowed(mask_of[q], v0 + u);
    if (!(in_place() && ok)) out[q * out_step + u] = ok ? in[q * in_step + u] : static_cast<T>(B::kNegInf);
  }
};

// this CTA's rows of the request (group, group + groups, ...) over chunk c; fills mask_of
template <int DT>
__device__ __forceinline__ Rows<DT> rows_of(const AdjustArgs &a, const Slices &s, int32_t i, int32_t c, int group,
                                            int32_t *mask_of) {
  using T = typename Bits<DT>::T;
  Rows<DT> r;
  r.rows = (s.d1 - s.d0 + a.bonus - group + a.groups - 1) / a.groups;
  r.v0 = c * a.chunk_len;
  r.len = min(a.chunk_len, a.V - r.v0);
  const int64_t row0 = static_cast<int64_t>(s.d0) + (a.bonus ? i : 0) + group;
  r.in = reinterpret_cast<const T *>(a.logits) + row0 * a.in_stride + r.v0;
  r.out = reinterpret_cast<T *>(a.out) + row0 * a.out_stride + r.v0;
  r.in_step = a.in_stride * a.groups;
  r.out_step = a.out_stride * a.groups;
  r.mask = a.mask;
  r.mask_words = a.mask_words;
  r.mask_of = mask_of;
  if (static_cast<int>(threadIdx.x) < r.rows) {
    const int64_t row = row0 + static_cast<int64_t>(threadIdx.x) * a.groups;
    const int32_t m = a.mask ? (a.mask_row ? __ldg(a.mask_row + row) : static_cast<int32_t>(row)) : -1;
    const bool row_bad = m < -1 || (m >= 0 && m >= a.mask_rows);
    mask_of[threadIdx.x] = row_bad ? -2 : m;
    if (row_bad) report(a);
  }
  return r;
}

// Every entry copied, masked.  kRowVecs: vectors of a chunk's row per thread,
// kAdjBatch / kRowVecs rows at a time; 0: the input and output rows do not lie
// equally far from a 16-byte boundary, entry by entry.
template <int DT, int kRowVecs>
__device__ __forceinline__ void stream_rows(const Rows<DT> &r) {
  using B = Bits<DT>;
  constexpr int EPV = 16 / sizeof(typename B::T);
  constexpr uint32_t kAll = (1u << EPV) - 1u;
  const int tid = threadIdx.x;
  const bool in_place = r.in_place();
  if (in_place && r.mask == nullptr) return;
  if (kRowVecs == 0) {
    for (int q = 0; q < r.rows; ++q)
      for (int u = tid; u < r.len; u += kAdjThreads) r.single(q, u);
    return;
  }
  constexpr int kPerRow = kRowVecs > 0 ? kRowVecs : 1, kRowsAtOnce = kAdjBatch / kPerRow;
  for (int q0 = 0; q0 < r.rows; q0 += kRowsAtOnce) {
    uint32_t ok[kAdjBatch];
    uint4 x[kAdjBatch];
#pragma unroll
    for (int b = 0; b < kAdjBatch; ++b) {
      const int q = q0 + b / kPerRow, k = tid + (b % kPerRow) * kAdjThreads;
      ok[b] = kNothing;
      if (q < r.rows) {
        const int head = r.head(q), v = r.v0 + head + k * EPV;
        if (head + (k + 1) * EPV <= r.len) {
          const int32_t m = r.mask_of[q];
          ok[b] = kAll;
          if (m >= 0)
            ok[b] = (head == 0) ? (__ldg(r.words(m) + (v >> 5)) >> (v & 31)) & kAll
                                : bits_at(r.words(m), r.mask_words, v, EPV);
          if (in_place && ok[b] == kAll) ok[b] = kNothing;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kAdjBatch; ++b) {
      const int q = q0 + b / kPerRow, k = tid + (b % kPerRow) * kAdjThreads;
      if (ok[b] != 0 && ok[b] != kNothing) x[b] = *(reinterpret_cast<const uint4 *>(r.in + q * r.in_step + r.head(q)) + k);
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
      *(reinterpret_cast<uint4 *>(r.out + q * r.out_step + r.head(q)) + k) = x[b];
    }
  }
  // what lies before the first and after the last boundary of each row
  for (int q = 0; q < r.rows; ++q) {
    const int head = r.head(q), tail = head + (r.len - head) / EPV * EPV;
    if (head == 0 && tail == r.len) continue;
    if (tid < head) r.single(q, tid);
    if (tid >= 32 && tail + tid - 32 < r.len) r.single(q, tail + tid - 32);
  }
}

// a bad request's rows, or the bad rows: NaN
template <int DT>
__device__ __forceinline__ void spoil_rows(const Rows<DT> &r, bool bad) {
  for (int q = 0; q < r.rows; ++q)
    if (bad || r.mask_of[q] == -2)
      for (int u = threadIdx.x; u < r.len; u += kAdjThreads)
        r.out[q * r.out_step + u] = static_cast<typename Bits<DT>::T>(Bits<DT>::kNaN);
}

// The n listed entries of every row: at(k, u, w, b) gives entry k's place in the
// chunk, count word and bias place; drafted(w, u, j) its occurrences among the
// drafts before position j.
template <int DT, typename At, typename Drafted>
__device__ __forceinline__ void apply_listed(const AdjustArgs &a, const Rows<DT> &r, const Factors &f, int n, int group,
                                             At at, Drafted drafted) {
  using B = Bits<DT>;
  using T = typename B::T;
  constexpr int kMany = 4;
  for (int m0 = threadIdx.x; m0 < n * r.rows; m0 += kMany * kAdjThreads) {
    uint32_t x[kMany];
    int32_t us[kMany], ws[kMany], bs[kMany];
    int qs[kMany];
#pragma unroll
    for (int e = 0; e < kMany; ++e) {
      const int m = m0 + e * kAdjThreads;
      qs[e] = -1;
      if (m < n * r.rows) {
        const int q = m / n;
        at(m - q * n, us[e], ws[e], bs[e]);
        x[e] = r.in[q * r.in_step + us[e]];  // beside the mask's word, not behind it
        if (r.mask_of[q] != -2 && r.allowed(r.mask_of[q], r.v0 + us[e])) qs[e] = q;
      }
    }
#pragma unroll
    for (int e = 0; e < kMany; ++e) {
      if (qs[e] < 0) continue;
      const int32_t c = drafted(ws[e], us[e], group + qs[e] * a.groups);
      const int32_t n_seen = (ws[e] & ~(kPromptBit | kDraftBit)) + c;
      float y = B::value(x[e]);
      const float bias = bs[e] != 0 ? __ldg(a.bias_values + bs[e] - 1) : 0.f;
      if (adjust_entry(f, n_seen, n_seen > 0 || (ws[e] & kPromptBit) != 0, bs[e] != 0, bias, y))
        r.out[qs[e] * r.out_step + us[e]] = static_cast<T>(B::bits(y));
    }
  }
}

// ---------------------------------------------------------------------------
// what a request has seen of a chunk, counted by the chunk's CTA
// ---------------------------------------------------------------------------
// in shared memory: counts | bias places (if any) | bitmap of the listed entries | their list
struct Seen {
  int32_t *cnt, *bidx;
  uint32_t *mark;
  uint16_t *list;
};
struct SeenShared {
  int32_t dtok[SVW_MAX_LEN], dpos[SVW_MAX_LEN], nd, nlist;
};
__host__ __device__ constexpr int seen_bytes(int chunk_len, bool bias) {
  return chunk_len * (4 * (bias ? 2 : 1) + 2) + chunk_len / 8;
}
__device__ __forceinline__ Seen seen_at(int32_t *at, int chunk_len, bool bias) {
  Seen s;
  s.cnt = at;
  s.bidx = bias ? at + chunk_len : nullptr;
  s.mark = reinterpret_cast<uint32_t *>(at + chunk_len * (bias ? 2 : 1));
  s.list = reinterpret_cast<uint16_t *>(s.mark + chunk_len / 32);
  return s;
}
__device__ __forceinline__ void clear_seen(const Seen &s, SeenShared &sh, int chunk_len) {
  const int words = chunk_len * (s.bidx ? 2 : 1) + chunk_len / 32;
  for (int u = threadIdx.x * 4; u < words; u += kAdjThreads * 4) *reinterpret_cast<int4 *>(s.cnt + u) = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) sh.nd = sh.nlist = 0;
}
// true: some token or bias value is out of range (this thread's)
__device__ __forceinline__ bool count_seen(const AdjustArgs &a, const Slices &s, const Seen &n, SeenShared &sh, int32_t v0,
                                           int32_t len) {
  const int tid = threadIdx.x;
  const uint32_t V = static_cast<uint32_t>(a.V);
  bool bad = false;
  auto look_at = [&](int32_t u) {
    const uint32_t bit = 1u << (u & 31);
    if (!(atomicOr(n.mark + (u >> 5), bit) & bit)) n.list[one_more(&sh.nlist)] = static_cast<uint16_t>(u);
  };
  const int32_t *hist = a.history + s.h0;
  const int32_t hn = s.h1 - s.h0, L = s.d1 - s.d0;
  // the first of each list on their way together
  const bool has_bias = s.b0 + tid < s.b1;
  int32_t bias_v = has_bias ? __ldg(a.bias_tokens + s.b0 + tid) : 0;
  float bias_x = has_bias ? __ldg(a.bias_values + s.b0 + tid) : 0.f;
  const int32_t draft = tid < L ? __ldg(a.tokens + s.d0 + tid) : 0;
  for (int32_t p0 = tid; p0 < hn; p0 += kAhead * kAdjThreads) {
    int32_t ahead[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) ahead[q] = (p0 + q * kAdjThreads < hn) ? __ldg(hist + p0 + q * kAdjThreads) : 0;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int32_t p = p0 + q * kAdjThreads, u = ahead[q] - v0;
      if (p >= hn) break;
      bad |= static_cast<uint32_t>(ahead[q]) >= V;
      if (u >= 0 && u < len) {
        if (p < s.pl)
          atomicOr(n.cnt + u, kPromptBit);
        else
          atomicAdd(n.cnt + u, 1);
        look_at(u);
      }
    }
  }
  for (int32_t p = s.b0 + tid; p < s.b1; p += kAdjThreads) {
    if (p != s.b0 + tid) {
      bias_v = __ldg(a.bias_tokens + p);
      bias_x = __ldg(a.bias_values + p);
    }
    const int32_t u = bias_v - v0;
    bad |= static_cast<uint32_t>(bias_v) >= V || !(bias_x < INFINITY);
    if (u >= 0 && u < len) {
      atomicMax(n.bidx + u, p + 1);
      look_at(u);
    }
  }
  if (tid < L) {
    const int32_t u = draft - v0;
    bad |= static_cast<uint32_t>(draft) >= V;
    if (u >= 0 && u < len) {
      const int e = atomicAdd(&sh.nd, 1);
      sh.dtok[e] = u;
      sh.dpos[e] = tid;
      look_at(u);
    }
  }
  return bad;
}
// occurrences of entry u among the chunk's drafts before position j
__device__ __forceinline__ int32_t drafted_before(const SeenShared &sh, int32_t u, int j) {
  int32_t n = 0;
  for (int d = 0; d < sh.nd; ++d) n += (sh.dtok[d] == u && sh.dpos[d] < j) ? 1 : 0;
  return n;
}

// In place, or rows that cannot be staged: streamed through registers, then the
// listed entries.
template <int DT, int kRowVecs>
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_chunks(const __grid_constant__ AdjustArgs a) {
  extern __shared__ int32_t dyn[];
  __shared__ SeenShared sh;
  __shared__ int32_t mask_of[SVW_MAX_LEN + 1];
  const int tid = threadIdx.x;
  const unsigned item = blockIdx.x / static_cast<unsigned>(a.groups);
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.groups));
  const int32_t i = static_cast<int32_t>(item / static_cast<unsigned>(a.chunks));
  Slices s = slices_of(a, i);  // all under way at once
  const Factors f = factors_of(a, i);
  const Seen seen = seen_at(dyn, a.chunk_len, a.cu_bias != nullptr);
  clear_seen(seen, sh, a.chunk_len);
  if (tid == 0 && (!rows_fine(a, s) || (i == 0 && s.d0 != 0) || (i == a.N - 1 && s.d1 != a.R))) report(a);
  if (!rows_fine(a, s)) return;
  const Rows<DT> r =
      rows_of<DT>(a, s, i, static_cast<int32_t>(item % static_cast<unsigned>(a.chunks)), group, mask_of);
  bool bad = !f.fine() || !lists_fine(a, s);
  if (bad) s.h1 = s.h0, s.b1 = s.b0;
  __syncthreads();
  stream_rows<DT, kRowVecs>(r);
  bad |= count_seen(a, s, seen, sh, r.v0, r.len);
  bad = __syncthreads_or(bad);  // also: every vector is written
  if (bad && tid == 0) report(a);
  spoil_rows(r, bad);
  if (bad) return;
  apply_listed(
      a, r, f, sh.nlist, group,
      [&](int k, int32_t &u, int32_t &w, int32_t &b) {
        u = seen.list[k];
        w = seen.cnt[u];
        b = seen.bidx ? seen.bidx[u] : 0;
      },
      [&](int32_t, int32_t u, int j) { return drafted_before(sh, u, j); });
}

// ---------------------------------------------------------------------------
// two launches: the requests' lists, then the rows
// ---------------------------------------------------------------------------
constexpr int kListThreads = 512;
constexpr int kListWords = 1 << 13;  // of a bitmap: 2^18 tokens of the vocabulary at a time
constexpr int kListCounts = 4096;    // distinct tokens counted at a time (6144: the rows in place, with that much less
                                     // L1 beside them, 110 us instead of 93)
__host__ __device__ constexpr int list_words(int V) {  // a multiple of four
  return V >= kListWords * 32 ? kListWords : ((V + 127) / 128) * 4;
}
__host__ __device__ constexpr int list_bytes(int V, bool bias) {
  return list_words(V) * 8 + kListCounts * 4 * (bias ? 3 : 2);
}

// Request i's distinct tokens, ascending, with their counts and last bias
// places: a bitmap of them in shared memory; a token's rank (the words' running
// counts and the bits below its own) is its place in the list and, less the
// window's start, in the arrays of tokens and counts.  (A hash table of the same
// tokens took 52 us for 8182 of them, 4.5 thousand distinct, in its probes.  With
// the list written from the bitmap's words, not by rank, the benchmark batch in
// place took 97 us where it takes 92.)
__global__ void __launch_bounds__(kListThreads, 2) adjust_lists(const __grid_constant__ AdjustArgs a) {
  extern __shared__ int32_t dyn[];
  const int words = list_words(a.V);
  uint32_t *bits = reinterpret_cast<uint32_t *>(dyn);
  int32_t *below = dyn + words;                                   // tokens in the words before
  int32_t *tok = below + words, *cnt = tok + kListCounts, *bid = cnt + kListCounts;  // by rank
  __shared__ int32_t warp_sum[kListThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int32_t i = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the rows may stream meanwhile
  Slices s = slices_of(a, i);
  if (tid == 0 && (!rows_fine(a, s) || (i == 0 && s.d0 != 0) || (i == a.N - 1 && s.d1 != a.R))) report(a);
  int32_t *offs = a.list_offs + static_cast<int64_t>(i) * (a.list_chunks + 2);
  if (!rows_fine(a, s)) return;  // its rows are not written
  const Factors f = factors_of(a, i);
  bool bad = !lists_fine(a, s);
  if (bad) s.h1 = s.h0, s.b1 = s.b0, s.d1 = s.d0;
  bad |= !f.fine();
  int4 *list = a.list + (static_cast<int64_t>(s.h0) + s.b0 + s.d0);  // room for one entry per token listed
  const int32_t *hist = a.history + s.h0;
  const int32_t hn = s.h1 - s.h0, L = s.d1 - s.d0;
  const uint32_t V = static_cast<uint32_t>(a.V);
  // every token of the history with its place, kAhead of a thread under way; the
  // first kAhead stay in registers
  int32_t held[kAhead];
#pragma unroll
  for (int q = 0; q < kAhead; ++q) held[q] = (tid + q * kListThreads < hn) ? __ldg(hist + tid + q * kListThreads) : -1;
  // and so do the first bias and the draft of a thread: one trip to memory for all lists
  const bool has_bias = s.b0 + tid < s.b1;
  const int32_t bias_held = has_bias ? __ldg(a.bias_tokens + s.b0 + tid) : 0;
  if (has_bias) bad |= !(__ldg(a.bias_values + s.b0 + tid) < INFINITY);
  const int32_t draft = tid < L ? __ldg(a.tokens + s.d0 + tid) : 0;
  auto each = [&](auto &&f) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      if (tid + q * kListThreads < hn) f(held[q], tid + q * kListThreads);
    for (int32_t p0 = tid + kAhead * kListThreads; p0 < hn; p0 += kAhead * kListThreads) {
      int32_t v[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) v[q] = (p0 + q * kListThreads < hn) ? __ldg(hist + p0 + q * kListThreads) : -1;
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (p0 + q * kListThreads < hn) f(v[q], p0 + q * kListThreads);
    }
  };
  // lists that begin before an earlier request's would share their room in the workspace
  for (int32_t j = tid; j < i; j += kListThreads)
    bad |= __ldg(a.cu + j) > s.d0 || (a.cu_history && __ldg(a.cu_history + j) > s.h0) ||
           (a.cu_bias && __ldg(a.cu_bias + j) > s.b0);
  const bool apart = __syncthreads_or(bad) == 0;  // the list may be written
  int32_t base = 0;  // entries of the ranges before
  for (int32_t lo = 0; lo < a.V; lo += words * 32) {
    const int32_t n_tok = min(a.V - lo, words * 32);
    for (int u = tid * 4; u < words; u += kListThreads * 4) *reinterpret_cast<int4 *>(bits + u) = make_int4(0, 0, 0, 0);
    __syncthreads();
    auto mark = [&](int32_t v) {
      bad |= static_cast<uint32_t>(v) >= V;
      const uint32_t u = static_cast<uint32_t>(v) - static_cast<uint32_t>(lo);
      if (u < static_cast<uint32_t>(n_tok)) atomicOr(bits + (u >> 5), 1u << (u & 31));
    };
    each([&](int32_t v, int32_t) { mark(v); });
    if (has_bias) mark(bias_held);
    for (int32_t p = s.b0 + tid + kListThreads; p < s.b1; p += kListThreads) {
      mark(__ldg(a.bias_tokens + p));
      bad |= !(__ldg(a.bias_values + p) < INFINITY);
    }
    if (tid < L) mark(draft);
    __syncthreads();
    // running counts of the words: a thread's stretch, a warp's, the block's
    const int per = (words + kListThreads - 1) / kListThreads, w0 = min(words, tid * per), w1 = min(words, w0 + per);
    int32_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[tid >> 5] = incl;
    __syncthreads();
    int32_t before = incl - mine, total = 0;
    for (int w = 0; w < kListThreads / 32; ++w) {
      before += w < (tid >> 5) ? warp_sum[w] : 0;
      total += warp_sum[w];
    }
    for (int w = w0; w < w1; ++w) {
      below[w] = before;
      const int32_t tok = lo + w * 32;
      if ((tok & ((1 << a.list_shift) - 1)) == 0 && tok < a.V) offs[tok >> a.list_shift] = base + before;
      before += __popc(bits[w]);
    }
    __syncthreads();
    // the counts of kListCounts ranks at a time
    for (int32_t r0 = 0; r0 < total; r0 += kListCounts) {
      const int32_t n = min(total - r0, kListCounts);
      for (int u = tid; u < n; u += kListThreads) {
        cnt[u] = 0;
        if (a.cu_bias) bid[u] = 0;
      }
      __syncthreads();
      // token v's place in the window; -1: outside
      auto place = [&](int32_t v) {
        const uint32_t u = static_cast<uint32_t>(v) - static_cast<uint32_t>(lo);
        if (u >= static_cast<uint32_t>(n_tok)) return -1;
        const int32_t r = below[u >> 5] + __popc(bits[u >> 5] & ((1u << (u & 31)) - 1u)) - r0;
        return (r >= 0 && r < n) ? r : -1;
      };
      each([&](int32_t v, int32_t p) {
        const int e = place(v);
        if (e < 0) return;
        tok[e] = v;
        if (p < s.pl)
          atomicOr(cnt + e, kPromptBit);
        else
          atomicAdd(cnt + e, 1);
      });
      if (has_bias) {
        const int e = place(bias_held);
        if (e >= 0) tok[e] = bias_held, atomicMax(bid + e, s.b0 + tid + 1);
      }
      for (int32_t p = s.b0 + tid + kListThreads; p < s.b1; p += kListThreads) {
        const int32_t v = __ldg(a.bias_tokens + p);
        const int e = place(v);
        if (e >= 0) tok[e] = v, atomicMax(bid + e, p + 1);
      }
      if (tid < L) {
        const int e = place(draft);
        if (e >= 0) tok[e] = draft, atomicOr(cnt + e, kDraftBit);
      }
      __syncthreads();
      for (int r = tid; apart && r < n; r += kListThreads)
        list[base + r0 + r] = make_int4(tok[r], cnt[r], a.cu_bias ? bid[r] : 0, 0);
      __syncthreads();
    }
    base += total;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    offs[a.list_chunks] = base;
    offs[a.list_chunks + 1] = bad ? 1 : 0;
    if (bad) report(a);
  }
}

// a CTA's part of its request's list, once it is complete: its chunk's, or (even) an equal share
struct Listed {
  const int4 *list;
  int n;
  bool bad;
};
__device__ __forceinline__ void wait_for_lists() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ Listed listed_of(const AdjustArgs &a, const Slices &s, int32_t i, int32_t c) {
  wait_for_lists();
  const int32_t *offs = a.list_offs + static_cast<int64_t>(i) * (a.list_chunks + 2);
  int32_t first, last;
  if (a.even) {
    const int64_t all = __ldcg(offs + a.list_chunks);
    first = static_cast<int32_t>(all * c / a.chunks);
    last = static_cast<int32_t>(all * (c + 1) / a.chunks);
  } else {
    const int32_t of = a.chunk_len >> a.list_shift;  // the lists' chunks in one of the CTAs'
    first = __ldcg(offs + c * of);
    last = __ldcg(offs + min((c + 1) * of, a.list_chunks));
  }
  Listed l;
  l.n = last - first;
  l.bad = __ldcg(offs + a.list_chunks + 1) != 0;
  l.list = a.list + (static_cast<int64_t>(s.h0) + s.b0 + s.d0 + first);
  return l;
}
// occurrences of token v among the request's drafts before position j
__device__ __forceinline__ int32_t drafted_before(const int32_t *drafts, int32_t w, int32_t v, int j) {
  int32_t m = 0;
  if (w & kDraftBit)
    for (int d = 0; d < j; ++d) m += (drafts[d] == v) ? 1 : 0;
  return m;
}

// Out of place: a row's chunk is copied to shared memory (bulk copies, the next
// rows' under way), masked and adjusted there, and copied out: the stream's
// bytes pass no register, and a listed entry costs no second trip to memory.
// Everything that a row's turn needs is in shared memory by then: the mask's
// words of the next row are fetched in the turn before, the list's first
// kListed entries and their biases at the start.
constexpr int kStages = 3;
constexpr int kListed = 256;
__host__ __device__ constexpr int stage_bytes(int es) { return list_chunk(es) * es + 16; }
__device__ __forceinline__ void bulk_s2g(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kAdjThreads, 7) adjust_staged(const __grid_constant__ AdjustArgs a) {
  using B = Bits<DT>;
  using T = typename B::T;
  constexpr int EPV = 16 / sizeof(T), kStage = stage_bytes(sizeof(T)), kWords = list_chunk(sizeof(T)) / 32;
  constexpr uint32_t kAll = (1u << EPV) - 1u;
  extern __shared__ __align__(16) unsigned char stages[];
  __shared__ int32_t drafts[SVW_MAX_LEN], mask_of[SVW_MAX_LEN + 1];
  __shared__ int4 held[kListed];
  __shared__ unsigned long long full[kStages];
  __shared__ uint32_t mask_word[2][kWords + 1];  // of this row and the next; one more for the last vector's reach
  const int tid = threadIdx.x;
  const unsigned item = blockIdx.x / static_cast<unsigned>(a.groups);
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.groups));
  const int32_t i = static_cast<int32_t>(item / static_cast<unsigned>(a.chunks));
  const int32_t c = static_cast<int32_t>(item % static_cast<unsigned>(a.chunks));
  const Slices s = slices_of(a, i);
  const Factors f = factors_of(a, i);
  if (!rows_fine(a, s)) return wait_for_lists();  // no CTA is done before the lists are
  const Rows<DT> r = rows_of<DT>(a, s, i, c, group, mask_of);
  if (tid < s.d1 - s.d0) drafts[tid] = __ldg(a.tokens + s.d0 + tid);
  // entry u of row q lies in the stage as far from a 16-byte boundary as in memory
  auto at = [&](int q) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r.in + q * r.in_step)) & 15u;
    return reinterpret_cast<T *>(stages + (q % kStages) * kStage + off);
  };
  auto interior = [&](int q, int &head) {  // bytes between the row's first and last boundary
    head = r.head(q);
    return static_cast<uint32_t>((r.len - head) / EPV * 16);
  };
  auto fetch = [&](int q) {  // by thread 0
    if (a.fault == 1 && blockIdx.x == 0) return;  // test-only
    int head;
    const uint32_t bytes = interior(q, head);
    mbar_arrive_expect_tx(&full[q % kStages], bytes);
    if (bytes) bulk_g2s(at(q) + head, r.in + q * r.in_step + head, bytes, &full[q % kStages]);
  };
  if (tid == 0) {
    for (int q = 0; q < kStages; ++q) mbar_init(&full[q], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int q = 0; q < min(kStages, r.rows); ++q) fetch(q);
  }
  if (tid < 2) mask_word[tid][kWords] = 0;
  __syncthreads();
  // word tid of the chunk in row q's mask
  const int words = (r.len + 31) / 32;
  auto mask_at = [&](int q) {
    return (q < r.rows && mask_of[q] >= 0 && tid < words) ? __ldg(r.words(mask_of[q]) + (r.v0 >> 5) + tid) : 0u;
  };
  if (tid < kWords) mask_word[0][tid] = mask_at(0);
  const Listed ls = listed_of(a, s, i, c);
  // an entry with its bias's value in the place of its place, and whether there is one
  auto entry = [&](int k) {
    int4 e = __ldcg(ls.list + k);
    e.w = e.z;
    if (e.z != 0) e.z = __float_as_int(__ldg(a.bias_values + e.z - 1));
    return e;
  };
  if (!ls.bad && tid < min(ls.n, kListed)) held[tid] = entry(tid);
  __syncthreads();
  int fetched = min(kStages, r.rows);  // rows
  bool ok = true;
  for (int q = 0; q < r.rows; ++q) {
    T *row = at(q);
    int head;
    const int bytes = static_cast<int>(interior(q, head));
    const int tail = head + bytes / static_cast<int>(sizeof(T)), edge = head + r.len - tail;
    const int32_t m = mask_of[q];
    const bool spoilt = ls.bad || m == -2;
    // the entry beyond the boundaries that this thread looks after
    const int mine = (tid < edge) ? (tid < head ? tid : tail + tid - head) : -1;
    if (mine >= 0) row[mine] = r.in[q * r.in_step + mine];
    const uint32_t next_word = mask_at(q + 1);
    const uint32_t *word = mask_word[q & 1];
    auto allowed = [&](int u) { return m < 0 || ((word[u >> 5] >> (u & 31)) & 1u); };
    ok = mbar_wait_bounded(&full[q % kStages], static_cast<uint32_t>((q / kStages) & 1));
    if (m >= 0 || spoilt) {
      if (mine >= 0) {
        if (spoilt)
          row[mine] = static_cast<T>(B::kNaN);
        else if (!allowed(mine))
          row[mine] = static_cast<T>(B::kNegInf);
      }
      for (int k = tid; k < bytes / 16; k += kAdjThreads) {
        uint4 *x = reinterpret_cast<uint4 *>(row + head) + k;
        const int u = head + k * EPV;
        if (spoilt) {
          const uint32_t w = (sizeof(T) == 2) ? B::kNaN * 0x10001u : B::kNaN;
          *x = make_uint4(w, w, w, w);
          continue;
        }
        const uint32_t allow = __funnelshift_r(word[u >> 5], word[(u >> 5) + 1], static_cast<uint32_t>(u & 31)) & kAll;
        if (allow == kAll) continue;
        uint4 y = *x;
        y.x = B::hide(y.x, allow, 0);
        y.y = B::hide(y.y, allow, 1);
        y.z = B::hide(y.z, allow, 2);
        y.w = B::hide(y.w, allow, 3);
        *x = y;
      }
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok) break;  // all threads: a stage whose copy is late is not filled again
    if (!spoilt) {
      for (int k = tid; k < ls.n; k += kAdjThreads) {
        const int4 e = k < kListed ? held[k] : entry(k);
        const int32_t u = e.x - r.v0;
        if (!allowed(u)) continue;
        const int32_t n = (e.y & ~(kPromptBit | kDraftBit)) + drafted_before(drafts, e.y, e.x, group + q * a.groups);
        float y = B::value(row[u]);
        if (adjust_entry(f, n, n > 0 || (e.y & kPromptBit) != 0, e.w != 0, __int_as_float(e.z), y))
          row[u] = static_cast<T>(B::bits(y));
      }
    }
    if (tid < kWords) mask_word[(q + 1) & 1][tid] = next_word;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (mine >= 0) r.out[q * r.out_step + mine] = row[mine];
    if (tid == 0) {
      if (bytes) bulk_s2g(r.out + q * r.out_step + head, row + head, static_cast<uint32_t>(bytes));
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      // the stage of the row before is free once its copy has read it
      if (q >= 1 && q - 1 + kStages < r.rows) {
        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        fetch(q - 1 + kStages);
        fetched = q + kStages;
      }
    }
  }
  if (tid == 0) {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (!ok) {  // a wait gave up: what is in flight lands before the CTA goes
      if (a.status) atomicOr(a.status, SVW_DEV_TIMEOUT);
      for (int q = max(0, fetched - kStages); q < fetched; ++q)
        mbar_wait_bounded(&full[q % kStages], static_cast<uint32_t>((q / kStages) & 1));
    }
  }
}

// In place (only what changes is written), or rows that do not lie alike: through registers.
template <int DT, int kRowVecs>
__global__ void __launch_bounds__(kAdjThreads, 4) adjust_rows(const __grid_constant__ AdjustArgs a) {
  __shared__ int32_t drafts[SVW_MAX_LEN], mask_of[SVW_MAX_LEN + 1];
  const int tid = threadIdx.x;
  const unsigned item = blockIdx.x / static_cast<unsigned>(a.groups);
  const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.groups));
  const int32_t i = static_cast<int32_t>(item / static_cast<unsigned>(a.chunks));
  const int32_t c = static_cast<int32_t>(item % static_cast<unsigned>(a.chunks));
  const Slices s = slices_of(a, i);
  const Factors f = factors_of(a, i);
  if (!rows_fine(a, s)) return wait_for_lists();  // no CTA is done before the lists are
  const Rows<DT> r = rows_of<DT>(a, s, i, a.even ? 0 : c, group, mask_of);
  if (tid < s.d1 - s.d0) drafts[tid] = __ldg(a.tokens + s.d0 + tid);
  __syncthreads();
  stream_rows<DT, kRowVecs>(r);
  const Listed ls = listed_of(a, s, i, c);
  __syncthreads();  // every vector is written
  if (!a.even || c == 0) spoil_rows(r, ls.bad);
  if (ls.bad) return;
  apply_listed(
      a, r, f, ls.n, group,
      [&](int k, int32_t &u, int32_t &w, int32_t &b) {
        const int4 e = __ldcg(ls.list + k);
        u = e.x - r.v0;
        w = e.y;
        b = e.z;
      },
      [&](int32_t w, int32_t u, int j) { return drafted_before(drafts, w, r.v0 + u, j); });
}

template <int DT>
void *chunks_kernel(int row_vecs) {
  switch (row_vecs) {
    case 0: return reinterpret_cast<void *>(adjust_chunks<DT, 0>);
    case 1: return reinterpret_cast<void *>(adjust_chunks<DT, 1>);
    case 2: return reinterpret_cast<void *>(adjust_chunks<DT, 2>);
    default: return reinterpret_cast<void *>(adjust_chunks<DT, 4>);
  }
}
template <int DT>
void *rows_kernel(int row_vecs) {  // full chunks
  return row_vecs == 0 ? reinterpret_cast<void *>(adjust_rows<DT, 0>)
                       : reinterpret_cast<void *>(adjust_rows<DT, kChunk * (DT == 1 ? 2 : 4) / 16 / kAdjThreads>);
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

constexpr int64_t kFew = 152;         // CTAs: one per SM
constexpr int64_t kShortList = 4096;  // tokens of a request's lists, on average, that its chunks count themselves
constexpr int64_t kSmall = 15;        // rows' chunks per SM of a small batch, if lists are short

// Whether the lists are worth a launch of their own: a chunk that counts for
// itself reads all its request's tokens, and its rows pass through registers.
// Rows' chunks per SM times (1 + tokens / 2048) is where the two are even on the
// GPU (us, chunks against lists; bf16, drawn tokens, masks):
//   16 requests of 4 rows of 134840, 14 per SM: 127 tokens 11.4 / 14.9, 1023 14.2 / 16.7, 3999 19.4 / 18.8;
//   40 of 1 of 52776, 3.4: 3999 tokens 12.2 / 14.7, 8191 17.8 / 18.3;
//   200 of 4 of 5169, 11: 127 tokens 12.7 / 15.2, 1023 19.7 / 18.8;  of 52776, 68: 127 tokens 51 / 40;
// the host is 10 us sooner done with one launch.
bool by_lists(int64_t N, int64_t V, int64_t rows, int64_t listed) {
  const int64_t chunks = (V + kChunk - 1) / kChunk, each = listed / N;
  return each > kShortList || rows * chunks * (2048 + each) > kSmall * kFew * 2048;
}

// CTAs of a request's rows, so that there are about `want` in all
int32_t row_groups(const AdjustArgs &a, int64_t want) {
  const int64_t rows = a.R / a.N + (a.bonus ? 1 : 0);  // of a request, on average
  return static_cast<int32_t>(std::max<int64_t>(1, std::min(want / (a.N * static_cast<int64_t>(a.chunks)), rows)));
}

// dynamic shared memory beyond the default, once per device
cudaError_t allow_shared() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(adjust_lists, cudaFuncAttributeMaxDynamicSharedMemorySize, list_bytes(1 << 20, true));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_staged<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * stage_bytes(2));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(adjust_staged<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * stage_bytes(4));
  done[dev] = e == cudaSuccess;
  return e;
}

}  // namespace

// offsets of each request's chunks, its end and whether it is bad | entries
size_t adjust_workspace(int64_t N, int64_t V, int64_t R, int64_t total_history, int64_t total_bias) {
  const int64_t listed = R + total_history + total_bias;
  if (!by_lists(N, V, R + N, listed)) return 0;
  return round256(static_cast<size_t>(N) * ((V + list_chunk(4) - 1) / list_chunk(4) + 2) * 4) + round256(static_cast<size_t>(listed) * sizeof(int4));
}

cudaError_t launch_adjust(const AdjustArgs &args, int dtype, cudaStream_t st) {
  AdjustArgs a = args;
  const int es = dtype == SVW_BF16 ? 2 : 4;
  const uintptr_t apart = reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out);
  const bool vec = (apart & 15u) == 0 && ((a.in_stride - a.out_stride) * es) % 16 == 0;
  const bool lists = a.ws && by_lists(a.N, a.V, a.R + a.N, a.R + a.total_history + a.total_bias);
  const bool staged = lists && vec && a.out != a.logits;
  a.chunk_len = staged ? list_chunk(es) : kChunk;
  a.list_shift = list_shift(es);
  a.list_chunks = static_cast<int32_t>((a.V + list_chunk(es) - 1) / list_chunk(es));
  // in place without a mask there is nothing to stream: the CTAs share out the lists evenly
  a.even = lists && a.out == a.logits && !a.mask;
  // smaller chunks where the batch would leave SMs without work
  while (!lists && a.chunk_len > 1024 && a.N * ((a.V + a.chunk_len - 1) / static_cast<int64_t>(a.chunk_len)) < 2 * kFew)
    a.chunk_len /= 2;
  a.chunks = (a.V + a.chunk_len - 1) / a.chunk_len;
  if (a.even) {
    a.chunk_len = a.V;
    a.chunks = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(a.chunks, 32 * kFew / a.N)));
  }
  // a small batch: as many CTAs as the SMs hold at once (40 requests of 16 rows of 5169 entries: two
  // per SM 20.3 us, four 14.4, eight 16.0)
  a.groups = row_groups(a, lists ? 8 * kFew : 4 * kFew);
  const int64_t grid = static_cast<int64_t>(a.N) * a.chunks * a.groups;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kAdjThreads);
  cfg.stream = st;
  void *argv[] = {&a};
  void *kernel = nullptr;
  if (lists) {
    a.list_offs = static_cast<int32_t *>(a.ws);
    a.list = reinterpret_cast<int4 *>(static_cast<char *>(a.ws) + round256(static_cast<size_t>(a.N) * (a.list_chunks + 2) * 4));
    cudaError_t e = allow_shared();
    if (e != cudaSuccess) return e;
    void *tm = timer_before("adjust_lists", st);
    adjust_lists<<<static_cast<unsigned>(a.N), kListThreads, list_bytes(a.V, a.cu_bias != nullptr), st>>>(a);
    timer_after(tm, st);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (staged) {
      cfg.dynamicSmemBytes = static_cast<size_t>(kStages) * stage_bytes(es);
      kernel = dtype == SVW_BF16 ? reinterpret_cast<void *>(adjust_staged<1>) : reinterpret_cast<void *>(adjust_staged<0>);
    } else {
      kernel = dtype == SVW_BF16 ? rows_kernel<1>(vec) : rows_kernel<0>(vec);
    }
  } else {
    const int row_vecs = vec ? (a.chunk_len * es / 16 + kAdjThreads - 1) / kAdjThreads : 0;  // 0, 1, 2 or 4
    cfg.dynamicSmemBytes = static_cast<size_t>(seen_bytes(a.chunk_len, a.cu_bias != nullptr));
    kernel = dtype == SVW_BF16 ? chunks_kernel<1>(row_vecs) : chunks_kernel<0>(row_vecs);
  }
  void *tm = timer_before("logits_adjust", st);
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, argv);
  timer_after(tm, st);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace svw
