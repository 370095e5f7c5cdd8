// steps_internal.h -- host-side declarations of the steps around a verification
// (logits_adjust, kv_append, paged_attention).  Not part of the public interface.
#pragma once

#include "svw_internal.h"

namespace svw {

// logits_adjust (adjust.cu)
struct AdjustArgs {
  const void *logits;
  void *out;
  int64_t in_stride, out_stride;  // row pitches in elements
  int32_t V, N;
  const int32_t *cu;
  int64_t R;
  int32_t bonus;  // 1: verify layout (a bonus row per request)
  const int32_t *tokens;
  const int32_t *history, *cu_history;
  int64_t total_history;
  const int32_t *prompt_len;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_tokens;
  const float *bias_values;
  const int32_t *cu_bias;
  int64_t total_bias;
  const uint32_t *mask;
  int64_t mask_rows, mask_words;
  const int32_t *mask_row;
  int32_t *status;
  int32_t fault;  // test-only (svw_set_fault): 1 = CTA 0 of adjust_staged copies nothing in
  void *ws;       // NULL: the chunks' CTAs count for themselves
  // set by the launcher
  int32_t chunk_len, chunks, groups;  // entries of a CTA's chunk; CTAs of a request's vocabulary, of its rows
  int32_t list_chunks, list_shift, even;  // chunks of the lists, of 2^shift entries; 1: CTAs of a request's vocabulary share its list evenly
  int32_t *list_offs;  // [N][list_chunks + 2] a request's chunks in its list, its end, whether it is bad
  int4 *list;          // token, count word, bias place
};
size_t adjust_workspace(int64_t N, int64_t V, int64_t R, int64_t total_history, int64_t total_bias);
cudaError_t launch_adjust(const AdjustArgs &a, int dtype, cudaStream_t stream);

// kv_append (append.cu)
struct AppendArgs {
  const void *k, *v, *q;
  void *q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs;  // token and head strides in elements
  int32_t Hq, Hkv, D;
  int32_t N;
  const int32_t *cu;
  int64_t T;
  const int32_t *kv_len, *positions;
  const float *cos_sin;
  int64_t max_pos;
  int32_t rot, interleaved;
  void *k_cache, *v_cache;
  int64_t kc[3], vc[3];  // page, head, row strides in elements
  const int32_t *table;
  int64_t table_stride;
  int32_t max_pages, n_pages, page_size;
  int32_t *status;
};
cudaError_t launch_append(const AppendArgs &a, int dtype, cudaStream_t stream);

// paged_attention (attention.cu)
// the unit that a worker's last segment begins and does not finish
struct alignas(16) AttendJoint {
  int32_t last;  // the worker that finishes the unit; -1: there is no such unit
  int32_t tok0, ntok0, ntok1, hk, pad[3];
};
struct AttendArgs {
  const void *q;
  int64_t q_ts, q_hs;
  int32_t Hq, Hkv, D;
  int32_t N;
  const int32_t *cu;
  int64_t T;
  const int32_t *kv_len;
  const void *k_cache, *v_cache;
  int64_t kc[3], vc[3];
  const int32_t *table;
  int64_t table_stride;
  int32_t max_pages, n_pages, page_size;
  float scale;
  int32_t causal, window;
  void *out;
  float *lse;
  int32_t *status;
  void *ws;
  int32_t tag;    // this call's, never 0
  int32_t fault;  // test-only (svw_set_fault): 1 = every second worker's values are not loaded, and a warp of the others leaves early
  // set by the launcher
  int32_t tile_tokens;  // tokens of a row tile
  int32_t part_rows;    // rows of a workspace part
  AttendJoint *joints;  // [workers]
  unsigned long long *marks;  // [2 workers] parts that are written, by the call's tag
  float2 *part_ml;      // [2 workers][part_rows] reference and sum
  float *part_o;        // [2 workers][part_rows][D] unnormalised output
};
size_t attention_workspace(int64_t T, int32_t G, int32_t D);  // G: query heads of a key head
cudaError_t launch_attention(const AttendArgs &a, cudaStream_t stream);

}  // namespace svw
