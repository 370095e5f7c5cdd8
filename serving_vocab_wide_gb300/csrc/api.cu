// api.cu -- the exported C ABI (see include/svw.h): host-side validation,
// workspace carving, and dispatch to the kernel launchers.  No allocation,
// no host synchronisation, no device-memory reads from the host.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <cuda_runtime.h>

#include "steps_internal.h"

namespace svw {
bool opd_supported(int64_t V, int esize);
}

namespace {

constexpr int64_t kMaxV = 1 << 20;  // sampler span cap (256 threads x 512 groups x 8)
constexpr int64_t kMaxHeadPositions = 1 << 20;  // length head: N k (32-bit offsets into its partials)

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int esize_of(svw_dtype d) { return d == SVW_E4M3 ? 1 : d == SVW_BF16 ? 2 : 4; }

}  // namespace

// one-shot kernel timer, per host thread (svw_time_next_launch)
namespace {
struct ArmedTimer {
  char kernel[64];
  cudaEvent_t begin;
  cudaEvent_t end;
  bool armed;
};
thread_local ArmedTimer g_timer = {};
}  // namespace

namespace svw {
void *timer_before(const char *kernel, cudaStream_t st) {
  if (!g_timer.armed || std::strncmp(kernel, g_timer.kernel, sizeof(g_timer.kernel)) != 0) return nullptr;
  g_timer.armed = false;
  if (cudaEventRecord(g_timer.begin, st) != cudaSuccess) return nullptr;
  return reinterpret_cast<void *>(g_timer.end);
}
void timer_after(void *end_event, cudaStream_t st) {
  if (end_event) cudaEventRecord(reinterpret_cast<cudaEvent_t>(end_event), st);
}

// test hooks: the wait deadline of every translation unit, and an injected fault
namespace {
constexpr int kMaxWaitSetters = 32;
std::mutex g_wait_mu;
cudaError_t (*g_wait_set[kMaxWaitSetters])(long long);
int g_nwait = 0;
std::atomic<int32_t> g_fault{0};
}  // namespace
cudaError_t register_wait_limit(cudaError_t (*set)(long long)) {
  std::lock_guard<std::mutex> lk(g_wait_mu);
  if (g_nwait < kMaxWaitSetters) g_wait_set[g_nwait++] = set;
  return cudaSuccess;
}
int32_t test_fault() { return g_fault.load(std::memory_order_relaxed); }
}  // namespace svw

// a new tag for every OPD and attention call (never 0): flags set by an earlier
// call never match it
static int32_t next_epoch() {
  static std::atomic<uint32_t> g_epoch{0x3c5a0000u};
  uint32_t ep = ++g_epoch;
  if (ep == 0) ep = ++g_epoch;
  return static_cast<int32_t>(ep);
}

extern "C" {

int32_t svw_version(void) { return 100; }

svw_status svw_set_wait_limit(int64_t cycles) {
  if (cycles <= 0) return SVW_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lk(svw::g_wait_mu);
  for (int q = 0; q < svw::g_nwait; ++q)
    if (svw::g_wait_set[q](static_cast<long long>(cycles)) != cudaSuccess) return SVW_ERR_CUDA;
  return SVW_OK;
}

svw_status svw_set_fault(int32_t kind) {
  if (kind < 0 || kind > 1) return SVW_ERR_INVALID_ARG;
  svw::g_fault.store(kind, std::memory_order_relaxed);
  return SVW_OK;
}

const char *svw_status_string(svw_status s) {
  switch (s) {
    case SVW_OK: return "SVW_OK";
    case SVW_ERR_INVALID_ARG: return "SVW_ERR_INVALID_ARG: invalid argument";
    case SVW_ERR_UNSUPPORTED: return "SVW_ERR_UNSUPPORTED: dtype or size not supported";
    case SVW_ERR_MISALIGNED: return "SVW_ERR_MISALIGNED: pointer alignment";
    case SVW_ERR_WORKSPACE: return "SVW_ERR_WORKSPACE: workspace missing or too small";
    case SVW_ERR_CUDA: return "SVW_ERR_CUDA: CUDA runtime or launch failure";
    case SVW_ERR_BAD_INPUT: return "SVW_ERR_BAD_INPUT: the device found an invalid or non-finite request / row";
    case SVW_ERR_TIMEOUT: return "SVW_ERR_TIMEOUT: a bounded wait inside a kernel gave up";
  }
  return "unknown svw_status";
}

svw_status svw_device_status(int32_t status_word) {
  if (status_word & SVW_DEV_TIMEOUT) return SVW_ERR_TIMEOUT;
  if (status_word & SVW_DEV_BAD_INPUT) return SVW_ERR_BAD_INPUT;
  return SVW_OK;
}

size_t svw_verify_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                 svw_dtype dtype) {
  if (n_requests <= 0 || total_draft_rows < 0 || V <= 0 || V > kMaxV) return 0;
  if (dtype != SVW_F32 && dtype != SVW_BF16) return 0;
  return svw::verify_layout(n_requests, total_draft_rows, V, esize_of(dtype)).total;
}

}  // extern "C"

// spec_verify and spec_verify_early: same validation, same results.  With
// check_only, every check that does not involve the workspace runs and the
// call returns SVW_OK without launching (spec_verify_noalloc's first step).
static svw_status verify_entry(bool early, const void *target_logits, const void *draft_logits, svw_dtype dtype,
                               int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                               int32_t max_len, const int32_t *draft_tokens, float temperature, uint64_t seed,
                               int32_t *accept_len, int32_t *next_token, int32_t *status,
                               unsigned long long *bytes_read, void *workspace, size_t workspace_bytes,
                               void *stream, bool check_only = false) {
  if (dtype != SVW_F32 && dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (V <= 0 || N <= 0 || total_draft_rows < 0 || max_len < 1) return SVW_ERR_INVALID_ARG;
  if (max_len > SVW_MAX_LEN || V > kMaxV) return SVW_ERR_UNSUPPORTED;
  const bool have_ws = check_only || workspace;
  if (!target_logits || !draft_logits || !cu_draft || !draft_tokens || !accept_len || !next_token || !have_ws)
    return have_ws ? SVW_ERR_INVALID_ARG : SVW_ERR_WORKSPACE;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return SVW_ERR_INVALID_ARG;
  const double kd = (temperature > 0.f) ? 1.4426950408889634 / static_cast<double>(temperature) : 0.0;
  if (temperature > 0.f && !(kd < 3.0e38)) return SVW_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(cu_draft, 4) ||
      !aligned(draft_tokens, 4) || !aligned(accept_len, 4) || !aligned(next_token, 4) ||
      (status && !aligned(status, 4)) || (bytes_read && !aligned(bytes_read, 8)) ||
      (!check_only && !aligned(workspace, 256)))
    return SVW_ERR_MISALIGNED;
  if (early && total_draft_rows + N >= (int64_t{1} << 31)) return SVW_ERR_UNSUPPORTED;  // int32 row records
  if (check_only) return SVW_OK;
  const svw::VerifyLayout lay = svw::verify_layout(N, total_draft_rows, V, es);
  const svw::EarlyLayout elay = svw::early_layout(N, total_draft_rows, V, es);
  if (workspace_bytes < (early ? elay.total : lay.total)) return SVW_ERR_WORKSPACE;

  const svw::ChunkPlan plan = svw::plan_chunks(V, es);
  const bool greedy = (temperature == 0.f);
  const bool vec = ((static_cast<int64_t>(V) * es) % 16 == 0) && aligned(target_logits, 16) &&
                   aligned(draft_logits, 16);
  svw::VerifyArgs a{};
  a.fault = svw::test_fault();
  a.target = target_logits;
  a.draft = draft_logits;
  a.V = V;
  a.N = N;
  a.cu = cu_draft;
  a.total_rows = total_draft_rows;
  a.rows_t = total_draft_rows + N;
  a.max_len = max_len;
  a.tokens = draft_tokens;
  a.k = static_cast<float>(kd);
  a.seed = seed;
  a.accept_len = accept_len;
  a.next_token = next_token;
  a.status = status;
  char *ws = static_cast<char *>(workspace);
  a.part = reinterpret_cast<svw::Partial *>(ws + lay.part_off);
  a.csr_bad = reinterpret_cast<int32_t *>(ws + lay.csr_bad_off);
  a.stats_grid = 0;  // set by the launcher
  a.C = plan.C;
  a.chunk_len = plan.chunk_len;
  const int64_t rows = greedy ? (total_draft_rows + N) : (2 * total_draft_rows + N);
  a.total_items = rows * plan.C;
  cudaError_t e;
  if (early) {
    a.cnt = reinterpret_cast<int32_t *>(ws + elay.cnt_off);
    a.rej = reinterpret_cast<int32_t *>(ws + elay.rej_off);
    a.badpos = reinterpret_cast<int32_t *>(ws + elay.badpos_off);
    a.stop = reinterpret_cast<int32_t *>(ws + elay.stop_off);
    a.pinfo = reinterpret_cast<int4 *>(ws + elay.pinfo_off);
    a.W = reinterpret_cast<int64_t *>(ws + elay.wave_off);
    a.waveA = reinterpret_cast<int32_t *>(ws + elay.wave_off + (SVW_MAX_LEN + 2) * sizeof(int64_t));
    a.nvalid = a.waveA + (SVW_MAX_LEN + 1);
    a.qnext = a.nvalid + 1;
    a.eres = reinterpret_cast<int4 *>(ws + elay.eres_off);
    a.erow = reinterpret_cast<float4 *>(ws + elay.erow_off);
    a.bytes_read = bytes_read;
    e = svw::launch_verify_early(a, dtype, vec, greedy, static_cast<cudaStream_t>(stream));
  } else {
    e = svw::launch_verify(a, dtype, vec, greedy, static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

namespace svw {
svw_status verify_check_args(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                             int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                             const int32_t *draft_tokens, float temperature, int32_t *accept_len,
                             int32_t *next_token, int32_t *status) {
  return verify_entry(false, target_logits, draft_logits, dtype, V, N, cu_draft, total_draft_rows, max_len,
                      draft_tokens, temperature, 0, accept_len, next_token, status, nullptr, nullptr, 0, nullptr,
                      true);
}
}  // namespace svw

extern "C" {

svw_status spec_verify(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                       int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                       int32_t max_len, const int32_t *draft_tokens, float temperature,
                       uint64_t seed, int32_t *accept_len, int32_t *next_token, int32_t *status,
                       void *workspace, size_t workspace_bytes, void *stream) {
  return verify_entry(false, target_logits, draft_logits, dtype, V, N, cu_draft, total_draft_rows, max_len,
                      draft_tokens, temperature, seed, accept_len, next_token, status, nullptr, workspace,
                      workspace_bytes, stream);
}

size_t svw_verify_early_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                       svw_dtype dtype) {
  if (n_requests <= 0 || total_draft_rows < 0 || V <= 0 || V > kMaxV) return 0;
  if (dtype != SVW_F32 && dtype != SVW_BF16) return 0;
  return svw::early_layout(n_requests, total_draft_rows, V, esize_of(dtype)).total;
}

static_assert(svw::kFilterMaxK == SVW_FILTER_MAX_K, "one top-k limit");

static size_t filtered_lists_bytes(int32_t N, int64_t R) {
  const size_t rows = static_cast<size_t>(2 * R + N);
  return (rows * 4 + 255) / 256 * 256 + 2 * ((rows * svw::kFilterMaxK * 4 + 255) / 256 * 256);
}

size_t svw_verify_filtered_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V,
                                          svw_dtype dtype) {
  const size_t v = svw_verify_workspace_size(n_requests, total_draft_rows, V, dtype);
  if (v == 0) return 0;
  const size_t f = filtered_lists_bytes(n_requests, total_draft_rows);
  return v > f ? v : f;
}

svw_status spec_verify_filtered(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                                int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                                const int32_t *draft_tokens, float temperature, int32_t top_k, float top_p,
                                uint64_t seed, int32_t *accept_len, int32_t *next_token, int32_t *status,
                                void *workspace, size_t workspace_bytes, void *stream) {
  if (dtype != SVW_F32 && dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (V <= 0 || N <= 0 || total_draft_rows < 0 || max_len < 1) return SVW_ERR_INVALID_ARG;
  if (max_len > SVW_MAX_LEN || V > kMaxV) return SVW_ERR_UNSUPPORTED;
  if (!(top_p > 0.f && top_p <= 1.f)) return SVW_ERR_INVALID_ARG;
  if (top_k < 1) return SVW_ERR_INVALID_ARG;
  if (top_k > SVW_FILTER_MAX_K) return SVW_ERR_UNSUPPORTED;
  if (!target_logits || !draft_logits || !cu_draft || !draft_tokens || !accept_len || !next_token ||
      !workspace)
    return workspace ? SVW_ERR_INVALID_ARG : SVW_ERR_WORKSPACE;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return SVW_ERR_INVALID_ARG;
  if (temperature == 0.f)
    // filtering keeps the argmax: greedy verification is unchanged
    return spec_verify(target_logits, draft_logits, dtype, V, N, cu_draft, total_draft_rows, max_len, draft_tokens,
                       0.f, seed, accept_len, next_token, status, workspace, workspace_bytes, stream);
  const double kd = 1.4426950408889634 / static_cast<double>(temperature);
  if (!(kd < 3.0e38)) return SVW_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(cu_draft, 4) ||
      !aligned(draft_tokens, 4) || !aligned(accept_len, 4) || !aligned(next_token, 4) ||
      (status && !aligned(status, 4)) || !aligned(workspace, 256))
    return SVW_ERR_MISALIGNED;
  if (workspace_bytes < svw_verify_filtered_workspace_size(N, total_draft_rows, V, dtype)) return SVW_ERR_WORKSPACE;
  if (svw::filter_smem_bytes(V, es, top_k) > 200 * 1024) return SVW_ERR_UNSUPPORTED;
  const size_t rows = static_cast<size_t>(2 * total_draft_rows + N);
  char *ws = static_cast<char *>(workspace);
  svw::FilterArgs a{};
  a.target = target_logits;
  a.draft = draft_logits;
  a.V = V;
  a.N = N;
  a.cu = cu_draft;
  a.R = total_draft_rows;
  a.rows_t = total_draft_rows + N;
  a.max_len = max_len;
  a.tokens = draft_tokens;
  a.k = static_cast<float>(kd);
  a.top_k = top_k;
  a.top_p = top_p;
  a.cand = svw::filter_candidates(top_k);
  a.gs = svw::filter_group(top_k);
  a.seed = seed;
  a.accept_len = accept_len;
  a.next_token = next_token;
  a.status = status;
  a.cnt = reinterpret_cast<int32_t *>(ws);
  const size_t off1 = (rows * 4 + 255) / 256 * 256;
  a.lidx = reinterpret_cast<int32_t *>(ws + off1);
  a.lp = reinterpret_cast<float *>(ws + off1 + (rows * svw::kFilterMaxK * 4 + 255) / 256 * 256);
  const bool vec = ((static_cast<int64_t>(V) * es) % 16 == 0) && aligned(target_logits, 16) &&
                   aligned(draft_logits, 16);
  const cudaError_t e = svw::launch_filtered(a, dtype, vec, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

svw_status spec_verify_early(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                             int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                             const int32_t *draft_tokens, float temperature, uint64_t seed, int32_t *accept_len,
                             int32_t *next_token, int32_t *status, unsigned long long *bytes_read,
                             void *workspace, size_t workspace_bytes, void *stream) {
  return verify_entry(true, target_logits, draft_logits, dtype, V, N, cu_draft, total_draft_rows, max_len,
                      draft_tokens, temperature, seed, accept_len, next_token, status, bytes_read, workspace,
                      workspace_bytes, stream);
}

// OPD workspace: flags int32 [R] | row constants float4 [R], each 256-aligned
static size_t opd_flags_bytes(int64_t R) { return static_cast<size_t>((R * 4 + 255) / 256 * 256); }
static size_t opd_rowc_bytes(int64_t R) { return static_cast<size_t>((R * 16 + 255) / 256 * 256); }

// flags [R] int32 | row constants [R] float4 | clamped-sum partials [R][kOpdFixParts] float2
size_t svw_opd_workspace_size(int64_t total_draft_rows) {
  if (total_draft_rows <= 0 || total_draft_rows > (int64_t{1} << 40)) return 0;
  return opd_flags_bytes(total_draft_rows) + opd_rowc_bytes(total_draft_rows) +
         static_cast<size_t>(total_draft_rows) * svw::kOpdFixParts * sizeof(float2);
}

svw_status opd_loss(const void *target_logits, const void *draft_logits, svw_dtype dtype,
                    int32_t V, int32_t N, const int32_t *cu_draft, int64_t total_draft_rows,
                    int32_t target_has_bonus_row, float temperature, float clip_c,
                    float lambda_ce, float grad_scale, float *loss, float *dlogits,
                    int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  if (dtype != SVW_F32 && dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (V <= 0 || total_draft_rows <= 0) return SVW_ERR_INVALID_ARG;
  if (target_has_bonus_row && (N <= 0 || !cu_draft)) return SVW_ERR_INVALID_ARG;
  if (!target_logits || !draft_logits || !loss) return SVW_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature)) return SVW_ERR_INVALID_ARG;
  if (!(clip_c > 0.f) || !std::isfinite(lambda_ce) || !std::isfinite(grad_scale))
    return SVW_ERR_INVALID_ARG;
  const double kd = 1.4426950408889634 / static_cast<double>(temperature);
  if (!(kd < 3.0e38)) return SVW_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!svw::opd_supported(V, es)) return SVW_ERR_UNSUPPORTED;
  if (!aligned(target_logits, es) || !aligned(draft_logits, es) || !aligned(loss, 4) ||
      (dlogits && !aligned(dlogits, 16)) || (cu_draft && !aligned(cu_draft, 4)) ||
      (status && !aligned(status, 4)) || (workspace && !aligned(workspace, 256)))
    return SVW_ERR_MISALIGNED;
  if (workspace && workspace_bytes < svw_opd_workspace_size(total_draft_rows)) return SVW_ERR_WORKSPACE;
  const bool bulk = ((static_cast<int64_t>(V) * es) % 16 == 0) && aligned(target_logits, 16) &&
                    aligned(draft_logits, 16);
  svw::OpdArgs a;
  a.fault = svw::test_fault();
  a.target = target_logits;
  a.draft = draft_logits;
  a.V = V;
  a.N = target_has_bonus_row ? N : 0;
  a.cu = cu_draft;
  a.R = total_draft_rows;
  a.has_bonus = target_has_bonus_row ? 1 : 0;
  a.k = static_cast<float>(kd);
  a.invT = static_cast<float>(1.0 / static_cast<double>(temperature));
  a.clip_c = clip_c;
  a.lambda_ce = lambda_ce;
  a.grad_scale = grad_scale;
  a.loss = loss;
  a.dlogits = dlogits;
  a.status = status;
  a.flags = static_cast<int32_t *>(workspace);
  a.epoch = next_epoch();
  a.rowc = workspace ? reinterpret_cast<float4 *>(static_cast<char *>(workspace) + opd_flags_bytes(total_draft_rows))
                     : nullptr;
  a.fixp = workspace ? reinterpret_cast<float2 *>(static_cast<char *>(workspace) + opd_flags_bytes(total_draft_rows) +
                                                  opd_rowc_bytes(total_draft_rows))
                     : nullptr;
  a.nbonus = 0;
  a.bpart = nullptr;
  a.csr_bad = nullptr;
  const cudaError_t e = svw::launch_opd(a, dtype, bulk, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

svw_status svw_time_next_launch(const char *kernel, void *begin_event, void *end_event) {
  if (!kernel) {
    g_timer.armed = false;
    return SVW_OK;
  }
  if (!begin_event || !end_event || std::strlen(kernel) >= sizeof(g_timer.kernel)) return SVW_ERR_INVALID_ARG;
  std::strncpy(g_timer.kernel, kernel, sizeof(g_timer.kernel));
  g_timer.begin = reinterpret_cast<cudaEvent_t>(begin_event);
  g_timer.end = reinterpret_cast<cudaEvent_t>(end_event);
  g_timer.armed = true;
  return SVW_OK;
}

size_t svw_verify_opd_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V, svw_dtype dtype) {
  if (n_requests <= 0 || total_draft_rows < 0 || V <= 0 || V > kMaxV) return 0;
  if (dtype != SVW_F32 && dtype != SVW_BF16) return 0;
  return svw::fused_layout(n_requests, total_draft_rows, V).total;
}

size_t svw_workspace_size(int32_t n_requests, int64_t total_draft_rows, int32_t V, int32_t max_len) {
  if (max_len < 1 || max_len > SVW_MAX_LEN) return 0;
  if (n_requests <= 0 || total_draft_rows < 0 || V <= 0 || V > kMaxV) return 0;
  size_t need = 0;
  for (svw_dtype dt : {SVW_F32, SVW_BF16}) {
    need = std::max(need, svw_verify_workspace_size(n_requests, total_draft_rows, V, dt));
    need = std::max(need, svw_verify_early_workspace_size(n_requests, total_draft_rows, V, dt));
    need = std::max(need, svw_verify_filtered_workspace_size(n_requests, total_draft_rows, V, dt));
    need = std::max(need, svw_verify_opd_workspace_size(n_requests, total_draft_rows, V, dt));
  }
  if (total_draft_rows > 0) need = std::max(need, svw_opd_workspace_size(total_draft_rows));
  return need;
}

svw_status spec_verify_opd(const void *target_logits, const void *draft_logits, svw_dtype dtype, int32_t V,
                           int32_t N, const int32_t *cu_draft, int64_t total_draft_rows, int32_t max_len,
                           const int32_t *draft_tokens, float temperature, float opd_temperature, uint64_t seed,
                           float clip_c, float lambda_ce, float grad_scale, int32_t *accept_len,
                           int32_t *next_token, float *loss, float *dlogits, int32_t *status, void *workspace,
                           size_t workspace_bytes, void *stream) {
  if (dtype != SVW_F32 && dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (V <= 0 || N <= 0 || total_draft_rows <= 0 || max_len < 1) return SVW_ERR_INVALID_ARG;
  if (max_len > SVW_MAX_LEN || V > kMaxV) return SVW_ERR_UNSUPPORTED;
  if (!target_logits || !draft_logits || !cu_draft || !draft_tokens || !accept_len || !next_token || !loss ||
      !workspace)
    return workspace ? SVW_ERR_INVALID_ARG : SVW_ERR_WORKSPACE;
  if (!(temperature >= 0.f) || !std::isfinite(temperature)) return SVW_ERR_INVALID_ARG;
  if (!(opd_temperature > 0.f) || !std::isfinite(opd_temperature)) return SVW_ERR_INVALID_ARG;
  if (temperature > 0.f && temperature != opd_temperature) return SVW_ERR_INVALID_ARG;  // shared softmaxes
  if (!(clip_c > 0.f) || !std::isfinite(lambda_ce) || !std::isfinite(grad_scale)) return SVW_ERR_INVALID_ARG;
  const double kd = 1.4426950408889634 / static_cast<double>(opd_temperature);
  if (!(kd < 3.0e38)) return SVW_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!aligned(target_logits, 16) || !aligned(draft_logits, 16) || !aligned(cu_draft, 4) ||
      !aligned(draft_tokens, 4) || !aligned(accept_len, 4) || !aligned(next_token, 4) || !aligned(loss, 4) ||
      (dlogits && !aligned(dlogits, 16)) || (status && !aligned(status, 4)) || !aligned(workspace, 256))
    return SVW_ERR_MISALIGNED;
  // one pass needs the 16-byte-pitched register-resident path
  if ((static_cast<int64_t>(V) * es) % 16 != 0 || !svw::opd_fast_supported(V, es)) return SVW_ERR_UNSUPPORTED;
  const svw::FusedLayout lay = svw::fused_layout(N, total_draft_rows, V);
  if (workspace_bytes < lay.total) return SVW_ERR_WORKSPACE;
  char *ws = static_cast<char *>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool greedy = (temperature == 0.f);

  svw::OpdArgs o;
  o.fault = svw::test_fault();
  o.target = target_logits;
  o.draft = draft_logits;
  o.V = V;
  o.N = N;
  o.cu = cu_draft;
  o.R = total_draft_rows;
  o.has_bonus = 1;
  o.k = static_cast<float>(kd);
  o.invT = static_cast<float>(1.0 / static_cast<double>(opd_temperature));
  o.clip_c = clip_c;
  o.lambda_ce = lambda_ce;
  o.grad_scale = grad_scale;
  o.loss = loss;
  o.dlogits = dlogits;
  o.status = status;
  o.flags = reinterpret_cast<int32_t *>(ws + lay.flags_off);
  o.rowc = reinterpret_cast<float4 *>(ws + lay.rowc_off);
  o.fixp = reinterpret_cast<float2 *>(ws + lay.fixp_off);
  o.epoch = next_epoch();
  o.nbonus = N;
  o.bpart = reinterpret_cast<float4 *>(ws + lay.bpart_off);
  o.csr_bad = reinterpret_cast<int32_t *>(ws + lay.csr_bad_off);
  int grid = 0;
  cudaError_t e = svw::launch_opd_fused_fast(o, dtype, &grid, st);
  if (e != cudaSuccess) return SVW_ERR_CUDA;

  svw::FusedArgs f;
  f.target = target_logits;
  f.draft = draft_logits;
  f.V = V;
  f.N = N;
  f.cu = cu_draft;
  f.total_rows = total_draft_rows;
  f.max_len = max_len;
  f.tokens = draft_tokens;
  f.k = o.k;
  f.seed = seed;
  f.rowc = o.rowc;
  f.bpart = o.bpart;
  f.bparts = svw::opd_cluster_size(V, es);
  f.csr_bad = o.csr_bad;
  f.csr_grid = grid;
  f.accept_len = accept_len;
  f.next_token = next_token;
  f.status = status;
  // the parts grid (tiny) first, so that the gradient fix-up can run beside
  // the finalize kernel's draw
  e = svw::launch_opd_fix(o, dtype, svw::kFixParts, st);
  if (e != cudaSuccess) return SVW_ERR_CUDA;
  e = svw::launch_fused_finalize(f, dtype, greedy, st);
  if (e != cudaSuccess) return SVW_ERR_CUDA;
  e = svw::launch_opd_fix(o, dtype, svw::kFixGradLast, st);  // rows with a clipped term, exactly
  return e == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

size_t svw_length_head_workspace_size(int32_t n_requests, int32_t k, int32_t hidden_out) {
  if (n_requests <= 0 || k <= 0 || k > SVW_MAX_LEN || hidden_out <= 0) return 0;
  if (static_cast<int64_t>(n_requests) * k > kMaxHeadPositions) return 0;
  return svw::length_head_gemm_bytes(n_requests, k, hidden_out);
}

svw_status length_head(const void *hidden, const void *w1, const float *b1, const float *w2, float b2, int32_t N,
                       int32_t k, int32_t H, int32_t hidden_out, float gamma, float *a_hat, int32_t *k_hat,
                       void *workspace, size_t workspace_bytes, void *stream) {
  if (N <= 0 || k <= 0 || H <= 0 || hidden_out <= 0) return SVW_ERR_INVALID_ARG;
  if (k > SVW_MAX_LEN || static_cast<int64_t>(N) * k > kMaxHeadPositions) return SVW_ERR_UNSUPPORTED;
  if (!hidden || !w1 || !b1 || !w2 || !a_hat || !k_hat) return SVW_ERR_INVALID_ARG;
  if (!workspace) return SVW_ERR_WORKSPACE;
  if (!(gamma > 0.f) || !std::isfinite(gamma) || !std::isfinite(b2)) return SVW_ERR_INVALID_ARG;
  if (!aligned(hidden, 16) || !aligned(w1, 16) || !aligned(b1, 4) || !aligned(w2, 4) || !aligned(a_hat, 4) ||
      !aligned(k_hat, 4) || !aligned(workspace, 256))
    return SVW_ERR_MISALIGNED;
  if (H % 8 != 0) return SVW_ERR_UNSUPPORTED;  // 16-byte rows for the GEMM
  if (workspace_bytes < svw_length_head_workspace_size(N, k, hidden_out)) return SVW_ERR_WORKSPACE;
  const int rc = svw::launch_length_head(hidden, w1, b1, w2, b2, N, k, H, hidden_out, gamma, a_hat, k_hat,
                                         workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  return rc == 0 ? SVW_OK : SVW_ERR_CUDA;
}

svw_status length_head_label(const int32_t *accept_len, const int32_t *cu_draft, const float *a_hat, int32_t N,
                             float *a_star, float *loss, void *stream) {
  if (N <= 0 || !accept_len || !cu_draft || !a_star || (loss && !a_hat)) return SVW_ERR_INVALID_ARG;
  if (!aligned(accept_len, 4) || !aligned(cu_draft, 4) || (a_hat && !aligned(a_hat, 4)) || !aligned(a_star, 4) ||
      (loss && !aligned(loss, 4)))
    return SVW_ERR_MISALIGNED;
  const int rc = svw::launch_length_label(accept_len, cu_draft, a_hat, N, a_star, loss,
                                          static_cast<cudaStream_t>(stream));
  return rc == 0 ? SVW_OK : SVW_ERR_CUDA;
}

size_t svw_logits_adjust_workspace_size(int32_t n_requests, int32_t V, int64_t total_draft_rows, int64_t total_history,
                                        int64_t total_bias) {
  if (n_requests <= 0 || V <= 0 || V > kMaxV || total_draft_rows < 0 || total_history < 0 || total_bias < 0 ||
      total_draft_rows > INT32_MAX || total_history > INT32_MAX || total_bias > INT32_MAX)
    return 0;
  return svw::adjust_workspace(n_requests, V, total_draft_rows, total_history, total_bias);
}

svw_status logits_adjust(const void *logits, int64_t logits_stride, svw_dtype dtype, int32_t V, int32_t N,
                         const int32_t *cu_draft, int64_t total_draft_rows, int32_t has_bonus_row,
                         const int32_t *draft_tokens, const int32_t *history, const int32_t *cu_history,
                         int64_t total_history, const int32_t *prompt_len, const float *repetition,
                         const float *frequency, const float *presence, const int32_t *bias_tokens,
                         const float *bias_values, const int32_t *cu_bias, int64_t total_bias,
                         const uint32_t *mask, int64_t mask_rows, const int32_t *mask_row, void *out,
                         int64_t out_stride, int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  if (dtype != SVW_F32 && dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (V <= 0 || N <= 0 || total_draft_rows < 0 || total_history < 0 || total_bias < 0 || mask_rows < 0)
    return SVW_ERR_INVALID_ARG;
  if (V > kMaxV || total_history > INT32_MAX || total_bias >= INT32_MAX || total_draft_rows > INT32_MAX - N ||
      mask_rows > INT32_MAX)
    return SVW_ERR_UNSUPPORTED;
  if (!logits || !out || !cu_draft || (total_draft_rows > 0 && !draft_tokens) ||
      (cu_history && total_history > 0 && !history) || (cu_bias && total_bias > 0 && (!bias_tokens || !bias_values)))
    return SVW_ERR_INVALID_ARG;
  const int64_t rows = total_draft_rows + (has_bonus_row ? N : 0);
  if (logits_stride < V || out_stride < V) return SVW_ERR_INVALID_ARG;
  // a mask row for each row, named or by its own number
  if (mask && !mask_row && mask_rows != rows) return SVW_ERR_INVALID_ARG;
  const int es = esize_of(dtype);
  if (!aligned(logits, es) || !aligned(out, es) || !aligned(cu_draft, 4) || !aligned(draft_tokens, 4) ||
      !aligned(history, 4) || !aligned(cu_history, 4) || !aligned(prompt_len, 4) || !aligned(repetition, 4) ||
      !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_tokens, 4) || !aligned(bias_values, 4) ||
      !aligned(cu_bias, 4) || !aligned(mask, 4) || !aligned(mask_row, 4) || !aligned(status, 4) ||
      !aligned(workspace, 256))
    return SVW_ERR_MISALIGNED;
  if (workspace &&
      workspace_bytes < svw_logits_adjust_workspace_size(N, V, total_draft_rows, total_history, total_bias))
    return SVW_ERR_WORKSPACE;
  if (rows == 0) return SVW_OK;  // no drafts and no bonus rows
  if (rows > INT64_MAX / 8 / std::max(logits_stride, out_stride)) return SVW_ERR_INVALID_ARG;
  // in place, or apart
  const char *i0 = static_cast<const char *>(logits), *o0 = static_cast<const char *>(out);
  const int64_t ib = ((rows - 1) * logits_stride + V) * es, ob = ((rows - 1) * out_stride + V) * es;
  if (i0 == o0 ? logits_stride != out_stride && rows > 1 : (i0 < o0 ? o0 - i0 < ib : i0 - o0 < ob))
    return SVW_ERR_INVALID_ARG;
  svw::AdjustArgs a{};
  a.logits = logits;
  a.out = out;
  a.in_stride = logits_stride;
  a.out_stride = out_stride;
  a.V = V;
  a.N = N;
  a.cu = cu_draft;
  a.R = total_draft_rows;
  a.bonus = has_bonus_row ? 1 : 0;
  a.tokens = draft_tokens;
  a.history = history;
  a.cu_history = cu_history;
  a.total_history = total_history;
  a.prompt_len = prompt_len;
  a.repetition = repetition;
  a.frequency = frequency;
  a.presence = presence;
  a.bias_tokens = bias_tokens;
  a.bias_values = bias_values;
  a.cu_bias = cu_bias;
  a.total_bias = total_bias;
  a.mask = mask;
  a.mask_rows = mask_rows;
  a.mask_words = (static_cast<int64_t>(V) + 31) / 32;
  a.mask_row = mask_row;
  a.status = status;
  a.fault = svw::test_fault();
  a.ws = workspace;
  return svw::launch_adjust(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

// the cache's own fields, checked once for all of its calls
static svw_status check_cache(const svw_paged_kv *c) {
  if (!c || !c->k || !c->v || !c->block_table) return SVW_ERR_INVALID_ARG;
  if (c->n_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 ||
      c->table_stride < c->max_pages)
    return SVW_ERR_INVALID_ARG;
  for (int d = 0; d < 3; ++d)
    if (c->k_stride[d] < 0 || c->v_stride[d] < 0) return SVW_ERR_INVALID_ARG;
  if (!aligned(c->block_table, 4)) return SVW_ERR_MISALIGNED;
  return SVW_OK;
}

// what kv_append and kv_append_norm take alike, checked and in the kernels' form
static svw_status append_args(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                              int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                              int64_t q_head_stride, void *q_out, svw_dtype dtype, int32_t n_q_heads, int32_t N,
                              const int32_t *cu_new, int64_t total_new, const int32_t *kv_len,
                              const int32_t *positions, const float *cos_sin, int64_t max_pos, int32_t rot_dim,
                              int32_t interleaved, const svw_paged_kv *cache, svw_dtype cache_dtype, int32_t *status,
                              svw::AppendArgs &a) {
  if ((dtype != SVW_F32 && dtype != SVW_BF16) || (cache_dtype != dtype && cache_dtype != SVW_E4M3))
    return SVW_ERR_UNSUPPORTED;
  if (N <= 0 || total_new < 0 || n_q_heads < 0) return SVW_ERR_INVALID_ARG;
  const svw_status cs = check_cache(cache);
  if (cs != SVW_OK) return cs;
  const int es = esize_of(dtype), ces = esize_of(cache_dtype);
  if (cache->head_dim > 1024 || total_new > INT32_MAX || n_q_heads > 4096 || cache->n_kv_heads > 4096)
    return SVW_ERR_UNSUPPORTED;
  if (!cu_new || !kv_len || (total_new > 0 && (!k || !v)) || (q == nullptr) != (q_out == nullptr))
    return SVW_ERR_INVALID_ARG;
  if (q && n_q_heads == 0) return SVW_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > cache->head_dim || (rot_dim > 0 && (!cos_sin || max_pos <= 0)))
    return SVW_ERR_INVALID_ARG;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0 || q_token_stride < 0 ||
      q_head_stride < 0)
    return SVW_ERR_INVALID_ARG;
  // the stride of a dimension of one is never used
  if (total_new <= 1) {
    k_token_stride = v_token_stride = 0;
    q_token_stride = static_cast<int64_t>(n_q_heads) * cache->head_dim;
  }
  if (cache->n_kv_heads == 1) k_head_stride = v_head_stride = 0;
  if (n_q_heads == 1) q_head_stride = cache->head_dim;
  // rotated in place only where every element keeps its place
  if (q && q == q_out &&
      (q_head_stride != cache->head_dim || q_token_stride != static_cast<int64_t>(n_q_heads) * cache->head_dim))
    return SVW_ERR_INVALID_ARG;
  if (!aligned(k, es) || !aligned(v, es) || !aligned(q, es) || !aligned(q_out, es) || !aligned(cache->k, ces) ||
      !aligned(cache->v, ces) || !aligned(cu_new, 4) || !aligned(kv_len, 4) || !aligned(positions, 4) ||
      !aligned(cos_sin, 4) || !aligned(status, 4))
    return SVW_ERR_MISALIGNED;
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.k_ts = k_token_stride;
  a.k_hs = k_head_stride;
  a.v_ts = v_token_stride;
  a.v_hs = v_head_stride;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.Hq = q ? n_q_heads : 0;
  a.Hkv = cache->n_kv_heads;
  a.D = cache->head_dim;
  a.N = N;
  a.cu = cu_new;
  a.T = total_new;
  a.kv_len = kv_len;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.max_pos = max_pos;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  for (int d = 0; d < 3; ++d) {
    a.kc[d] = cache->k_stride[d];
    a.vc[d] = cache->v_stride[d];
  }
  a.table = cache->block_table;
  a.table_stride = cache->table_stride;
  a.max_pages = cache->max_pages;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.status = status;
  return SVW_OK;
}

svw_status kv_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                     int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                     int64_t q_head_stride, void *q_out, svw_dtype dtype, int32_t n_q_heads, int32_t N,
                     const int32_t *cu_new, int64_t total_new, const int32_t *kv_len, const int32_t *positions,
                     const float *cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                     const svw_paged_kv *cache, int32_t *status, void *stream) {
  svw::AppendArgs a{};
  const svw_status s = append_args(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, q,
                                   q_token_stride, q_head_stride, q_out, dtype, n_q_heads, N, cu_new, total_new,
                                   kv_len, positions, cos_sin, max_pos, rot_dim, interleaved, cache, dtype, status, a);
  if (s != SVW_OK || total_new == 0) return s;
  return svw::launch_append(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

svw_status kv_append_norm(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                          int64_t q_head_stride, void *q_out, svw_dtype dtype, int32_t n_q_heads, int32_t N,
                          const int32_t *cu_new, int64_t total_new, const int32_t *kv_len, const int32_t *positions,
                          const float *k_weight, const float *q_weight, float eps, const float *cos_sin,
                          int64_t max_pos, int32_t rot_dim, int32_t interleaved, const svw_paged_kv *cache,
                          svw_dtype cache_dtype, const float *k_scale, const float *v_scale, int32_t *status,
                          void *stream) {
  svw::AppendNormArgs a{};
  const svw_status s = append_args(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, q,
                                   q_token_stride, q_head_stride, q_out, dtype, n_q_heads, N, cu_new, total_new,
                                   kv_len, positions, cos_sin, max_pos, rot_dim, interleaved, cache, cache_dtype,
                                   status, a);
  if (s != SVW_OK) return s;
  if (!(eps >= 0.f) || !std::isfinite(eps) || (q_weight && !q)) return SVW_ERR_INVALID_ARG;
  if (cache_dtype != SVW_E4M3 && (k_scale || v_scale)) return SVW_ERR_INVALID_ARG;
  if (!aligned(k_weight, 4) || !aligned(q_weight, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return SVW_ERR_MISALIGNED;
  if (total_new == 0) return SVW_OK;
  a.k_weight = k_weight;
  a.q_weight = q_weight;
  a.eps = eps;
  a.codes = cache_dtype == SVW_E4M3 ? 1 : 0;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return svw::launch_append_norm(a, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

svw_status kv_gather(const svw_paged_kv *cache, svw_dtype cache_dtype, const float *k_scale, const float *v_scale,
                     int32_t N, const int32_t *cu_out, int64_t total_out, const int32_t *first, void *k_out,
                     void *v_out, svw_dtype out_dtype, int32_t *status, void *stream) {
  if ((cache_dtype != SVW_F32 && cache_dtype != SVW_BF16 && cache_dtype != SVW_E4M3) ||
      (out_dtype != SVW_F32 && out_dtype != SVW_BF16))
    return SVW_ERR_UNSUPPORTED;
  if (N <= 0 || total_out < 0) return SVW_ERR_INVALID_ARG;
  const svw_status cs = check_cache(cache);
  if (cs != SVW_OK) return cs;
  if (cache->head_dim > 1024 || total_out > INT32_MAX || cache->n_kv_heads > 4096) return SVW_ERR_UNSUPPORTED;
  if (!cu_out || (total_out > 0 && !k_out && !v_out)) return SVW_ERR_INVALID_ARG;
  if (cache_dtype != SVW_E4M3 && (k_scale || v_scale)) return SVW_ERR_INVALID_ARG;
  const int ces = esize_of(cache_dtype), es = esize_of(out_dtype);
  if (!aligned(cache->k, ces) || !aligned(cache->v, ces) || !aligned(k_out, es) || !aligned(v_out, es) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(cu_out, 4) || !aligned(first, 4) || !aligned(status, 4))
    return SVW_ERR_MISALIGNED;
  if (total_out == 0) return SVW_OK;
  svw::GatherArgs a{};
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  for (int d = 0; d < 3; ++d) {
    a.kc[d] = cache->k_stride[d];
    a.vc[d] = cache->v_stride[d];
  }
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.Hkv = cache->n_kv_heads;
  a.D = cache->head_dim;
  a.N = N;
  a.cu = cu_out;
  a.T = total_out;
  a.first = first;
  a.table = cache->block_table;
  a.table_stride = cache->table_stride;
  a.max_pages = cache->max_pages;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = status;
  return svw::launch_gather(a, cache_dtype, out_dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SVW_OK
                                                                                                          : SVW_ERR_CUDA;
}

size_t svw_paged_attention_workspace_size(int64_t total_new, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim) {
  if (total_new < 0 || n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads != 0 ||
      n_q_heads / n_kv_heads > 64 || (head_dim != 64 && head_dim != 128))
    return 0;
  return svw::attention_workspace(total_new, n_q_heads / n_kv_heads, head_dim);
}

// paged_attention, or with codes paged_attention_fp8
static svw_status attention_entry(bool codes, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                  svw_dtype dtype, int32_t n_q_heads, int32_t N, const int32_t *cu_new,
                                  int64_t total_new, const int32_t *kv_len, const svw_paged_kv *cache,
                                  const float *k_scale, const float *v_scale, float scale, int32_t causal,
                                  int32_t window, void *out, float *lse, int32_t *status, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (dtype != SVW_BF16) return SVW_ERR_UNSUPPORTED;
  if (N <= 0 || total_new < 0 || n_q_heads <= 0) return SVW_ERR_INVALID_ARG;
  const svw_status cs = check_cache(cache);
  if (cs != SVW_OK) return cs;
  const int32_t Hkv = cache->n_kv_heads, D = cache->head_dim, ps = cache->page_size;
  if (n_q_heads % Hkv != 0) return SVW_ERR_INVALID_ARG;
  if (n_q_heads / Hkv > 64 || (D != 64 && D != 128) || ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0 ||
      total_new > INT32_MAX / n_q_heads || static_cast<int64_t>(cache->max_pages) * ps > (int64_t{1} << 30))
    return SVW_ERR_UNSUPPORTED;
  if (!cu_new || !kv_len || (total_new > 0 && (!q || !out))) return SVW_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || (window > 0 && !causal)) return SVW_ERR_INVALID_ARG;
  if (q_token_stride < 0 || q_head_stride < 0) return SVW_ERR_INVALID_ARG;
  // the stride of a dimension of one is never used: any multiple of 16 bytes will do
  svw_paged_kv c = *cache;
  if (total_new <= 1) q_token_stride = D;
  if (n_q_heads == 1) q_head_stride = D;
  if (c.n_pages == 1) c.k_stride[0] = c.v_stride[0] = D;
  if (c.n_kv_heads == 1) c.k_stride[1] = c.v_stride[1] = D;
  int64_t odd = q_token_stride | q_head_stride, odd_cache = 0;
  bool shared = q_token_stride == 0 || q_head_stride == 0;  // a dimension repeated by a stride of zero
  for (int d = 0; d < 3; ++d) {
    odd_cache |= c.k_stride[d] | c.v_stride[d];
    shared |= c.k_stride[d] == 0 || c.v_stride[d] == 0;
  }
  if (shared) return SVW_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(cache->k, 16) || !aligned(cache->v, 16) || (odd & 7) ||
      (odd_cache & (codes ? 15 : 7)) || !aligned(out, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(lse, 4) || !aligned(cu_new, 4) || !aligned(kv_len, 4) || !aligned(status, 4) ||
      !aligned(workspace, 256))
    return SVW_ERR_MISALIGNED;
  if (total_new == 0) return SVW_OK;
  if (!workspace || workspace_bytes < svw_paged_attention_workspace_size(total_new, n_q_heads, Hkv, D))
    return SVW_ERR_WORKSPACE;
  svw::AttendArgs a{};
  a.q = q;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.Hq = n_q_heads;
  a.Hkv = Hkv;
  a.D = D;
  a.N = N;
  a.cu = cu_new;
  a.T = total_new;
  a.kv_len = kv_len;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  for (int d = 0; d < 3; ++d) {
    a.kc[d] = c.k_stride[d];
    a.vc[d] = c.v_stride[d];
  }
  a.table = cache->block_table;
  a.table_stride = cache->table_stride;
  a.max_pages = cache->max_pages;
  a.n_pages = cache->n_pages;
  a.page_size = ps;
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.ws = workspace;
  a.tag = next_epoch();
  a.fault = svw::test_fault();
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = codes ? svw::launch_attention_fp8(a, st) : svw::launch_attention(a, st);
  return e == cudaSuccess ? SVW_OK : SVW_ERR_CUDA;
}

svw_status paged_attention(const void *q, int64_t q_token_stride, int64_t q_head_stride, svw_dtype dtype,
                           int32_t n_q_heads, int32_t N, const int32_t *cu_new, int64_t total_new,
                           const int32_t *kv_len, const svw_paged_kv *cache, float scale, int32_t causal,
                           int32_t window, void *out, float *lse, int32_t *status, void *workspace,
                           size_t workspace_bytes, void *stream) {
  return attention_entry(false, q, q_token_stride, q_head_stride, dtype, n_q_heads, N, cu_new, total_new, kv_len, cache,
                         nullptr, nullptr, scale, causal, window, out, lse, status, workspace, workspace_bytes, stream);
}

svw_status paged_attention_fp8(const void *q, int64_t q_token_stride, int64_t q_head_stride, svw_dtype dtype,
                               int32_t n_q_heads, int32_t N, const int32_t *cu_new, int64_t total_new,
                               const int32_t *kv_len, const svw_paged_kv *cache, const float *k_scale,
                               const float *v_scale, float scale, int32_t causal, int32_t window, void *out,
                               float *lse, int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  return attention_entry(true, q, q_token_stride, q_head_stride, dtype, n_q_heads, N, cu_new, total_new, kv_len, cache,
                         k_scale, v_scale, scale, causal, window, out, lse, status, workspace, workspace_bytes, stream);
}

}  // extern "C"
