// attention.cu -- attention of a chunk of new tokens over a paged cache
// (paged_attention).
//
// New token t of request i and query head h see keys j in [lo, hi):
//   hi = causal ? min(kv_len, p + 1) : kv_len,  lo = window ? max(0, p + 1 - window) : 0,
// p = kv_len - n_i + t its place;  out = sum_j softmax_j(scale q . k_j) v_j,
// lse = log sum_j exp(scale q . k_j).
//
// Work.  The G = n_q_heads / n_kv_heads query heads of a key head share its
// keys, so the rows of a tile are (token, head of the group) pairs: a unit is
// (request, up to two tiles of 128 rows, key head), and its keys are cut into
// tiles of 128.  All units' key tiles form one line, in a fixed order, that
// the CTAs (one per SM) share out evenly: lengths may be as ragged as they
// like, and one long request fills the GPU.  A CTA walks its stretch of the
// line unit by unit ("segments"); a unit that several CTAs share is left as
// partial results in the workspace (unnormalised output, reference and sum of
// each row) and joined by attention_join, in the order of the line, so results
// do not depend on timing.
//
// A CTA.  One warp loads (TMA: queries once per segment, each page's keys and
// values as 128-byte-swizzled boxes into a ring), one thread issues the
// products on the tensor cores (tcgen05.mma, fp32 accumulators in tensor
// memory), two warpgroups ("stages") do the softmax, each with a score tile
// and an output accumulator of its own, so that one's exponentials run beside
// the other's products.  With two row tiles, stage s owns tile s and both
// read the same keys; with one, the stages take alternate key tiles and their
// two accumulators are added at the end.
//   scores  S[128 rows, 128 keys] = Q K^T, both K-major from shared memory;
//   softmax a thread per row: running reference M and sum l in base 2;
//   output  O[128 rows, D] += P V with P (bf16) written over S in tensor
//           memory and V read as it lies, keys along K (MN-major).
// The reference: exp2(x - M) is exact algebra for any M, so M follows the
// row's maximum only when that has outgrown it by more than 8 (a factor 256:
// far from overflow, and the same relative rounding of P); only then are l
// and O multiplied by 2^(M - M').  P is rounded to bf16, the operand type of
// the second product; l sums the unrounded weights in fp32.
//
// Masks are ranges of places: scores outside [lo, hi) become -inf by
// selection (their products may be anything), key tiles that no row of the
// unit sees are never loaded, and value rows beyond kv_len in the last tile,
// which may hold NaN, are zeroed in shared memory before the product.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "svw_device.cuh"
#include "svw_internal.h"

namespace svw {

namespace {

constexpr int kRows = 128;     // rows of a score tile (the MMA's M)
constexpr int kKeys = 128;     // keys of a tile
constexpr int kThreads = 384;  // loader, MMA issuer, two idle warps; two softmax warpgroups
constexpr int kSoftWarps = 8;
constexpr int kSegRing = 4;
constexpr int kMaxGrid = 152;   // CTAs: one per SM
constexpr int kUnitCost = 1;    // a unit's fixed cost on the line, in key tiles
constexpr float kGrow = 8.f;    // the reference lags the maximum by at most this (base 2)
constexpr float kNaN = __builtin_nanf("");

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;                // 128-byte columns of a tile
  static constexpr int kTile = kRows * D * 2;           // bytes of a query, key or value tile
  static constexpr int kHalf = kRows * 128;             // bytes of one of its halves
  static constexpr int kRing = (D == 128) ? 5 : 12;     // key and value tiles in flight
};

// one stretch of a unit
struct Segment {
  int32_t tiles;   // key tiles (0: the end of the CTA's work)
  int32_t tok0;    // first token of row tile 0
  int32_t ntok0;   // tokens of row tile 0
  int32_t ntok1;   // tokens of row tile 1 (0: one row tile, stages alternate)
  int32_t pos0;    // place of tok0
  int32_t key0;    // first key of the segment
  int32_t kv;      // keys of the request
  int32_t hk;      // key head
  int32_t part;    // workspace part (-1: the unit is complete)
};

struct Control {
  unsigned long long full[12], empty[12];
  unsigned long long q_full[2], q_empty[2];
  unsigned long long s_full[2], p_full[2];
  unsigned long long o_full, o_free;
  unsigned long long seg_full[kSegRing], seg_empty[kSegRing];
  Segment seg[kSegRing];
  int32_t seg_bad[kSegRing];
  uint32_t tmem;
  int32_t err;
  int64_t total, scan[kThreads / 32];
  int32_t first_req;
  int64_t first_at;
  int32_t issued, q_issued;  // ring tiles, query tiles
  float2 ml[2][kRows];       // reference and sum of each stage's rows
};
constexpr int kControlBytes = 3072;
static_assert(sizeof(Control) <= kControlBytes, "control block");

using Joint = AttendJoint;

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D[tmem] (+)= A B^T, bf16 in, fp32 accumulate; A from shared or from tensor memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 consecutive columns of this thread's lane; the registers hold them after tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
  uint32_t *u = reinterpret_cast<uint32_t *>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *r) {
  const uint32_t *u = reinterpret_cast<const uint32_t *>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor of a 128-byte-swizzled tile: start address
// >> 4 (bits 0-13), leading-dimension offset >> 4 (16-29), stride-dimension
// offset >> 4 (32-45), version (46), swizzle mode 2 = 128-byte (61-63).
// K-major (queries, keys: rows of 64 elements of the head): the stride offset
// is the 1024 bytes between eight-row atoms, the leading one is not used.
// MN-major (values: rows of 64 elements along N, eight keys an atom): the
// stride offset is the 1024 bytes between atoms along K (the keys), the
// leading one the distance of the halves along N.
__device__ __forceinline__ uint64_t sw128(uint32_t saddr, uint32_t lead) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// Instruction descriptor of kind::f16: fp32 D (bits 4-5), bf16 A and B (7-9,
// 10-12), B MN-major (16), N >> 3 (17-22), M >> 4 (24-28).
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? (1u << 16) : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------------------
// the line of work
// ---------------------------------------------------------------------------
struct Request {
  int32_t c0, n, kv;
  bool bad;  // its keys cannot be read: one empty tile per unit, NaN results
};
// false: its range of new tokens is invalid, nothing of it is written
__device__ __forceinline__ bool read_request(const AttendArgs &a, int32_t i, Request &r) {
  const int32_t c0 = __ldg(a.cu + i), c1 = __ldg(a.cu + i + 1);
  r.c0 = c0;
  r.n = c1 - c0;
  r.kv = __ldg(a.kv_len + i);
  r.bad = r.kv < 0 || r.kv > a.max_pages * a.page_size;  // the product fits (checked by the host)
  if (r.bad) r.kv = 0;
  return c0 >= 0 && c1 >= c0 && c1 <= a.T;
}
// the key tiles [k0, k1) * 128 that the unit of tokens [t0, t0 + nt) sees: at least one (which may be empty)
__device__ __forceinline__ void unit_keys(const AttendArgs &a, const Request &r, int32_t t0, int32_t nt, int32_t &k0,
                                          int32_t &k1) {
  const int32_t first = r.kv - r.n + t0;  // place of the unit's first token
  int32_t hi = r.kv;
  if (a.causal) hi = min(hi, first + nt);
  int32_t lo = 0;
  if (a.window > 0) lo = max(0, first + 1 - min(a.window, first + 1 > 0 ? first + 1 : 1));
  k0 = lo / kKeys;
  k1 = max(k0 + 1, (hi + kKeys - 1) / kKeys);
}
// the length of request i's part of the line
__device__ __forceinline__ int64_t request_cost(const AttendArgs &a, const Request &r) {
  int64_t c = 0;
  for (int32_t t0 = 0; t0 < r.n; t0 += 2 * a.tile_tokens) {
    int32_t k0, k1;
    unit_keys(a, r, t0, min(2 * a.tile_tokens, r.n - t0), k0, k1);
    c += k1 - k0 + kUnitCost;
  }
  return c * a.Hkv;
}

// bounded wait of one lane for the whole warp; false: it gave up
__device__ __forceinline__ bool warp_wait(unsigned long long *bar, uint32_t parity) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait_bounded(bar, parity) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, AttendArgs a) {
  using Sh = Shape<D>;
  extern __shared__ __align__(1024) unsigned char dyn[];
  Control &sm = *reinterpret_cast<Control *>(dyn);
  const uint32_t base = smem_u32(dyn);
  const uint32_t q_smem = base + kControlBytes, ring = q_smem + 2 * Sh::kTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (base & 1023u) {  // the swizzle atoms need it; never seen
    if (tid == 0 && a.status) atomicOr(a.status, SVW_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < Sh::kRing; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], kSoftWarps / 2);
    }
    mbar_init(&sm.o_full, 2);
    mbar_init(&sm.o_free, kSoftWarps);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], kSoftWarps + 1);
    }
    sm.err = 0;
    sm.issued = 0;
    sm.q_issued = 0;
    sm.first_req = a.N;
    sm.first_at = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- this CTA's stretch of the line ----
  const int32_t per = (a.N + kThreads - 1) / kThreads;
  const int32_t r0 = min(a.N, tid * per), r1 = min(a.N, r0 + per);
  int64_t mine = 0;
  bool wrong = false;
  for (int32_t i = r0; i < r1; ++i) {
    Request r;
    if (read_request(a, i, r))
      mine += request_cost(a, r);
    else
      wrong = true;
    wrong |= r.bad || (i == 0 && r.c0 != 0) || (i == a.N - 1 && r.c0 + r.n != a.T);
  }
  if (wrong && cta == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, W = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.scan[w];
    W += sm.scan[w];
  }
  const int64_t b = W * cta / P, e = W * (cta + 1) / P;
  if (b < e && before <= b && b < before + mine) {
    for (int32_t i = r0; i < r1; ++i) {
      Request r;
      const int64_t c = read_request(a, i, r) ? request_cost(a, r) : 0;
      if (b < before + c) {
        sm.first_req = i;
        sm.first_at = before;
        break;
      }
      before += c;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sm.tmem;
  const int G = a.Hq / a.Hkv;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ------------------------------- loader -------------------------------
      const int box = min(a.page_size, kKeys);       // rows of a page's box
      const int boxes = kKeys / box;                 // pages of a key tile
      const int shift = 31 - __clz(a.page_size);
      int64_t at = sm.first_at;
      int32_t count = 0, qc = 0, k = 0;  // ring tiles, query tiles, segments so far
      bool ok = true;
      Joint joint = {W, -1, 0, 0, 0, 0, 0};
      for (int32_t i = sm.first_req; i < a.N && at < e && ok; ++i) {
        Request r;
        if (!read_request(a, i, r)) continue;
        for (int32_t t0 = 0; t0 < r.n && at < e && ok; t0 += 2 * a.tile_tokens) {
          const int32_t nt = min(2 * a.tile_tokens, r.n - t0);
          int32_t k0, k1;
          unit_keys(a, r, t0, nt, k0, k1);
          const int64_t cost = k1 - k0 + kUnitCost;
          if (at + cost * a.Hkv <= b) {  // all heads of these tokens lie before the stretch
            at += cost * a.Hkv;
            continue;
          }
          for (int32_t hk = 0; hk < a.Hkv && at < e && ok; ++hk, at += cost) {
            const int32_t j0 = static_cast<int32_t>(max(static_cast<int64_t>(0), b - at - kUnitCost));
            const int32_t j1 = static_cast<int32_t>(min(static_cast<int64_t>(k1 - k0), e - at - kUnitCost));
            if (j0 >= j1) continue;
            const int sl = k % kSegRing;
            ok = k < kSegRing || warp_wait(&sm.seg_empty[sl], static_cast<uint32_t>((k / kSegRing - 1) & 1));
            if (!ok) break;
            const bool whole = (j0 == 0 && j1 == k1 - k0);
            const int32_t ntok0 = min(nt, a.tile_tokens), ntok1 = nt - ntok0;
            if (lane == 0) {
              Segment &s = sm.seg[sl];
              s.tiles = j1 - j0;
              s.tok0 = r.c0 + t0;
              s.ntok0 = ntok0;
              s.ntok1 = ntok1;
              s.pos0 = r.kv - r.n + t0;
              s.key0 = (k0 + j0) * kKeys;
              s.kv = r.kv;
              s.hk = hk;
              s.part = whole ? -1 : 2 * cta + (j0 == 0 ? 1 : 0);
              sm.seg_bad[sl] = r.bad ? 1 : 0;
              if (j0 == 0 && !whole) {
                joint.last = static_cast<int32_t>(((at + cost) * P + W - 1) / W - 1);
                joint.tok0 = s.tok0;
                joint.ntok0 = ntok0;
                joint.ntok1 = ntok1;
                joint.hk = hk;
              }
              mbar_arrive(&sm.seg_full[sl]);
            }
            ++k;
            // the queries
            for (int s = 0; s < (ntok1 > 0 ? 2 : 1) && ok; ++s, ++qc) {
              const int qs = qc & 1;
              ok = qc < 2 || warp_wait(&sm.q_empty[qs], static_cast<uint32_t>((qc / 2 - 1) & 1));
              if (ok && lane == 0) {
                mbar_arrive_expect_tx(&sm.q_full[qs], static_cast<uint32_t>(G * a.tile_tokens * D * 2));
                for (int h = 0; h < Sh::kHalves; ++h)
                  tma_load_3d(q_smem + qs * Sh::kTile + h * Sh::kHalf, &tmQ, h * 64, hk * G,
                              r.c0 + t0 + s * a.tile_tokens, smem_u32(&sm.q_full[qs]));
              }
            }
            // the keys and values, a lane per page
            bool bad = false;
            for (int32_t j = j0; j < j1 && ok; ++j) {
              const int32_t key = (k0 + j) * kKeys;
              const int32_t have = max(0, min(kKeys, r.kv - key));
              const int need = (have + box - 1) / box;  // pages that hold keys of the request
              int32_t page = 0;
              if (lane < need) {
                page = __ldg(a.table + i * a.table_stride + ((key + lane * box) >> shift));
                if (page < 0 || page >= a.n_pages) {
                  bad = true;
                  page = a.n_pages;  // outside the tensor: reads as zeros
                }
              }
              const int row = key & (a.page_size - 1);  // 0 unless a page holds several tiles
              for (int v = 0; v < 2 && ok; ++v, ++count) {
                const int s = count % Sh::kRing;
                ok = count < Sh::kRing || warp_wait(&sm.empty[s], static_cast<uint32_t>((count / Sh::kRing - 1) & 1));
                if (!ok) break;
                if (v == 1 && j == j1 - 1) {
                  // the last arrival of the segment carries this to its epilogue
                  const bool any = __any_sync(0xffffffffu, bad);
                  if (any && lane == 0) {
                    sm.seg_bad[sl] = 1;
                    if (a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
                  }
                }
                if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], static_cast<uint32_t>(need * box * D * 2));
                __syncwarp();
                if (lane < need && lane < boxes) {
                  const uint32_t dst = ring + s * Sh::kTile + lane * box * 128;
                  for (int h = 0; h < Sh::kHalves; ++h)
                    tma_load_4d(dst + h * Sh::kHalf, v ? &tmV : &tmK, h * 64, row, hk, page, smem_u32(&sm.full[s]));
                }
              }
            }
          }
        }
      }
      // the end marker
      if (ok) ok = k < kSegRing || warp_wait(&sm.seg_empty[k % kSegRing], static_cast<uint32_t>((k / kSegRing - 1) & 1));
      if (lane == 0) {
        if (ok) {
          sm.seg[k % kSegRing].tiles = 0;
          mbar_arrive(&sm.seg_full[k % kSegRing]);
        } else {
          atomicOr(&sm.err, 1);
        }
        sm.issued = count;
        sm.q_issued = qc;
        a.joints[cta] = joint;
      }
    } else if (warp == 1 && lane == 0) {
      // ----------------------------- MMA issuer -----------------------------
      constexpr uint32_t id_s = idesc(kKeys, false), id_o = idesc(D, true);
      int32_t count = 0, qc = 0, k = 0, sc[2] = {0, 0};
      bool ok = true;
      auto wait = [&](unsigned long long *bar, int32_t n) {  // the n-th completion of bar
        if (ok && !mbar_wait_bounded(bar, static_cast<uint32_t>(n & 1))) ok = false;
        return ok;
      };
      auto wait_ring = [&](int32_t c) {
        const bool r = wait(&sm.full[c % Sh::kRing], c / Sh::kRing);
        tc_after();
        return r;
      };
      auto scores = [&](int s, int32_t q, int32_t c) {
        const uint32_t qa = q_smem + (q & 1) * Sh::kTile, ka = ring + (c % Sh::kRing) * Sh::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk / 4) * Sh::kHalf + (kk % 4) * 32;
          mma_ss(tmem + s * kKeys, sw128(qa + off, 16), sw128(ka + off, 16), id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(smem_u32(&sm.s_full[s]));
      };
      auto output = [&](int s, int32_t c, bool acc) {
        const uint32_t va = ring + (c % Sh::kRing) * Sh::kTile;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(tmem + 2 * kKeys + s * D, tmem + s * kKeys + kk * 8, sw128(va + kk * 2048, Sh::kHalf), id_o,
                 (acc || kk > 0) ? 1u : 0u);
      };
      auto release = [&](int32_t c) { tc_commit(smem_u32(&sm.empty[c % Sh::kRing])); };
      while (ok) {
        const int sl = k % kSegRing;
        if (!wait(&sm.seg_full[sl], k / kSegRing)) break;
        const int32_t n = sm.seg[sl].tiles;
        const bool two = sm.seg[sl].ntok1 > 0;
        if (n == 0) break;
        mbar_arrive(&sm.seg_empty[sl]);
        if (!wait(&sm.q_full[qc & 1], qc / 2)) break;
        if (two && !wait(&sm.q_full[(qc + 1) & 1], (qc + 1) / 2)) break;
        // key tile j: ring tile count + 2 j, values one behind
        const int lead = two ? 1 : 2;  // a stage's next key tile
        if (!wait_ring(count)) break;
        scores(0, qc, count);
        if (two) scores(1, qc + 1, count);
        release(count);
        if (!two && n > 1) {
          if (!wait_ring(count + 2)) break;
          scores(1, qc, count + 2);
          release(count + 2);
        }
        for (int32_t j = 0; j < n && ok; ++j) {
          const int32_t vt = count + 2 * j + 1, kt = count + 2 * (j + lead);
          const bool more = j + lead < n;
          for (int s = two ? 0 : (j & 1); s < (two ? 2 : (j & 1) + 1) && ok; ++s) {
            if (!wait(&sm.p_full[s], sc[s])) break;
            ++sc[s];
            if (j == 0 && k > 0 && s == 0 && !wait(&sm.o_free, k - 1)) break;
            if (!wait_ring(vt)) break;
            output(s, vt, j >= lead);
            if (!two || s == 1) release(vt);
            if (more) {
              if (!wait_ring(kt)) break;
              scores(s, two ? qc + s : qc, kt);
              if (!two || s == 1) release(kt);
            }
          }
        }
        if (!ok) break;
        // every product of the segment: its queries and accumulators
        tc_commit(smem_u32(&sm.q_empty[qc & 1]));
        if (two) tc_commit(smem_u32(&sm.q_empty[(qc + 1) & 1]));
        tc_commit(smem_u32(&sm.o_full));
        mbar_arrive(&sm.o_full);  // carries what the loader wrote about the segment
        count += 2 * n;
        qc += two ? 2 : 1;
        ++k;
      }
      if (!ok) atomicOr(&sm.err, 1);
    }
  } else {
    // ------------------------------- softmax --------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int s = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t t_s = tmem + lanes + s * kKeys, t_o = tmem + lanes + 2 * kKeys;
    const float k2 = a.scale * kLog2e;
    const int tok_of_row = row / G, head_of_row = row % G;
    int32_t count = 0, sc = 0, k = 0;
    bool ok = true;
    while (true) {
      const int sl = k % kSegRing;
      if (!(ok = warp_wait(&sm.seg_full[sl], static_cast<uint32_t>((k / kSegRing) & 1)))) break;
      const Segment g = sm.seg[sl];
      if (g.tiles == 0) break;
      const bool two = g.ntok1 > 0;
      const int tile = two ? s : 0;
      const int32_t ntok = tile ? g.ntok1 : g.ntok0;
      const int32_t pos = g.pos0 + tile * a.tile_tokens + tok_of_row;
      int32_t hi = g.kv, lo = 0;
      if (a.causal) hi = min(hi, pos + 1);
      if (a.window > 0) lo = max(0, pos + 1 - min(a.window, max(pos + 1, 1)));
      const bool live = tok_of_row < ntok;
      const bool warp_live = __any_sync(0xffffffffu, live);
      if (!live) hi = lo;  // rows of no token: nothing to see
      float M = -INFINITY, l = 0.f;
      bool first = true;
      for (int32_t j = two ? 0 : s; j < g.tiles; j += two ? 1 : 2) {
        const int32_t key = g.key0 + j * kKeys;
        if (!(ok = warp_wait(&sm.s_full[s], static_cast<uint32_t>(sc & 1)))) break;
        ++sc;
        tc_after();
        if (warp_live) {
          float x[kKeys];
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) tmem_ld32(t_s + c, x + c);
          tmem_wait_ld();
          if (!__all_sync(0xffffffffu, key >= lo && key + kKeys <= hi)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (key + c < lo || key + c >= hi) x[c] = -INFINITY;
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < kKeys; ++c) mx[c & 3] = fmaxf(mx[c & 3], x[c]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * k2;
          const bool grow = top > M + kGrow || (M == -INFINITY && top > M);
          const float f = grow ? (M == -INFINITY ? 0.f : ex2(M - top)) : 1.f;
          if (grow) M = top;
          l *= f;
          if (!first && __any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(t_o + s * D + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] *= f;
              tmem_st32(t_o + s * D + c, o);
            }
          }
          const float ref = (M == -INFINITY) ? 0.f : M;
          const float2 kk = make_float2(k2, k2), nr = make_float2(-ref, -ref);
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const float2 d = __ffma2_rn(make_float2(x[c + 2 * u], x[c + 2 * u + 1]), kk, nr);
              const float2 p = make_float2(ex2(d.x), ex2(d.y));
              if (u & 1)
                sum1 = __fadd2_rn(sum1, p);
              else
                sum0 = __fadd2_rn(sum0, p);
              w[u] = pack_bf16(p.x, p.y);
            }
            tmem_st16(t_s + c / 2, w);
          }
          const float2 t = __fadd2_rn(sum0, sum1);
          l += t.x + t.y;
        }
        if (key + kKeys > g.kv) {
          // value rows beyond the request's keys: whatever is there must not meet a weight of zero
          const int32_t vt = count + 2 * j + 1;
          if (!(ok = warp_wait(&sm.full[vt % Sh::kRing], static_cast<uint32_t>((vt / Sh::kRing) & 1)))) break;
          const int r0v = max(0, g.kv - key);
          unsigned char *v = dyn + (ring - base) + (vt % Sh::kRing) * Sh::kTile;
          for (int u = r0v * 8 + quad * 32 + lane; u < kKeys * 8; u += 128)
#pragma unroll
            for (int h = 0; h < Sh::kHalves; ++h)
              *reinterpret_cast<uint4 *>(v + h * Sh::kHalf + u * 16) = make_uint4(0, 0, 0, 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[s]);
        first = false;
      }
      if (!ok) break;
      // ---- the segment's results ----
      if (!(ok = warp_wait(&sm.o_full, static_cast<uint32_t>(k & 1)))) break;
      tc_after();
      const bool bad = *reinterpret_cast<volatile int32_t *>(&sm.seg_bad[sl]) != 0;
      // stages that alternated share the row: half the columns each
      float w0 = 1.f, w1 = 0.f;
      int c0 = 0, c1 = D;
      const bool both = !two && g.tiles > 1;
      if (!two) {
        sm.ml[s][row] = make_float2(M, l);
        named_sync(1, kSoftWarps * 32);
        const float2 m0 = sm.ml[0][row], m1 = sm.ml[1][row];
        M = both ? fmaxf(m0.x, m1.x) : m0.x;
        w0 = (m0.x == -INFINITY) ? 0.f : ex2(m0.x - M);
        w1 = (!both || m1.x == -INFINITY) ? 0.f : ex2(m1.x - M);
        l = w0 * m0.y + (both ? w1 * m1.y : 0.f);
        c0 = s * (D / 2);
        c1 = c0 + D / 2;
        named_sync(1, kSoftWarps * 32);
      }
      if (bad) l = kNaN;
      const int32_t tok = g.tok0 + tile * a.tile_tokens + tok_of_row;
      const int64_t orow = static_cast<int64_t>(tok) * a.Hq + g.hk * G + head_of_row;
      const int prow = tile * kRows + row;
      if (warp_live) {
        const float inv = (g.part >= 0) ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        for (int c = c0; c < c1; c += 32) {
          float o[32];
          tmem_ld32(t_o + (two ? s * D : 0) + c, o);
          if (both) {
            float o1[32];
            tmem_ld32(t_o + D + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = o[u] * w0 + o1[u] * w1;
          } else {
            tmem_wait_ld();
          }
          if (!live) continue;
          if (g.part < 0) {
            uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * D + c);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              dst[u] = make_uint4(pack_bf16(o[8 * u] * inv, o[8 * u + 1] * inv), pack_bf16(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                  pack_bf16(o[8 * u + 4] * inv, o[8 * u + 5] * inv), pack_bf16(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
          } else {
            float4 *dst = reinterpret_cast<float4 *>(a.part_o + (static_cast<int64_t>(g.part) * a.part_rows + prow) * D + c);
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          }
        }
        if (live && (two || s == 0)) {
          if (g.part >= 0)
            a.part_ml[static_cast<int64_t>(g.part) * a.part_rows + prow] = make_float2(M, l);
          else if (a.lse)
            a.lse[orow] = (l == 0.f) ? -INFINITY : (M + log2f(l)) * kLn2;
        }
      }
      tc_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.o_free);
        mbar_arrive(&sm.seg_empty[sl]);
      }
      count += 2 * g.tiles;
      ++k;
    }
    if (!ok && lane == 0) atomicOr(&sm.err, 1);
  }
  __syncthreads();
  if (sm.err) {
    // a wait gave up: what is in flight lands before the CTA goes
    if (tid == 0) {
      if (a.status) atomicOr(a.status, SVW_DEV_TIMEOUT);
      for (int32_t c = max(0, sm.issued - Sh::kRing); c < sm.issued; ++c)
        mbar_wait_bounded(&sm.full[c % Sh::kRing], static_cast<uint32_t>((c / Sh::kRing) & 1));
      for (int32_t c = max(0, sm.q_issued - 2); c < sm.q_issued; ++c)
        mbar_wait_bounded(&sm.q_full[c & 1], static_cast<uint32_t>((c / 2) & 1));
    }
    if (tid == 32) {
      mbar_init(&sm.seg_full[0], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      tc_commit(smem_u32(&sm.seg_full[0]));
      mbar_wait_bounded(&sm.seg_full[0], 0);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// A unit that CTAs c .. last shared: each row's parts brought to one reference
// and added, in the order of the line.  A warp per row.
template <int D>
__global__ void __launch_bounds__(256) attention_join(AttendArgs a, int P) {
  constexpr int E = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const Joint jt = a.joints[c];
  if (jt.last < 0) return;
  const int lane = threadIdx.x & 31, warps = static_cast<int>(gridDim.y) * 8;
  const int G = a.Hq / a.Hkv;
  const int rows0 = jt.ntok0 * G, rows = rows0 + jt.ntok1 * G;
  for (int r = static_cast<int>(blockIdx.y) * 8 + (threadIdx.x >> 5); r < rows; r += warps) {
    const int tile = r >= rows0 ? 1 : 0, in_tile = r - tile * rows0;
    const int prow = tile * kRows + in_tile;
    // the part of CTA q: its last segment for the first, its first one for the others
    auto part = [&](int q) { return static_cast<int64_t>(2 * q + (q == c ? 1 : 0)) * a.part_rows + prow; };
    auto some = [&](int q) { return q == c || jt.total * q / P < jt.total * (q + 1) / P; };
    float M = -INFINITY;
    for (int q = c + lane; q <= jt.last; q += 32)
      if (some(q)) M = fmaxf(M, a.part_ml[part(q)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float l = 0.f, acc[E];
#pragma unroll
    for (int u = 0; u < E; ++u) acc[u] = 0.f;
#pragma unroll 4
    for (int q = c; q <= jt.last; ++q) {
      if (!some(q)) continue;
      const float2 ml = a.part_ml[part(q)];
      const float w = (ml.x == -INFINITY) ? 0.f : ex2(ml.x - M);
      l += (ml.x == -INFINITY && ml.y == 0.f) ? 0.f : (ml.x == -INFINITY ? ml.y : w * ml.y);
      const float *o = a.part_o + part(q) * D + lane * E;
#pragma unroll
      for (int u = 0; u < E; ++u) acc[u] = fmaf(w, o[u], acc[u]);
    }
    const int tok = jt.tok0 + tile * a.tile_tokens + in_tile / G;
    const int64_t orow = static_cast<int64_t>(tok) * a.Hq + jt.hk * G + in_tile % G;
    const float inv = (l == 0.f) ? 0.f : 1.f / l;
    uint32_t *dst = reinterpret_cast<uint32_t *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + orow * D + lane * E);
#pragma unroll
    for (int u = 0; u < E / 2; ++u) dst[u] = pack_bf16(acc[2 * u] * inv, acc[2 * u + 1] * inv);
    if (a.lse && lane == 0) a.lse[orow] = (l == 0.f) ? -INFINITY : (M + log2f(l)) * kLn2;
  }
}

// the driver's tensor-map encoder, looked up once through the runtime
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool encode(CUtensorMap *map, const void *ptr, int rank, const int64_t *dims, const int64_t *strides, const int *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], es[4];
  for (int r = 0; r < rank; ++r) {
    d[r] = static_cast<cuuint64_t>(dims[r]);
    bx[r] = static_cast<cuuint32_t>(box[r]);
    es[r] = 1;
    if (r > 0) st[r - 1] = static_cast<cuuint64_t>(strides[r]) * 2;
  }
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(ptr), d, st, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tile_tokens(int32_t Hq, int32_t Hkv) { return kRows / (Hq / Hkv); }
// rows of a workspace part: two row tiles unless every unit fits one
int part_rows(int64_t T, int32_t Hq, int32_t Hkv) { return T <= tile_tokens(Hq, Hkv) ? kRows : 2 * kRows; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

template <int D>
cudaError_t launch(AttendArgs a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  const int G = a.Hq / a.Hkv, box = a.page_size < kKeys ? a.page_size : kKeys;
  const int64_t qd[3] = {D, a.Hq, a.T}, qs[3] = {1, a.q_hs, a.q_ts};
  const int qb[3] = {64, G, a.tile_tokens};
  const int64_t cd[4] = {D, a.page_size, a.Hkv, a.n_pages};
  const int64_t ks[4] = {1, a.kc[2], a.kc[1], a.kc[0]}, vs[4] = {1, a.vc[2], a.vc[1], a.vc[0]};
  const int cb[4] = {64, box, 1, 1};
  if (!encode(&mq, a.q, 3, qd, qs, qb) || !encode(&mk, a.k_cache, 4, cd, ks, cb) || !encode(&mv, a.v_cache, 4, cd, vs, cb))
    return cudaErrorInvalidValue;
  constexpr int smem = kControlBytes + (2 + Shape<D>::kRing) * Shape<D>::kTile;
  static std::mutex mu;
  static bool attr_done[64] = {};
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_done[dev]) {
      cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      attr_done[dev] = true;
    }
  }
  const int P = sms[dev] < kMaxGrid ? sms[dev] : kMaxGrid;
  void *tm = timer_before("paged_attention", st);
  paged_attention_kernel<D><<<P, kThreads, smem, st>>>(mq, mk, mv, a);
  timer_after(tm, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(P), 4, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  tm = timer_before("attention_join", st);
  e = cudaLaunchKernelEx(&cfg, attention_join<D>, a, P);
  timer_after(tm, st);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// joints | (reference, sum) of each part's rows | their outputs
size_t attention_workspace(int64_t T, int32_t Hq, int32_t Hkv, int32_t D) {
  const size_t rows = static_cast<size_t>(2 * kMaxGrid) * part_rows(T, Hq, Hkv);
  return round256(sizeof(Joint) * kMaxGrid) + round256(rows * sizeof(float2)) + round256(rows * D * sizeof(float));
}

cudaError_t launch_attention(const AttendArgs &args, cudaStream_t st) {
  AttendArgs a = args;
  a.tile_tokens = tile_tokens(a.Hq, a.Hkv);
  a.part_rows = part_rows(a.T, a.Hq, a.Hkv);
  const size_t rows = static_cast<size_t>(2 * kMaxGrid) * a.part_rows;
  char *ws = static_cast<char *>(a.ws);
  a.joints = reinterpret_cast<Joint *>(ws);
  a.part_ml = reinterpret_cast<float2 *>(ws + round256(sizeof(Joint) * kMaxGrid));
  a.part_o = reinterpret_cast<float *>(ws + round256(sizeof(Joint) * kMaxGrid) + round256(rows * sizeof(float2)));
  return a.D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace svw
