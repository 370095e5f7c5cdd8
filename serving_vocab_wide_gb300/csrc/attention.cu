// attention.cu -- attention of a chunk of new tokens over a paged cache
// (paged_attention).
//
// New token t of request i and query head h see keys j in [lo, hi):
//   hi = causal ? min(kv_len, p + 1) : kv_len,  lo = window ? max(0, p + 1 - window) : 0,
// p = kv_len - n_i + t its place;  out = sum_j softmax_j(scale q . k_j) v_j,
// lse = log sum_j exp(scale q . k_j).
//
// Work.  The G = n_q_heads / n_kv_heads query heads of a key head share its
// keys, so the rows of a tile are (token, head of the group) pairs, 128 of
// them (the tensor core's M).  A unit is (request, row tile or pair of row
// tiles, key head), and its keys are cut into tiles.  All units' key tiles form
// one line, in a fixed order, that the workers share out evenly: lengths may
// be as ragged as they like, and one long request fills the GPU.  A worker
// walks its stretch of the line unit by unit ("segments"); a unit that several
// workers share is left as partial results in the workspace (unnormalised
// output, reference and sum of each row) and joined by attention_join, in the
// order of the line, so results do not depend on timing.
//
// A CTA (one per SM) has two stages, each with a score tile and an output
// accumulator in tensor memory and softmax warps of its own, so that one's
// exponentials run beside the other's products.  Per worker one warp loads, or
// one for the keys and one for the values (TMA: queries once per segment, each
// page's keys and values as 128-byte-swizzled boxes into a ring), and one thread
// issues the products (tcgen05.mma, fp32 accumulators in tensor memory):
//   scores  S[128 rows, keys] = Q K^T, both K-major from shared memory;
//   softmax running reference M and sum l of each row in base 2;
//   output  O[128 rows, D] += P V with P (bf16) written over S in tensor
//           memory and V read as it lies, keys along K (MN-major).
// Two ways to use the stages, by the rows that a request brings on average:
//   narrow  (up to 128: decoding, verifying; bound by the bytes of the keys) a
//           stage is a worker: its own units, its own loads, key tiles of 64,
//           two score buffers so that the next scores are there when a softmax
//           ends.  Small tiles keep bytes in flight while values wait for their
//           weights: with key tiles of 128 shared by the stages (alternating)
//           the ring held 160 KB of which two slots were under way, 2.0 us a
//           tile against 1.47 us of its bytes' time.
//   wide    (more: prompts; bound by the products) the CTA is one worker, a unit
//           is two row tiles, one a stage, reading the same key tiles of 128.
//           (Two threads to a row, 64 keys each, exchanging their maxima: 557 us
//           against 469, more warps contending for the exponentials.)  Heads of
//           64 leave room in tensor memory for weights apart from the scores,
//           and the next scores are formed beside the softmax of these (128
//           heads of 64, two prompts over 4381 keys: 187 -> 177 us).
// Measured (us; 32 query heads, 8 key heads of 128; of 6.78 TB/s and 1898
// TFLOP/s): 64 decoding requests over 1000 to 16000 keys 209 (98%); 2220 new
// tokens of 256 requests over 512 to 8192 keys 448 (95%); 17 tokens over 131000
// keys 95 (83%); two prompts of 2048 over 8192 keys 371 to 391 in short runs
// (1580 to 1670 TFLOP/s, 83 to 88%) and 417 to 432 in long ones, at the power
// limit (75 to 78%).
// The reference: exp2(x - M) is exact algebra for any M, so M follows the
// row's maximum only when that has outgrown it by more than 8 (a factor 256:
// far from overflow, and the same relative rounding of P); only then are l
// and O multiplied by 2^(M - M').  P is rounded to bf16, the operand type of
// the second product; l sums the unrounded weights in fp32.
//
// Masks are ranges of places: scores outside [lo, hi) become -inf by
// selection (their products may be anything), key tiles and pages that no row
// of the unit sees are never loaded, value rows beyond kv_len in the last tile,
// which may hold NaN, are zeroed in shared memory before the product, and a row
// to which another token's NaN or infinity got is formed again (redo_rows).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "steps_internal.h"
#include "svw_device.cuh"

namespace svw {

namespace {

constexpr int kRows = 128;     // rows of a score tile (the MMA's M)
constexpr int kSegRing = 4;
constexpr int kThreads = 384;  // loaders and issuers; two softmax warpgroups, one a stage
constexpr int kMaxGrid = 152;  // CTAs: one per SM
constexpr float kGrow = 8.f;   // the reference lags the maximum by at most this (base 2)
constexpr float kNaN = __builtin_nanf("");

template <int D, bool kWide>
struct Shape {
  static constexpr int kWorkers = kWide ? 1 : 2;           // of a CTA
  static constexpr int kKeys = kWide ? 128 : 64;           // keys of a tile
  static constexpr int kTiles = kWide ? 2 : 1;             // row tiles of a unit, at most
  static constexpr int kBufs = kWide ? 1 : 2;              // score buffers of a stage
  static constexpr bool kApart = kWide && D == 64;         // weights in columns of their own, not over their scores
  static constexpr int kSoftWarps = kWide ? 8 : 4;         // softmax warps of a worker
  // a unit's fixed cost on the line, in key tiles (one or three: 10 prompts of 1 to 1275 tokens 92 or 83 us instead
  // of 85, 117 requests of 68 tokens 300 or 305 instead of 299; narrow with three, 2220 tokens 452 instead of 448)
  static constexpr int kUnitCost = 2;
  static constexpr int kHalves = D / 64;                   // 128-byte columns of a tile
  static constexpr int kQTile = kRows * D * 2;             // bytes of a query tile
  static constexpr int kQHalf = kRows * 128;               // bytes of one of its columns
  static constexpr int kTile = kKeys * D * 2;              // of a key or value tile
  static constexpr int kHalf = kKeys * 128;
  static constexpr int kRing = (D == 128) ? 5 : 11;        // key and value tiles in flight of a worker
  static constexpr int kControl = (D == 128 ? 3 : 4) << 10;  // a whole number of swizzle atoms
  static constexpr int kSmem = kControl + 2 * kQTile + kWorkers * kRing * kTile;
  // columns of tensor memory: scores of stage st, buffer u at st * 128 + u * 64; outputs at 256 + st * D; weights:
  __host__ __device__ static constexpr int weights(int st, int u) { return kApart ? 384 + st * 64 : st * 128 + u * 64; }
};
static_assert(Shape<128, true>::kSmem <= 232448 && Shape<128, false>::kSmem <= 232448, "shared memory");
static_assert(Shape<64, true>::kSmem <= 232448 && Shape<64, false>::kSmem <= 232448, "shared memory");

// one stretch of a unit
struct Segment {
  int32_t tiles;   // key tiles (0: the end of the worker's stretch)
  int32_t tok0;    // first token of row tile 0
  int32_t ntok0;   // tokens of row tile 0
  int32_t ntok1;   // tokens of row tile 1
  int32_t pos0;    // place of tok0
  int32_t key0;    // first key of the segment
  int32_t kv;      // keys of the request
  int32_t hk;      // key head
  int32_t req;     // request
  int32_t part;    // workspace part (-1: the unit is complete)
  int32_t first;   // the workers that share the unit
  int32_t last;
};

template <int kRing>
struct Lane {  // of a worker
  unsigned long long full[kRing], empty[kRing];
  unsigned long long seg_full[kSegRing], seg_empty[kSegRing];
  Segment seg[kSegRing];
  int32_t seg_bad[kSegRing];  // 1: a page that is none of the cache's, 2: every token is bad
  int32_t issued[2], q_issued;  // key tiles, value tiles; query tiles
  int32_t first_req;
  int64_t first_at;
};
template <int kRing, int kWorkers>
struct Control {
  Lane<kRing> lane[kWorkers];
  unsigned long long q_full[2], q_empty[2];
  unsigned long long s_full[4], p_full[4];  // 2 * stage + score buffer
  unsigned long long s_read[2];             // by stage (apart): the scores are in registers
  unsigned long long o_full[2], o_free[2], o_step[2];  // by stage: a segment's outputs; read; each tile's (narrow, apart)
  unsigned long long drain[2];  // by worker: its issuer's products, once a wait has given up
  uint32_t tmem;
  int32_t err;
  int32_t complete[2];  // by stage: every part of the unit is there
  int64_t scan[20];
};

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
// D[tmem] (+)= A B^T over 64 elements of K, bf16 in, fp32 accumulate: four
// products of 16 in one piece, so that their descriptors step by constants
// (one product at a time, from one thread, an issue took 63 cycles, about what
// a 128 x 128 x 16 product lasts; in fours from a converged warp at most 39).
// A and B K-major in shared memory: 32 bytes a step.
__device__ __forceinline__ void mma_ss_x4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 x, %1;\n\tmov.b64 y, %2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
      "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t"
      "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t"
      "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A in tensor memory (8 columns a step), B MN-major in shared memory (16 rows of 128 bytes a step)
__device__ __forceinline__ void mma_ts_x4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b32 x, %1;\n\tmov.b64 y, %2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t"
      "add.u32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, 1;\n\t"
      "add.u32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, 1;\n\t"
      "add.u32 x, x, 8;\n\tadd.s64 y, y, 128;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// one thread of a converged warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *r) {
  uint32_t *u = reinterpret_cast<uint32_t *>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *r) {
  const uint32_t *u = reinterpret_cast<const uint32_t *>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *u) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
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

// Four lanes' 16-byte pieces transposed: lane 4 i + c has piece c of lanes
// 4 i + r, r = 0 .. 3, so that they store 64 bytes of a row in one piece.
__device__ __forceinline__ void turn_pieces(uint32_t (&p)[4][4]) {
#pragma unroll
  for (int bit = 1; bit < 4; bit <<= 1) {
    const bool up = (threadIdx.x & bit) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? p[k][w] : p[k + bit][w], bit);
        (up ? p[k][w] : p[k + bit][w]) = got;
      }
    }
  }
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
// the first key that a token at place pos sees
__device__ __forceinline__ int32_t first_key(const AttendArgs &a, int32_t pos) {
  return a.window > 0 ? max(0, pos + 1 - min(a.window, max(pos + 1, 1))) : 0;
}
// of request r's token t0, and so of those after it
__device__ __forceinline__ int32_t unit_first(const AttendArgs &a, const Request &r, int32_t t0) {
  return first_key(a, r.kv - r.n + t0);
}
// the key tiles [k0, k1) that the unit of tokens [t0, t0 + nt) sees: at least one (which may be empty)
template <int kKeys>
__device__ __forceinline__ void unit_keys(const AttendArgs &a, const Request &r, int32_t t0, int32_t nt, int32_t &k0,
                                          int32_t &k1) {
  int32_t hi = r.kv;
  if (a.causal) hi = min(hi, r.kv - r.n + t0 + nt);
  k0 = unit_first(a, r, t0) / kKeys;
  k1 = max(k0 + 1, (hi + kKeys - 1) / kKeys);
}
// the length of request r's part of the line
template <typename Sh>
__device__ __forceinline__ int64_t request_cost(const AttendArgs &a, const Request &r) {
  const int32_t step = Sh::kTiles * a.tile_tokens;
  int64_t c = 0;
  for (int32_t t0 = 0; t0 < r.n; t0 += step) {
    int32_t k0, k1;
    unit_keys<Sh::kKeys>(a, r, t0, min(step, r.n - t0), k0, k1);
    c += k1 - k0 + Sh::kUnitCost;
  }
  return c * a.Hkv;
}

// bounded wait of a converged warp; false: it gave up
__device__ __forceinline__ bool warp_wait(unsigned long long *bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}
// the parity of a barrier's n-th completion
__device__ __forceinline__ uint32_t par(int32_t n) { return static_cast<uint32_t>(n & 1); }

// -------------------------------- the loader --------------------------------
// A worker's keys, values or both (kinds [kFrom, kTo)).  The copies of a tile's
// pages go out one by one, 0.1 us each, so the wide form has a warp for each
// kind; the keys' loader also announces the segments and loads the queries.
template <int D, bool kWide, int kFrom, int kTo, typename C>
__device__ __forceinline__ void load_worker(const CUtensorMap &tmQ, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                            const AttendArgs &a, C &sm, int wk, int worker, int64_t W, int64_t b,
                                            int64_t e, int64_t workers, uint32_t q_smem, uint32_t ring) {
  using Sh = Shape<D, kWide>;
  auto &ln = sm.lane[wk];
  const int lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const int box = min(a.page_size, Sh::kKeys);  // rows of a page's box
  const int shift = 31 - __clz(a.page_size);
  const int32_t step = Sh::kTiles * a.tile_tokens;
  int64_t at = ln.first_at;
  int32_t count = 0, qc = 0, k = 0;  // tiles of a kind, query tiles, segments so far
  int32_t sent[2] = {0, 0};
  bool ok = true;
  Joint joint = {-1, 0, 0, 0, 0, {}};
  for (int32_t i = ln.first_req; i < a.N && at < e && ok; ++i) {
    Request r;
    if (!read_request(a, i, r)) continue;
    const int32_t *table = a.table + i * a.table_stride;
    for (int32_t t0 = 0; t0 < r.n && at < e && ok; t0 += step) {
      const int32_t nt = min(step, r.n - t0);
      int32_t k0, k1;
      unit_keys<Sh::kKeys>(a, r, t0, nt, k0, k1);
      const int64_t cost = k1 - k0 + Sh::kUnitCost;
      if (at + cost * a.Hkv <= b) {  // all heads of these tokens lie before the stretch
        at += cost * a.Hkv;
        continue;
      }
      for (int32_t hk = 0; hk < a.Hkv && at < e && ok; ++hk, at += cost) {
        const int32_t j0 = static_cast<int32_t>(max(static_cast<int64_t>(0), b - at - Sh::kUnitCost));
        const int32_t j1 = static_cast<int32_t>(min(static_cast<int64_t>(k1 - k0), e - at - Sh::kUnitCost));
        if (j0 >= j1) continue;
        // the segment's pages, 32 ids at a time, the next 32 under way
        const int32_t first_page = unit_first(a, r, t0) >> shift;
        const int32_t p_end = (min(r.kv, (k0 + j1) * Sh::kKeys) + a.page_size - 1) >> shift;
        int32_t p_base = ((k0 + j0) * Sh::kKeys) >> shift;
        int32_t ids = (p_base + lane < p_end) ? __ldg(table + p_base + lane) : 0;
        int32_t next_ids = (p_base + 32 + lane < p_end) ? __ldg(table + p_base + 32 + lane) : 0;
        const int sl = k % kSegRing;
        ok = kFrom > 0 || k < kSegRing || warp_wait(&ln.seg_empty[sl], par(k / kSegRing - 1));
        if (!ok) break;
        const bool whole = (j0 == 0 && j1 == k1 - k0);
        const int32_t ntok0 = min(nt, a.tile_tokens), ntok1 = nt - ntok0;
        if (kFrom == 0 && lane == 0) {
          Segment &s = ln.seg[sl];
          s.tiles = j1 - j0;
          s.tok0 = r.c0 + t0;
          s.ntok0 = ntok0;
          s.ntok1 = ntok1;
          s.pos0 = r.kv - r.n + t0;
          s.key0 = (k0 + j0) * Sh::kKeys;
          s.kv = r.kv;
          s.hk = hk;
          s.req = i;
          s.part = whole ? -1 : 2 * worker + (j0 == 0 ? 1 : 0);
          // position x of the line is worker ((x + 1) workers - 1) / W's
          s.first = static_cast<int32_t>(((at + Sh::kUnitCost + 1) * workers - 1) / W);
          s.last = static_cast<int32_t>(((at + cost) * workers - 1) / W);
          ln.seg_bad[sl] = r.bad ? 2 : 0;
          if (j0 == 0 && !whole) {
            joint.last = s.last;
            joint.tok0 = s.tok0;
            joint.ntok0 = ntok0;
            joint.ntok1 = ntok1;
            joint.hk = hk;
          }
          mbar_arrive(&ln.seg_full[sl]);
        }
        ++k;
        // the queries: the two tiles of a wide unit, one buffer each; the worker's one otherwise
        ok = kFrom > 0 || qc == 0 || warp_wait(&sm.q_empty[wk], par(qc - 1));
        if (kFrom == 0 && ok && lane == 0) {
          const int tiles = kWide ? 2 : 1;
          mbar_arrive_expect_tx(&sm.q_full[wk], static_cast<uint32_t>(tiles * G * a.tile_tokens * D * 2));
          for (int s = 0; s < tiles; ++s)
            for (int h = 0; h < Sh::kHalves; ++h)
              tma_load_3d(q_smem + s * Sh::kQTile + h * Sh::kQHalf, &tmQ, h * 64, hk * G, r.c0 + t0 + s * a.tile_tokens,
                          smem_u32(&sm.q_full[wk]));
        }
        if (ok) ++qc;
        // the keys and values, a lane per page
        bool bad = false;
        for (int32_t j = j0; j < j1 && ok; ++j, ++count) {
          const int32_t key = (k0 + j) * Sh::kKeys;
          const int32_t have = max(0, min(Sh::kKeys, r.kv - key));
          const int need = (have + box - 1) / box;  // pages that hold keys of the request
          if ((key >> shift) >= p_base + 32) {      // a tile's pages never straddle 32: it has a power of two of them
            p_base += 32;
            ids = next_ids;
            next_ids = (p_base + 32 + lane < p_end) ? __ldg(table + p_base + 32 + lane) : 0;
          }
          const int32_t id = (key + lane * box) >> shift;
          int32_t page = __shfl_sync(0xffffffffu, ids, min(31, id - p_base));
          if (lane < need && (page < 0 || page >= a.n_pages)) {
            bad |= id >= first_page;  // those before lie behind every token's window
            page = a.n_pages;         // outside the tensor: reads as zeros
          }
          const int row = key & (a.page_size - 1);  // 0 unless a page holds several tiles
          for (int v = kFrom; v < kTo && ok; ++v) {
            const int n = 2 * count + v, s = n % Sh::kRing;
            ok = n < Sh::kRing || warp_wait(&ln.empty[s], par(n / Sh::kRing - 1));
            if (a.fault == 1 && v == 1 && worker % 2 == 0) ok = false;  // test-only: no values come
            if (!ok) break;
            if (v == 0 && j == j1 - 1 && __any_sync(0xffffffffu, bad) && lane == 0) {
              ln.seg_bad[sl] = 1;  // the last keys' arrival carries this to the segment's epilogue
              if (a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
            }
            if (lane == 0) mbar_arrive_expect_tx(&ln.full[s], static_cast<uint32_t>(need * box * D * 2));
            ++sent[v];
            __syncwarp();
            if (lane < need) {
              const uint32_t dst = ring + s * Sh::kTile + lane * box * 128;
              for (int h = 0; h < Sh::kHalves; ++h)
                tma_load_4d(dst + h * Sh::kHalf, v ? &tmV : &tmK, h * 64, row, hk, page, smem_u32(&ln.full[s]));
            }
          }
        }
      }
    }
  }
  // the end marker
  if (kFrom == 0 && ok) ok = k < kSegRing || warp_wait(&ln.seg_empty[k % kSegRing], par(k / kSegRing - 1));
  if (lane == 0) {
    if (!ok) atomicOr(&sm.err, 1);
    for (int v = kFrom; v < kTo; ++v) ln.issued[v] = sent[v];
    if (kFrom == 0) {
      if (ok) {
        ln.seg[k % kSegRing].tiles = 0;
        mbar_arrive(&ln.seg_full[k % kSegRing]);
      }
      ln.q_issued = qc;
      a.joints[worker] = joint;
    }
  }
}

// ------------------------------ the MMA issuer ------------------------------
// A converged warp per worker; one of its threads issues.  (On two prompts of
// 2048 new tokens over 8192, 370 us: an issuer for each stage of the wide form,
// products interleaving as they come, 471, since both stages then wait for
// their products at the same time; taking turns, 435.)
template <int D, bool kWide, typename C>
__device__ __forceinline__ void issue_worker(C &sm, int wk, uint32_t q_smem, uint32_t ring, uint32_t tmem) {
  using Sh = Shape<D, kWide>;
  constexpr uint32_t id_s = idesc(Sh::kKeys, false), id_o = idesc(D, true);
  auto &ln = sm.lane[wk];
  // a place in the ring: slot and parity of its next completion
  struct At {
    int slot;
    uint32_t parity;
    __device__ void two_on() {  // the next tile of the same kind
      slot += 2;
      if (slot >= Sh::kRing) {
        slot -= Sh::kRing;
        parity ^= 1u;
      }
    }
  };
  At kt = {0, 0}, vt = {1, 0};
  int32_t k = 0, sc[2] = {0, 0};
  bool ok = true;
  auto wait_ring = [&](const At &t) { return ok = ok && warp_wait(&ln.full[t.slot], t.parity); };
  // by the elected thread: into score buffer u of stage st, from it into the stage's output
  auto scores = [&](int st, int u, const At &t) {
    const uint64_t qa = sw128(q_smem + (kWide ? st * Sh::kQTile : 0), 16), ka = sw128(ring + t.slot * Sh::kTile, 16);
#pragma unroll
    for (int h = 0; h < Sh::kHalves; ++h)
      mma_ss_x4(tmem + st * 128 + u * 64, qa + h * (Sh::kQHalf >> 4), ka + h * (Sh::kHalf >> 4), id_s, h);
    tc_commit(smem_u32(&sm.s_full[2 * st + u]));
  };
  auto output = [&](int st, int u, const At &t, bool acc) {
    const uint64_t va = sw128(ring + t.slot * Sh::kTile, Sh::kHalf);
#pragma unroll
    for (int h = 0; h < Sh::kKeys / 64; ++h)  // a row's weights of 64 keys take 32 columns
      mma_ts_x4(tmem + 256 + st * D, tmem + Sh::weights(st, u) + h * 32, va + h * 512, id_o, (acc || h > 0) ? 1u : 0u);
    if (!kWide || Sh::kApart) tc_commit(smem_u32(&sm.o_step[st]));
  };
  auto release = [&](const At &t) { tc_commit(smem_u32(&ln.empty[t.slot])); };
  while (ok) {
    const int sl = k % kSegRing;
    if (!(ok = warp_wait(&ln.seg_full[sl], par(k / kSegRing)))) break;
    const int32_t n = ln.seg[sl].tiles;
    __syncwarp();
    if (n == 0) break;
    if (elect_one()) mbar_arrive(&ln.seg_empty[sl]);
    if (!(ok = warp_wait(&sm.q_full[wk], par(k)))) break;
    // the first scores: both stages of the wide form, both buffers of the narrow one
#pragma unroll
    for (int u = 0; u < (kWide ? 1 : 2); ++u) {
      if (u < n) {
        if (!wait_ring(kt)) break;
        tc_after();
        if (elect_one()) {
          scores(kWide ? 0 : wk, u, kt);
          if (kWide) scores(1, 0, kt);
          release(kt);
        }
        kt.two_on();
      }
    }
    constexpr int kLead = kWide ? 1 : 2;  // a score buffer's next key tile
    for (int32_t j = 0; j < n && ok; ++j) {
      const bool more = j + kLead < n;
      if (Sh::kApart) {
        // the next scores as soon as these are read, beside the softmax of these
        if (more && !wait_ring(kt)) break;
#pragma unroll
        for (int i = 0; i < 2 && ok; ++i) {
          if (more && !(ok = warp_wait(&sm.s_read[i], par(sc[i])))) break;
          tc_after();
          if (elect_one()) {
            if (more) scores(i, 0, kt);
            if (more && i == 1) release(kt);
            if (i == 1 && j == max(0, n - 2)) tc_commit(smem_u32(&sm.q_empty[0]));
          }
        }
        if (!ok || !wait_ring(vt)) break;
#pragma unroll
        for (int i = 0; i < 2 && ok; ++i) {
          if (!(ok = warp_wait(&sm.p_full[2 * i], par(sc[i])))) break;
          ++sc[i];
          if (j == 0 && k > 0 && !(ok = warp_wait(&sm.o_free[i], par(k - 1)))) break;
          tc_after();
          if (elect_one()) {
            output(i, 0, vt, j > 0);
            if (i == 1) release(vt);
          }
        }
        vt.two_on();
        if (more) kt.two_on();
        continue;
      }
      if (!wait_ring(vt)) break;
      if (kWide && more && !wait_ring(kt)) break;  // there long before; narrow: its values' weights come first
#pragma unroll
      for (int i = 0; i < (kWide ? 2 : 1); ++i) {
        const int st = kWide ? i : wk, u = kWide ? 0 : (j & 1);
        if (!(ok = warp_wait(&sm.p_full[2 * st + u], par(sc[kWide ? i : u])))) break;
        ++sc[kWide ? i : u];
        if (j == 0 && k > 0 && !(ok = warp_wait(&sm.o_free[st], par(k - 1)))) break;
        tc_after();
        if (elect_one()) {
          output(st, u, vt, j > 0);
          if (!kWide || i == 1) release(vt);
          if (kWide && more) {
            scores(st, 0, kt);
            if (i == 1) release(kt);
          }
          // every score of the segment is under way: the queries may be replaced after them
          if (kWide && i == 1 && j == max(0, n - 2)) tc_commit(smem_u32(&sm.q_empty[0]));
        }
        if (!kWide) {
          if (more && !wait_ring(kt)) break;
          tc_after();
          if (elect_one()) {
            if (more) {
              scores(st, u, kt);
              release(kt);
            }
            if (j == max(0, n - 3)) tc_commit(smem_u32(&sm.q_empty[wk]));
          }
        }
      }
      vt.two_on();
      if (more) kt.two_on();
    }
    if (!ok) break;
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < (kWide ? 2 : 1); ++i) {
        tc_commit(smem_u32(&sm.o_full[kWide ? i : wk]));
        mbar_arrive(&sm.o_full[kWide ? i : wk]);  // carries what the loader wrote about the segment
      }
    }
    ++k;
  }
  if (!ok && elect_one()) atomicOr(&sm.err, 1);
}

// ---------------------------------------------------------------------------
// units that several workers shared
// ---------------------------------------------------------------------------
// the part of worker c + q: its last segment for the first, its first one for the others
__device__ __forceinline__ int part_of(int c, int q) { return 2 * (c + q) + (q == 0 ? 1 : 0); }

// Each row's parts brought to one reference and added, in the order of the
// line: warp w of `warps` takes rows w, w + warps, ...; the first kAhead parts'
// outputs are under way beside the references and sums.
template <int D, int kAhead>
__device__ __forceinline__ void join_rows(const AttendArgs &a, const Joint &jt, int c, int w, int warps) {
  constexpr int E = D / 32;
  const int G = a.Hq / a.Hkv;
  const int rows0 = jt.ntok0 * G, rows = rows0 + jt.ntok1 * G;
  const int lane = threadIdx.x & 31;
  const int n = jt.last - c + 1;
  for (int r = w; r < rows; r += warps) {
    const int tile = r >= rows0 ? 1 : 0, in_tile = r - tile * rows0;
    auto at = [&](int q) {  // rows of all parts: below 2^18
      return static_cast<uint32_t>(part_of(c, q) * a.part_rows + tile * kRows + in_tile);
    };
    auto load = [&](int q, float *o) {
      const float *src = a.part_o + (at(q) * D + lane * E);
      if (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
        o[0] = v.x, o[1] = v.y, o[E - 2] = v.z, o[E - 1] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
        o[0] = v.x, o[1] = v.y;
      }
    };
    float o[kAhead][E];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (u < n) load(u, o[u]);
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) ml = __ldcg(a.part_ml + at(lane));
    float M = ml.x;
    for (int q = lane + 32; q < n; q += 32) M = fmaxf(M, __ldcg(&a.part_ml[at(q)].x));
#pragma unroll
    for (int u = 16; u > 0; u >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, u));
    float l = 0.f, acc[E];
#pragma unroll
    for (int u = 0; u < E; ++u) acc[u] = 0.f;
    for (int q0 = 0; q0 < n; q0 += 32) {
      if (q0 > 0) {
        ml = make_float2(-INFINITY, 0.f);
        if (q0 + lane < n) ml = __ldcg(a.part_ml + at(q0 + lane));
      }
      const float wt = (ml.x == -INFINITY) ? 0.f : ex2(ml.x - M);
      const float wl = (ml.x == -INFINITY) ? ml.y : wt * ml.y;  // an empty part has 0, a bad one NaN
      const int m = min(32, n - q0);
      for (int b = 0; b < m; b += kAhead) {
        if (q0 + b > 0) {
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (b + u < m) load(q0 + b + u, o[u]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const float wu = __shfl_sync(0xffffffffu, wt, min(31, b + u)), lu = __shfl_sync(0xffffffffu, wl, min(31, b + u));
          if (b + u < m) {
            l += lu;
#pragma unroll
            for (int v = 0; v < E; ++v) acc[v] = (wu == 0.f) ? acc[v] : fmaf(wu, o[u][v], acc[v]);
          }
        }
      }
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

// The join by whoever comes last, where units have few rows (one launch less:
// 6 us of a short call).  A worker's softmax warps, having written a part, mark
// it with the call's tag and look at the marks of the unit's other parts; the
// fence between the two lets the last of them see all marks, and it joins (two
// may both see them all: they write the same results).  No worker waits for
// another.  The joiner takes the marks off again, so that a graph that replays
// a call with its tag finds none.  A mark is 64 bits of the tag and the part's
// number: what else has been in the workspace does not look like one.
//
// A warp that has given up a wait must not leave the others at a barrier.  So
// all four of a stage vote before each part, and once at their end: one that
// goes votes too, its next barrier being the others' next one, and they go with
// it.  Behind a vote nothing waits for anything but the four.
__device__ __forceinline__ bool all_here(int s, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.and.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(1 + s), "r"(kRows)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ unsigned long long mark_of(const AttendArgs &a, int part) {
  return static_cast<unsigned long long>(static_cast<uint32_t>(a.tag)) * 0x9e3779b97f4a7c15ull ^
         static_cast<unsigned long long>(part + 1);
}
// false: a warp has gone
template <int D>
__device__ __forceinline__ bool mark_and_join(const AttendArgs &a, const Segment &g, int s, int row, int32_t *complete) {
  const Joint jt = {g.last, g.tok0, g.ntok0, g.ntok1, g.hk, {}};
  const int n = g.last - g.first + 1;
  __threadfence();  // this thread's share of the part
  if (!all_here(s, true)) return false;
  if (row == 0) {
    *complete = 1;
    *reinterpret_cast<volatile unsigned long long *>(a.marks + g.part) = mark_of(a, g.part);
    __threadfence();
  }
  named_sync(1 + s, kRows);
  for (int q = row; q < n; q += kRows) {
    const int part = part_of(g.first, q);
    if (*reinterpret_cast<volatile unsigned long long *>(a.marks + part) != mark_of(a, part)) *complete = 0;
  }
  named_sync(1 + s, kRows);
  if (*reinterpret_cast<volatile int32_t *>(complete) == 0) return true;
  __threadfence();
  join_rows<D, 8>(a, jt, g.first, row >> 5, kRows / 32);
  for (int q = row; q < n; q += kRows) a.marks[part_of(g.first, q)] = 0;
  return true;
}

// ---------------------------- what a mask hides -----------------------------
// A hidden key's weight is zero, and zero times a NaN or an infinity is NaN.  So
// a row with a NaN among its outputs, where a key hidden from one of the warp's
// rows holds such a value, is formed again, by the warp, from the keys that it
// sees (the sum of its weights needs nothing: scores are hidden by selection).
// Keys that a mask hides within a segment are few; a NaN that a row sees is its
// result.  (The look at the outputs' sum costs 1% of two prompts' time, 4% where
// units have 2 tiles.)
__device__ __forceinline__ const __nv_bfloat16 *cache_row(const AttendArgs &a, const void *cache, const int64_t (&st)[3],
                                                          const int32_t *table, int32_t hk, int32_t j) {
  const int32_t page = __ldg(table + j / a.page_size);
  if (page < 0 || page >= a.n_pages) return nullptr;  // behind every token's window
  return static_cast<const __nv_bfloat16 *>(cache) + page * st[0] + hk * st[1] + (j % a.page_size) * st[2];
}
// does a value of keys [from, to) hold a NaN or an infinity?  A lane per key.
template <int D>
__device__ __forceinline__ bool odd_values(const AttendArgs &a, const int32_t *table, int32_t hk, int32_t from, int32_t to) {
  bool odd = false;
  for (int32_t j = from + (threadIdx.x & 31); j < to; j += 32) {
    const __nv_bfloat16 *v = cache_row(a, a.v_cache, a.vc, table, hk, j);
    if (!v) continue;
#pragma unroll 4
    for (int e = 0; e < D; e += 8) {
      const uint4 w = *reinterpret_cast<const uint4 *>(v + e);
      for (uint32_t x : {w.x, w.y, w.z, w.w}) odd |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
    }
  }
  return __any_sync(0xffffffffu, odd);
}
// Of a warp: rows `again` (by lane) of the segment's keys [key0, key1).  from_prow: lane 0's row of the part, -1: the
// outputs are the result.  bad_page: the segment has a page that is none of the cache's; rows that see one of its keys
// become NaN, and the lane is told so (the others are right, whatever unit they share).
template <int D>
__device__ __noinline__ bool redo_rows(const AttendArgs &a, uint32_t again, bool bad_page, int32_t req, int32_t hk,
                                       int32_t key0, int32_t key1, int32_t lo, int32_t hi, float M, float inv,
                                       int32_t orow, int64_t from_prow) {
  constexpr int E = D / 32, kMany = 8;  // elements of a lane; keys under way
  const int lane = threadIdx.x & 31;
  const int32_t *table = a.table + req * a.table_stride;
  auto put = [&](int from, int32_t row, int e, float x, float by) {
    if (from_prow >= 0)
      a.part_o[(from_prow + from) * D + lane * E + e] = x;
    else
      static_cast<__nv_bfloat16 *>(a.out)[static_cast<int64_t>(row) * D + lane * E + e] = __float2bfloat16_rn(x * by);
  };
  bool spoilt = false;
  if (bad_page) {
    const int32_t from = max(lo, key0), to = orow >= 0 ? min(hi, key1) : 0;
    for (int32_t p = from / a.page_size; !spoilt && from < to && p <= (to - 1) / a.page_size; ++p)
      if (const int32_t page = __ldg(table + p); page < 0 || page >= a.n_pages) spoilt = true;
    const uint32_t rows = __ballot_sync(0xffffffffu, spoilt);
    for (uint32_t left = rows; left; left &= left - 1) {
      const int32_t row = __shfl_sync(0xffffffffu, orow, __ffs(left) - 1);
      for (int e = 0; e < E; ++e) put(__ffs(left) - 1, row, e, kNaN, 1.f);
    }
    again &= ~rows;
    if (!again) return spoilt;
  }
  const bool mine = (again >> lane) & 1u;
  const int32_t lo_most = __reduce_max_sync(0xffffffffu, mine ? lo : 0);
  const int32_t hi_least = __reduce_min_sync(0xffffffffu, mine ? hi : INT32_MAX);
  if (!odd_values<D>(a, table, hk, key0, min(lo_most, key1)) && !odd_values<D>(a, table, hk, max(hi_least, key0), key1))
    return spoilt;
  const float k2 = a.scale * kLog2e;
  auto load = [&](const __nv_bfloat16 *p, float *x) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 f = bf16x2_f2(p ? *reinterpret_cast<const uint32_t *>(p + lane * E + e) : 0u);
      x[e] = f.x, x[e + 1] = f.y;
    }
  };
  for (; again; again &= again - 1) {
    const int from = __ffs(again) - 1;
    const int32_t row = __shfl_sync(0xffffffffu, orow, from);
    const float ref = __shfl_sync(0xffffffffu, M, from), by = __shfl_sync(0xffffffffu, inv, from);
    const int32_t begin = max(__shfl_sync(0xffffffffu, lo, from), key0);
    const int32_t end = min(__shfl_sync(0xffffffffu, hi, from), key1);
    float q[E], acc[E];
    load(static_cast<const __nv_bfloat16 *>(a.q) + row / a.Hq * a.q_ts + row % a.Hq * a.q_hs, q);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int32_t j0 = begin; j0 < end; j0 += kMany) {
      float k[kMany][E], v[kMany][E], s[kMany];
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        const bool in = j0 + u < end;
        load(in ? cache_row(a, a.k_cache, a.kc, table, hk, j0 + u) : nullptr, k[u]);
        load(in ? cache_row(a, a.v_cache, a.vc, table, hk, j0 + u) : nullptr, v[u]);
        s[u] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s[u] = fmaf(q[e], k[u][e], s[u]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < kMany; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
      for (int u = 0; u < kMany; ++u) {
        if (j0 + u >= end) break;
        const float p = __bfloat162float(__float2bfloat16_rn(ex2(fmaf(s[u], k2, -ref))));  // as the product takes it
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(p, v[u][e], acc[e]);
      }
      bool all_nan = true;  // and so they stay: a cache full of NaN is soon done with
#pragma unroll
      for (int e = 0; e < E; ++e) all_nan &= acc[e] != acc[e];
      if (__all_sync(0xffffffffu, all_nan)) break;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) put(from, row, e, acc[e], by);
  }
  return spoilt;
}

// ------------------------------- the softmax --------------------------------
// Of stage s: a thread has one row and all keys of a tile.
template <int D, bool kWide, bool kInside, typename C>
__device__ __forceinline__ void softmax_stage(const AttendArgs &a, C &sm, int s, unsigned char *ring_ptr, uint32_t tmem) {
  using Sh = Shape<D, kWide>;
  auto &ln = sm.lane[kWide ? 0 : s];
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int row = quad * 32 + lane;
  const int G = a.Hq / a.Hkv;
  const int tok_of_row = row / G, head_of_row = row - tok_of_row * G;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const uint32_t t_s = tmem + lanes + s * 128, t_p = tmem + lanes + Sh::weights(s, 0);
  const uint32_t t_o = tmem + lanes + 256 + s * D;
  const float k2 = a.scale * kLog2e;
  int32_t count = 0, k = 0, steps = 0, sc[2] = {0, 0};  // ring tiles, segments, outputs, score tiles by buffer
  bool ok = true, voted = false;  // voted: the stage's warps have agreed to go
  while (true) {
    const int sl = k % kSegRing;
    if (!(ok = warp_wait(&ln.seg_full[sl], par(k / kSegRing)))) break;
    const Segment g = ln.seg[sl];
    if (g.tiles == 0) break;
    const int tile = kWide ? s : 0;
    const int32_t pos = g.pos0 + tile * a.tile_tokens + tok_of_row;
    int32_t hi = g.kv, lo = first_key(a, pos);
    if (a.causal) hi = min(hi, pos + 1);
    const bool live = tok_of_row < (tile ? g.ntok1 : g.ntok0);
    const bool warp_live = __any_sync(0xffffffffu, live);
    if (!live) hi = INT32_MAX, lo = 0;  // rows of no token: never masked, never looked at
    float M = -INFINITY, l = 0.f;
    for (int32_t j = 0; j < g.tiles; ++j) {
      const int u = Sh::kBufs == 1 ? 0 : (j & 1);  // score buffer
      const int32_t key = g.key0 + j * Sh::kKeys;
      if (!(ok = warp_wait(&sm.s_full[2 * s + u], par(sc[u])))) break;
      ++sc[u];
      tc_after();
      const uint32_t t_su = t_s + u * 64;
      if (warp_live) {
        float x[Sh::kKeys];
#pragma unroll
        for (int c = 0; c < Sh::kKeys; c += 32) tmem_ld32(t_su + c, x + c);
        tmem_wait_ld();
        if (Sh::kApart) {
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_read[s]);
        }
        if (!__all_sync(0xffffffffu, key >= lo && key + Sh::kKeys <= hi)) {
          const int32_t from = key - lo;  // key + c is seen where 0 <= c + from < hi - lo
          const uint32_t seen = static_cast<uint32_t>(max(0, hi - lo));
#pragma unroll
          for (int c = 0; c < Sh::kKeys; ++c)
            if (static_cast<uint32_t>(c + from) >= seen) x[c] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < Sh::kKeys; c += 4)
#pragma unroll
          for (int v = 0; v < 4; ++v) mx[v] = fmaxf(mx[v], x[c + v]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * k2;
        const bool grow = live && (top > M + kGrow || (M == -INFINITY && top > M));
        const float f = grow ? (M == -INFINITY ? 0.f : ex2(M - top)) : 1.f;
        if (grow) M = top;
        l *= f;
        const float ref = (M == -INFINITY) ? 0.f : M;
        const float2 kk = make_float2(k2, k2), nr = make_float2(-ref, -ref);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
        uint32_t w[Sh::kKeys / 2];
#pragma unroll
        for (int c = 0; c < Sh::kKeys / 2; ++c) {
          const float2 d = __ffma2_rn(make_float2(x[2 * c], x[2 * c + 1]), kk, nr);
          const float2 p = make_float2(ex2(d.x), ex2(d.y));
          if (c & 1)
            sum1 = __fadd2_rn(sum1, p);
          else
            sum0 = __fadd2_rn(sum0, p);
          w[c] = pack_bf16(p.x, p.y);
          if (!Sh::kApart && (c & 7) == 7) tmem_st8(t_p + u * 64 + (c - 7), w + (c - 7));
        }
        const float2 t = __fadd2_rn(sum0, sum1);
        l += t.x + t.y;
        // the outputs so far are complete, and the weights read (wide, not apart: the scores' arrival said so)
        const bool rescale = j > 0 && __any_sync(0xffffffffu, grow);
        if (Sh::kApart ? j > 0 : (!kWide && rescale)) {
          if (!(ok = warp_wait(&sm.o_step[s], par(steps + j - 1)))) break;
          tc_after();
        }
        if (rescale) {
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int v = 0; v < 16; ++v) o[v] *= f;
            tmem_st16(t_o + c, o);
          }
        }
        if (Sh::kApart) {
#pragma unroll
          for (int c = 0; c < Sh::kKeys / 2; c += 8) tmem_st8(t_p + u * 64 + c, w + c);
        }
      } else if (Sh::kApart) {
        if (lane == 0) mbar_arrive(&sm.s_read[s]);
        // no further ahead than the others: two arrivals of a warp must not fall into one phase of p_full
        if (j > 0 && !(ok = warp_wait(&sm.o_step[s], par(steps + j - 1)))) break;
      }
      if (key + Sh::kKeys > g.kv) {
        // value rows beyond the request's keys: whatever is there must not meet a weight of zero
        const int32_t vt = count + 2 * j + 1;
        if (!(ok = warp_wait(&ln.full[vt % Sh::kRing], par(vt / Sh::kRing)))) break;
        unsigned char *v = ring_ptr + (vt % Sh::kRing) * Sh::kTile;
        for (int w = max(0, g.kv - key) * 8 + row; w < Sh::kKeys * 8; w += kRows)
#pragma unroll
          for (int q = 0; q < Sh::kHalves; ++q) *reinterpret_cast<uint4 *>(v + q * Sh::kHalf + w * 16) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[2 * s + u]);
    }
    if (!ok) break;
    // ---- the segment's results ----
    if (!(ok = warp_wait(&sm.o_full[s], par(k)))) break;
    tc_after();
    if (warp_live) {
      const int32_t bad = *reinterpret_cast<volatile int32_t *>(&ln.seg_bad[sl]);
      if (bad == 2) l = kNaN;
      const int32_t tok = g.tok0 + tile * a.tile_tokens + tok_of_row;
      const int32_t orow = live ? tok * a.Hq + g.hk * G + head_of_row : -1;  // below 2^31, checked by the host
      const int64_t prow = static_cast<int64_t>(max(g.part, 0)) * a.part_rows + tile * kRows + row;
      const float inv = (g.part >= 0) ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      int32_t to[4];  // the rows of this lane's four, and its piece of each
#pragma unroll
      for (int q = 0; q < 4; ++q) to[q] = __shfl_sync(0xffffffffu, orow, (lane & ~3) + q);
      const int piece = lane & 3;
      // does the segment have keys hidden from one of the rows?  Then their outputs' sum is looked at for a NaN
      const int32_t key1 = min(g.kv, g.key0 + g.tiles * Sh::kKeys);
      const bool hides = __any_sync(0xffffffffu, live && (lo > g.key0 || hi < key1));
      float2 odd = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(t_o + c, o);
        tmem_wait_ld();
        if (hides) {
#pragma unroll
          for (int v = 0; v < 32; v += 2) odd = __fadd2_rn(odd, make_float2(o[v], o[v + 1]));
        }
        uint32_t p[4][4];
        if (g.part < 0) {
#pragma unroll
          for (int v = 0; v < 16; ++v) p[v >> 2][v & 3] = pack_bf16(o[2 * v] * inv, o[2 * v + 1] * inv);
          turn_pieces(p);
          __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(a.out) + c + piece * 8;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (to[q] >= 0)
              *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(to[q]) * D) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
        } else {
          float *dst = a.part_o + (prow - piece) * D + c + piece * 4;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int v = 0; v < 16; ++v) p[v >> 2][v & 3] = __float_as_uint(o[h * 16 + v]);
            turn_pieces(p);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (to[q] >= 0) *reinterpret_cast<uint4 *>(dst + q * D + h * 16) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
          }
        }
      }
      // a weight of zero times a NaN or an infinity of a hidden key?
      const float sum = odd.x + odd.y;
      const uint32_t again = __ballot_sync(0xffffffffu, live && sum != sum && l == l && (lo > g.key0 || hi < key1));
      if (again != 0 || bad == 1) {
        __syncwarp();  // the rows are written
        if (redo_rows<D>(a, again, bad == 1, g.req, g.hk, g.key0, key1, lo, hi, M, inv, orow, g.part >= 0 ? prow - lane : -1))
          l = kNaN;
      }
      if (live) {
        if (g.part >= 0)
          a.part_ml[prow] = make_float2(M, l);
        else if (a.lse)
          a.lse[orow] = (l == 0.f) ? -INFINITY : (M + log2f(l)) * kLn2;
      }
    }
    tc_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.o_free[s]);
      mbar_arrive(&ln.seg_empty[sl]);
    }
    if (kInside && g.part >= 0) {
      if (a.fault == 1 && s == 1 && quad == 3) ok = false;  // test-only: as if this warp's wait had run out
      if (!ok || (voted = !mark_and_join<D>(a, g, s, row, &sm.complete[s]))) break;
    }
    count += 2 * g.tiles;
    steps += g.tiles;
    ++k;
  }
  if (kInside && !voted) all_here(s, ok);
  if (!ok) {
    tmem_wait_st();  // before another warp frees the columns
    tc_before();
    if (lane == 0) atomicOr(&sm.err, 1);
  }
}

// kInside: narrow, units joined by the last worker
template <int D, bool kWide, bool kInside>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttendArgs a) {
  using Sh = Shape<D, kWide>;
  using C = Control<Sh::kRing, Sh::kWorkers>;
  static_assert(sizeof(C) <= Sh::kControl, "control block");
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(1024) unsigned char dyn[];
  C &sm = *reinterpret_cast<C *>(dyn);
  const uint32_t base = smem_u32(dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (base & 1023u) {  // the swizzle atoms need it; never seen
    if (tid == 0 && a.status) atomicOr(a.status, SVW_DEV_TIMEOUT);
    if (tid < Sh::kWorkers) a.joints[blockIdx.x * Sh::kWorkers + tid].last = -1;  // nothing to join
    return;
  }
  if (tid == 0) {
    for (int w = 0; w < Sh::kWorkers; ++w) {
      auto &ln = sm.lane[w];
      for (int s = 0; s < Sh::kRing; ++s) {
        mbar_init(&ln.full[s], 1);
        mbar_init(&ln.empty[s], 1);
      }
      for (int s = 0; s < kSegRing; ++s) {
        mbar_init(&ln.seg_full[s], 1);
        mbar_init(&ln.seg_empty[s], Sh::kSoftWarps + 1);
      }
      ln.issued[0] = ln.issued[1] = 0;
      ln.q_issued = 0;
      ln.first_req = a.N;
      ln.first_at = 0;
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.drain[s], 1);
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.o_full[s], 2);
      mbar_init(&sm.o_free[s], 4);
      mbar_init(&sm.o_step[s], 1);
      mbar_init(&sm.s_read[s], 4);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 4);
    }
    sm.err = 0;
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

  // ---- the line, and the workers' stretches of it ----
  const int32_t per = (a.N + kThreads - 1) / kThreads;
  const int32_t r0 = min(a.N, tid * per), r1 = min(a.N, r0 + per);
  int64_t mine = 0;
  bool wrong = false;
  for (int32_t i = r0; i < r1; ++i) {
    Request r;
    if (read_request(a, i, r))
      mine += request_cost<Sh>(a, r);
    else
      wrong = true;
    wrong |= r.bad || (i == 0 && r.c0 != 0) || (i == a.N - 1 && r.c0 + r.n != a.T);
  }
  if (wrong && blockIdx.x == 0 && a.status) atomicOr(a.status, SVW_DEV_BAD_INPUT);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, W = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.scan[w];
    W += sm.scan[w];
  }
  // no empty stretch before the last: every worker that shares a unit has a part
  const int64_t workers = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x) * Sh::kWorkers, W));
  auto line = [&](int64_t w) { return W * min(w, workers) / workers; };  // where worker w's stretch begins
  for (int w = 0; w < Sh::kWorkers; ++w) {
    const int64_t id = static_cast<int64_t>(blockIdx.x) * Sh::kWorkers + w;
    const int64_t b = line(id), e = line(id + 1);
    if (b < e && before <= b && b < before + mine) {
      int64_t at = before;
      for (int32_t i = r0; i < r1; ++i) {
        Request r;
        const int64_t c = read_request(a, i, r) ? request_cost<Sh>(a, r) : 0;
        if (b < at + c) {
          sm.lane[w].first_req = i;
          sm.lane[w].first_at = at;
          break;
        }
        at += c;
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sm.tmem;
  const uint32_t q_smem = base + Sh::kControl, ring = q_smem + 2 * Sh::kQTile;
  constexpr int kRingBytes = Sh::kRing * Sh::kTile;

  // loaders and an issuer per worker; softmax warps from the fifth on
  if (warp < 4) {
    // the launch has 168 registers for each of 384 threads: 128 * 72 + 256 * 216
    if (kWide) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int wk = kWide ? 0 : warp >> 1;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * Sh::kWorkers + wk;
    const uint32_t my_q = q_smem + wk * Sh::kQTile, my_ring = ring + wk * kRingBytes;
    if (warp == 1 || (!kWide && warp == 3))
      issue_worker<D, kWide>(sm, wk, my_q, my_ring, tmem);
    else if (!kWide)
      load_worker<D, kWide, 0, 2>(tmQ, tmK, tmV, a, sm, wk, static_cast<int>(id), W, line(id), line(id + 1), workers, my_q, my_ring);
    else if (warp == 0)
      load_worker<D, kWide, 0, 1>(tmQ, tmK, tmV, a, sm, wk, static_cast<int>(id), W, line(id), line(id + 1), workers, my_q, my_ring);
    else if (warp == 2)
      load_worker<D, kWide, 1, 2>(tmQ, tmK, tmV, a, sm, wk, static_cast<int>(id), W, line(id), line(id + 1), workers, my_q, my_ring);
  } else {
    if (kWide) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int st = (warp - 4) >> 2;
    softmax_stage<D, kWide, kInside>(a, sm, st, dyn + (ring - base) + (kWide ? 0 : st * kRingBytes), tmem);
  }
  __syncthreads();
  if (sm.err) {
    // a wait gave up: what is in flight lands before the CTA goes
    if (tid == 0) {
      if (a.status) atomicOr(a.status, SVW_DEV_TIMEOUT);
      for (int w = 0; w < Sh::kWorkers; ++w) {
        auto &ln = sm.lane[w];
        // each slot's last tile: 2 n + v is the n-th of kind v
        uint32_t seen = 0;
        for (int32_t c = 2 * max(ln.issued[0], ln.issued[1]) - 1, q = 0; c >= 0 && q < 3 * Sh::kRing; --c, ++q) {
          if (c / 2 >= ln.issued[c & 1] || (seen >> (c % Sh::kRing) & 1u)) continue;
          seen |= 1u << (c % Sh::kRing);
          mbar_wait_bounded(&ln.full[c % Sh::kRing], par(c / Sh::kRing));
        }
        if (ln.q_issued > 0) mbar_wait_bounded(&sm.q_full[w], par(ln.q_issued - 1));
      }
    }
    if ((warp == 1 || warp == 3) && (warp >> 1) < Sh::kWorkers) {
      // an issuer's products: a commit by the thread that issued them, on a barrier of its own (earlier commits may
      // still be on their way to all others)
      unsigned long long *bar = &sm.drain[warp >> 1];
      if (elect_one()) {
        tc_commit(smem_u32(bar));
        mbar_wait_bounded(bar, 0);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// The join as a kernel of its own: a unit's rows over the blocks of a column.
// (One after the other, eight rows a warp, the joins of two prompts took 50 us.)
template <int D, bool kWide>
__global__ void __launch_bounds__(256, kWide ? 4 : 3) attention_join(const __grid_constant__ AttendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const Joint jt = a.joints[c];
  if (jt.last < 0) return;
  join_rows<D, kWide ? 4 : 8>(a, jt, c, static_cast<int>(blockIdx.y) * 8 + (threadIdx.x >> 5),
                              static_cast<int>(gridDim.y) * 8);
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
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// rows of the workspace's parts, two per worker: a row tile (no more rows than
// there are tokens) of the narrow form's 2 * kMaxGrid workers, or the two of the
// wide form's kMaxGrid
int narrow_rows(int64_t T, int G) { return static_cast<int>(T * G < kRows ? (T * G + 7) / 8 * 8 : kRows); }
size_t all_part_rows(int64_t T, int G) { return static_cast<size_t>(2 * 2 * kMaxGrid) * narrow_rows(T, G); }

template <int D, bool kWide, bool kInside>
cudaError_t launch(AttendArgs a, cudaStream_t st) {
  static_assert(!(kWide && kInside), "many rows are joined by a kernel of their own");
  using Sh = Shape<D, kWide>;
  CUtensorMap mq, mk, mv;
  const int G = a.Hq / a.Hkv, box = a.page_size < Sh::kKeys ? a.page_size : Sh::kKeys;
  const int64_t qd[3] = {D, a.Hq, a.T}, qs[3] = {1, a.q_hs, a.q_ts};
  const int qb[3] = {64, G, a.tile_tokens};
  const int64_t cd[4] = {D, a.page_size, a.Hkv, a.n_pages};
  const int64_t ks[4] = {1, a.kc[2], a.kc[1], a.kc[0]}, vs[4] = {1, a.vc[2], a.vc[1], a.vc[0]};
  const int cb[4] = {64, box, 1, 1};
  if (!encode(&mq, a.q, 3, qd, qs, qb) || !encode(&mk, a.k_cache, 4, cd, ks, cb) || !encode(&mv, a.v_cache, 4, cd, vs, cb))
    return cudaErrorInvalidValue;
  static std::mutex mu;
  static bool attr_done[64] = {};
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_done[dev]) {
      cudaError_t e =
          cudaFuncSetAttribute(paged_attention_kernel<D, kWide, kInside>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      attr_done[dev] = true;
    }
  }
  const int P = sms[dev] < kMaxGrid ? sms[dev] : kMaxGrid;
  a.part_rows = kWide ? 2 * kRows : narrow_rows(a.T, G);
  void *tm = timer_before("paged_attention", st);
  paged_attention_kernel<D, kWide, kInside><<<P, kThreads, Sh::kSmem, st>>>(mq, mk, mv, a);
  timer_after(tm, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || kInside) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // blocks for a unit's rows, on average (in a larger one a warp has several); two rows a warp when wide
  const int64_t rows = std::min<int64_t>(a.part_rows, a.T * G / a.N + 1);
  cfg.gridDim = dim3(static_cast<unsigned>(P * Sh::kWorkers), static_cast<unsigned>(kWide ? (rows + 15) / 16 : (rows + 7) / 8), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  tm = timer_before("attention_join", st);
  e = cudaLaunchKernelEx(&cfg, attention_join<D, kWide>, a);
  timer_after(tm, st);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

// joints | the parts' marks | (reference, sum) of each part's rows | their outputs
constexpr size_t kJointBytes = (sizeof(Joint) * 2 * kMaxGrid + 255) / 256 * 256;
constexpr size_t kMarkBytes = (sizeof(unsigned long long) * 2 * 2 * kMaxGrid + 255) / 256 * 256;
size_t attention_workspace(int64_t T, int32_t G, int32_t D) {
  const size_t rows = all_part_rows(T, G);
  return kJointBytes + kMarkBytes + round256(rows * sizeof(float2)) + rows * D * sizeof(float);
}

cudaError_t launch_attention(const AttendArgs &args, cudaStream_t st) {
  AttendArgs a = args;
  const int G = a.Hq / a.Hkv;
  a.tile_tokens = tile_tokens(a.Hq, a.Hkv);
  char *ws = static_cast<char *>(a.ws);
  a.joints = reinterpret_cast<Joint *>(ws);
  a.marks = reinterpret_cast<unsigned long long *>(ws + kJointBytes);
  a.part_ml = reinterpret_cast<float2 *>(ws + kJointBytes + kMarkBytes);
  a.part_o = reinterpret_cast<float *>(ws + kJointBytes + kMarkBytes + round256(all_part_rows(a.T, G) * sizeof(float2)));
  // The rows of a request, on average: up to one tile's the bytes of its keys
  // bound the work (128 rows are 128 flop per byte, the ridge lies at 280), and
  // more would read the keys once per tile in the narrow form.
  const bool wide = a.T * G > static_cast<int64_t>(kRows) * a.N;
  // A short call of few tokens: joined by the last worker.  (The launch that this
  // saves is 6 us of the host's time.  On the GPU, against a kernel of its own, 32
  // query heads of 128 on 8 key heads: one token over 777 keys 12.5 and 12.9 us,
  // over 60000 48.6 and 50.0, 32 tokens over 4000 88.2 and 87.8; with 64 on 4, so
  // that one warpgroup joins 16 rows of many parts, 4 tokens over 2000 21.6 and 16.6.)
  const bool inside = !wide && a.T <= 32 && a.T * G <= 16 * static_cast<int64_t>(a.N);
  if (a.D == 128)
    return wide ? launch<128, true, false>(a, st) : inside ? launch<128, false, true>(a, st) : launch<128, false, false>(a, st);
  return wide ? launch<64, true, false>(a, st) : inside ? launch<64, false, true>(a, st) : launch<64, false, false>(a, st);
}

}  // namespace svw
