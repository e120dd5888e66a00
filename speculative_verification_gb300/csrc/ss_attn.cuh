// ss_attn.cuh -- attention of a step's new tokens over the paged cache, on the
// tensor cores (ss_attn_bf16.cu and ss_attn_int4.cu instantiate it).
//
// The mathematics.  For a row n (one query of one head) and the keys j it
// sees, x_nj = scale log2(e) q_n.k_j, with a reference r_n (below):
//   p_nj = 2^(x_nj - r_n),  out_n = sum_j p_nj v_j / sum_j p_nj,
//   lse_n = ln 2 (r_n + log2 sum_j p_nj).
// Any r_n gives the same result; it only has to keep the powers in range.  The
// running maximum is the usual choice; here (bf16) r_n starts at 0 and moves
// only when some x_nj passes it by more than 16 (or the first ones lie below
// -32), so the accumulated sums are rarely rescaled and a tile needs no maximum
// over its keys at all (2 x 4096-token prompt chunks: 390 us when every item's
// first tile took its maximum and masks were tested per row, 341 since).
// Largest weights in [2^-32, 2^16] round no worse than those around 1, as bf16
// is relative; but they meet the values in fp32, whose range is that much
// narrower for the values.  Over 4 bits the weights are f16, whose range is
// short: there r_n is set at the first keys, and moves when a later one passes
// them by much (kSlack, kTop below).
//
// The transposed product.  A tile is 128 keys of one kv head; the rows are the
// new tokens of one request times the query heads that share the kv head,
// kN of them per work item (16 .. 128).  The first product is S^T = K Q^T
// (M = 128 keys, N = rows, K = head_dim), the second O^T += V^T P^T (M = 128
// channels, N = rows, K = 128 keys).  So the keys, not the rows, fill the 128
// lanes of tensor memory: a decode step with 4 or 8 rows wastes no lane, every
// thread owns one key (its page, mask and, in 4 bits, its step and low value),
// and K and V enter the tensor cores exactly as they lie in the cache ([key]
// [channel], K as a K-major and V as an M-major operand).
//
// 4 bits.  A row stands for s n + m, n = 0..15.  The tensor cores multiply the
// exact integers, and s and m enter in fp32:
//   q.k = s_k (q.n) + m_k sum(q)
//   sum_j p v = sum_j (p s_v) (n - 8) + sum_j p (m_v + 8 s_v),
// the first in fp32 on the thread that owns the key, the second by rounding
// p s_v to f16, plus one fp32 sum per row.  f16 has the range for it because
// the references then also count the keys' magnitudes and keep the largest
// weight near f16's upper end (kSlack, kTop).
//
// Roundings: P to bf16 (4 bits: p s_v to f16, whose 11 bits leave only the
// result's own rounding to see; weights 2^22 below a row's largest and smaller
// lose bits, 2^33 below it they are 0), the result to bf16; everything else is
// fp32 (sums of p on the unrounded values).
//
// The split.  The tiles of all (request, kv head, block of rows) items are put
// in one line and cut into as many equal parts as there are CTAs (one per SM);
// the lengths are read on the device, so the launch does not depend on them.
// A CTA's part is whole items and at most two pieces of items; the pieces'
// (O, r, l) go to the workspace, and the last of an item's CTAs to arrive adds
// them up in the CTAs' order.
//
// Warps: 0 tensor copies (one box per page and 64 channels, straight from the
// page table), 1 the first and 2 the second product's tcgen05.mma, 3 the next
// item's queries and masks, then the softmax warps (128 threads per 8 to 32
// rows) and for 4 bits those that unpack.
//
// Measured on one GB300, and what bounds it: bf16, 32 requests of 1-8 drafts
// over 1-32k tokens (32 heads on 8, dim 128): 244 us, 6.68 TB/s, the cache's
// bytes.  2 x 4096-token prompt chunks in a window of 1024: 313 us, 412
// TFLOP/s; 16 trees over 2-12k tokens, dim 64: 85 us; both by the chain of one
// tile's softmax, 2900 clocks for 128 x 128 weights (the powers alone take
// 1024), in which all softmax warps are in one phase.  4 bits, 32 x 1 token over
// 8-64k: 365 us, 3.43 TB/s, 1390 clocks a tile, the unpacking's and the waits'
// latency; 48 x 1-8 drafts, 64 rows, of which 44 % are without a query: 325 us,
// instruction issue (54 % of the slots).  One token of one request: 12 us, all
// latency.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "ss.h"
#include "ss_cache.h"
#include "ss_ptx.cuh"

namespace ssa {
using namespace ss;

constexpr int kTile = 128;                // keys per tile
constexpr int kMaxCtas = 256;             // the workspace's limit on the grid
constexpr int kMaxDevices = 64;
constexpr uint32_t kPolls = 1u << 14;     // bounded waits: polls that each sleep up to kSleepNs, 60 ms in all
constexpr uint32_t kSleepNs = 50000;
constexpr int kInfo = 16;                 // tiles whose page masks are kept
constexpr int kPairs = 8;                 // tiles whose (s, m) pairs are kept
constexpr float kUnset = 3.0e38f;         // in a piece: minus the reference of a row that has seen nothing
// How far a score (log2) may pass its row's reference, and for bf16 how far the
// first ones may lie below the reference 0: as little as costs nothing (8 and 16:
// prompt 311 -> 324 us, trees 85 -> 92; 32 and 64 no faster).  4 bits: of the
// score plus its key's magnitude, so that f16 holds the weights (65504 at most,
// 2^-24 their unit); there a reference that is set or moved puts the largest
// weight at 2^kTop (48 x 1-8 drafts 338 -> 322 us against references that
// start at 0, which also lost small weights beside a large one): from its
// first key on a row's largest weight is in [2^8, 2^15].  Beside one sink 2^20
// other keys that count as much together then stand at 2^-12 or above, where f16
// still has all its bits (down to 2^-14); and 7 binades, 4.9 of a score, are left
// before the next move.
template <bool kPacked> constexpr float kSlack = kPacked ? 15.0f : 16.0f;
constexpr float kDeep = 32.0f;
constexpr float kTop = 8.0f;
constexpr int kSlotFloats = 128 * 130;    // one piece: up to 128 rows of 128 channels, r and l

struct AttnArgs {
  CacheView c;
  TableView t;
  int32_t num_requests, num_heads, group, max_queries, total_queries;
  uint32_t group_mul, group_shift;  // n / group = (n * group_mul >> 32) >> group_shift, n < 2^31
  int32_t block_rows;  // rows of an item (the kernel's kLive)
  int32_t table_end;   // slots of a table row, at most 2^31 - 1
  int32_t few_tiles;   // the requests' tiles for one head stay below 2^31, whatever the lengths
  int32_t most_tiles;  // that a call may have for one head
  const int32_t* offsets;
  const int32_t* kv_len;
  const int32_t* parents;
  const uint8_t* q;
  int64_t q_token, q_head;  // bytes
  uint16_t* out;
  int64_t out_token, out_head;  // elements
  float* lse;
  float scale_log2;
  int32_t window, sinks;
  int32_t stall;  // 0, or the barriers that the self-test stalls (SS_STALL_*)
  int32_t* status;
  int32_t* counters;  // [kMaxCtas], zero between calls
  int32_t* gave_up;   // 0 until a CTA gives up on a wait
  float* pieces;      // [kMaxCtas][2][kSlotFloats]
};

ss_status launch_bf16(const AttnArgs& a, cudaStream_t s);
ss_status launch_int4(const AttnArgs& a, cudaStream_t s);

// Rank-4 tensor map (channel bytes, slot, head, page) of K or V.
bool make_cache_map(CUtensorMap* m, void* base, const CacheView& c, int box_slots);

// Rank-3 tensor map (channels, head, token) of the queries: boxes of a block's
// tokens times a group's heads where blocks of `rows` rows start at tokens,
// else of one row.
bool make_query_map(CUtensorMap* m, const AttnArgs& a, int rows);

#ifdef __CUDACC__

// One work item of a CTA: consecutive tiles of one (request, kv head, block).
// A request's rows are its tokens times the heads of a group, token major.
struct Item {
  int32_t r, head, row0, rows;    // block of rows row0 .. row0 + rows - 1
  int32_t tiles, tile0, all;      // this CTA's tiles, the first one's number, the item's total
  int32_t nsink, sink_end;        // tiles of the first tokens, their keys end here
  int32_t origin, end;            // keys of the other tiles
  int32_t base, qbegin;
  int32_t cta0, cta1, piece;      // the CTAs that share the item; this CTA's piece
  int32_t pad;
  const int32_t* row;
};

// kLive: rows of an item; kN: rows of the second product's MMAs (16 at least);
// kNS: columns of the first product (4 bits: two per row).
template <int kLive, bool kPacked, int kHalves>
struct Cfg {
  static constexpr int kN = kLive < 16 ? 16 : kLive;
  static constexpr int kNS = kPacked ? 2 * kLive : kN;
  static constexpr int kGroups = kLive <= 16 ? 1 : kLive == 32 ? 2 : kPacked ? 2 : 4;  // softmax warpgroups
  static constexpr int kCols = kLive / kGroups;              // rows per softmax thread
  // 4 bits, few rows: two warpgroups take turns at the tiles, each with a sum
  // and an accumulator of its own, joined at the item's end.  What a tile asks
  // of one is mostly latency then (1300 clocks, where copying it takes 750).
  static constexpr int kStreams = kPacked && kLive <= 16 ? 2 : 1;
  static constexpr int kSoft = 128 * kGroups * kStreams;
  static constexpr int kPerTile = kSoft / kStreams;          // softmax threads of one tile
  // 4 bits: one warpgroup unpacks K; V, twice the work, has two that take turns
  // where the softmax leaves the registers
  static constexpr int kVGroups = kLive <= 16 ? 2 : 1;
  static constexpr int kUnpack = kPacked ? 128 * (1 + kVGroups) : 0;
  static constexpr int kThreads = 128 + kSoft + kUnpack;
  // Registers per thread by warpgroup where one size does not fit all: the
  // launch's kThreads x kRegs are shared out again (all or none of them).
  static constexpr int kRegs = kThreads > 640 ? 80 : kThreads > 512 ? 96 : kThreads > 384 ? 128 : 168;
  static constexpr bool kSplit = kPacked || kLive == 128;
  static constexpr int kRegs0 = kStreams == 2 ? 56 : 64;                                   // copies, MMAs, queries
  static constexpr int kRegsSoft = !kPacked || kStreams == 2 ? 104 : kLive >= 64 ? 152 : 136;
  static constexpr int kRegsUnpack = kLive >= 64 ? 56 : 72;
  static_assert(!kSplit || kRegs0 + kSoft / 128 * kRegsSoft + kUnpack / 128 * kRegsUnpack <= kThreads / 128 * kRegs,
                "a warpgroup would wait for registers for ever");
  static constexpr int kStage = kHalves * 16384;             // 128 keys x 64 channels x 2 bytes per half
  static constexpr int kQ = kPacked ? kNS * 128 : kHalves * kN * 128;
  static constexpr int kNQ = 2;                              // items prepared ahead
  static constexpr int kQBufs = kLive >= 128 ? 1 : 2;        // of which with their queries
  static constexpr int kPitch = kN >= 64 ? 128 : kN * 2;     // bytes per key of a P block
  static constexpr int kP = kTile * kN * 2;
  // a second buffer of P where it costs K and V no slot of their ring (128 rows:
  // 16 trees 95 us with one, 108 with two and a ring of three)
  static constexpr int kPBufs = kLive >= 128 ? 1 : 2;
  static constexpr int kRawRow = 32 * kHalves;               // packed bytes per key
  static constexpr int kRaw = kPacked ? 2 * kTile * kRawRow + 2 * kTile * 4 : 0;
  static constexpr int kRawStages = kPacked ? 4 : 1;
  // V's unpacking in a loop where the other warps' code is long: together they
  // are bound by instruction fetch (48 x 1-8 drafts of 64 rows: 353 us, 414
  // unrolled); unrolled with its loads ahead of the wait where it is latency
  // that counts.
  static constexpr int kUnrollV = kLive >= 64 ? 1 : 2 * kHalves;
  static constexpr int kUnrollPV = kLive >= 64 ? 1 : 8;  // likewise (2 x 4096 prompt: 311 us, 318 unrolled)
  // the static arrays, rounded up
  static constexpr int kMeta = kNQ * (static_cast<int>(sizeof(Item)) + kN * 36 + 64 + 512) + kStreams * kN * 36 + 1536 +
                               (kPacked ? 2 * kPairs * kTile * 4 : 0);
  static constexpr int kBudget = 232448 - 1024 - kQBufs * kQ - kPBufs * kP - kRawStages * kRaw - kMeta;
  // K and V have a ring each, so that whoever waits for a slot has used the
  // slot's previous contents itself: a parity wait tells two phases apart, no
  // more.  4 bits: only V's is in shared memory, K's two slots are columns.
  static constexpr int kMost = kPacked ? 4 : 8;
  static constexpr int kRing = kBudget / kStage < kMost ? kBudget / kStage : kMost;
  static constexpr int kKs = kPacked ? 2 : kRing / 2, kVs = kPacked ? kRing : kRing - kKs;
  static constexpr int kSmem = 1024 + kRing * kStage + kQBufs * kQ + kPBufs * kP + kRawStages * kRaw;
  // tensor-memory columns: S x 2, O x 2, and for 4 bits K x 2 (four channels per column)
  static constexpr uint32_t kOCol = 2 * kNS, kKCol = kOCol + 2 * kStreams * kN;
  static constexpr uint32_t kKCols = kPacked ? 16 * kHalves : 0;
  static constexpr uint32_t kUsed = kKCol + 2 * kKCols;
  static constexpr uint32_t kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kKs >= 1 && kVs >= 2, "a tile in use and one on its way");
  static_assert(!kPacked || (kVs % kVGroups == 0 && kRawStages % kVGroups == 0), "a warpgroup's slots are its own");
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// The waits give up after kPolls polls, or at once when another wait of the CTA
// has given up before (*dead).  The caller goes on (single-role warps stop, the
// softmax at its next item); nothing it computes then is used.  What follows
// from a wait's outcome is decided for whole warps, and no barrier depends on
// it.  One block of PTX, small where it is not taken: the code around it is
// bound by instruction fetch.
__device__ __forceinline__ bool wait_more(uint32_t bar, uint32_t parity, int32_t* dead) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n, d;\n\t"
      "mov.u32 n, %4;\n\t"
      "poll:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %5;\n\t"
      "@p bra over;\n\t"
      "ld.volatile.shared.u32 d, [%3];\n\t"
      "setp.ne.u32 q, d, 0;\n\t"
      "@q bra over;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra poll;\n\t"
      "st.volatile.shared.u32 [%3], 1;\n\t"
      "over:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(smem_addr(dead)), "n"(kPolls), "n"(kSleepNs)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_or_dead(uint64_t* bar, uint32_t parity, int32_t* dead) {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  return wait_more(smem_addr(bar), parity, dead);
}

// A wait for the end of an item, which may be long: given up when another wait
// of the CTA has (each of those is for a tile or less, about 60 ms), or after a
// minute.
__device__ __forceinline__ bool wait_item(uint64_t* bar, uint32_t parity, int32_t* dead) {
#pragma unroll 1
  for (uint32_t i = 0; i < 1024 * kPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "n"(kSleepNs)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<volatile int32_t*>(dead) != 0) return false;
  }
  *reinterpret_cast<volatile int32_t*>(dead) = 1;
  return false;
}

// A bounded wait for what the waiter itself has in flight, whether the CTA has
// given up or not: nothing may write into the CTA's memory after its end.
__device__ __forceinline__ bool wait_drained(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "n"(kSleepNs)
        : "memory");
    if (done) return true;
  }
  return false;
}

// Two barriers at once: the polls' latencies overlap.
__device__ __forceinline__ void wait_both(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1,
                                          int32_t* dead) {
  const bool d0 = mbar_try_wait(bar0, parity0), d1 = mbar_try_wait(bar1, parity1);
  if (!d0) wait_or_dead(bar0, parity0, dead);
  if (!d1) wait_or_dead(bar1, parity1, dead);
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t w,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// 16 bytes by the thread's own asynchronous copy (zeros where `there` is
// false), and an arrival on `bar` once the thread's copies so far are done.
__device__ __forceinline__ void async_load16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared-memory matrix descriptor: low word the start address and the leading
// byte offset, high word the stride byte offset, version 1 and the swizzle
// layout (2: 128 bytes, 4: 64, 6: 32).
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) {
  return (sbo >> 4) | (1u << 14) | (layout << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32);
}

// Instruction descriptors: fp32 accumulator, M = 128.  kind::f16 with A and B
// both bf16 or both f16, `mn`: both M-/N-major instead of K-major; kind::f8f6f4
// with e4m3.
template <int kN, bool kF16 = false>
__device__ __forceinline__ constexpr uint32_t instr_desc(bool mn) {
  return (1u << 4) | (kF16 ? 0u : (1u << 7) | (1u << 10)) | (mn ? (3u << 15) : 0u) | (static_cast<uint32_t>(kN >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

template <int kN>
__device__ __forceinline__ constexpr uint32_t instr_desc_e4m3() {
  return (1u << 4) | (static_cast<uint32_t>(kN >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// True in one lane of the warp.  Inside `if (elect_one())` the compiler knows
// that one lane runs and keeps descriptors in uniform registers: 6 instructions
// per MMA, where a test of the lane number takes 14.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// e4m3, A in tensor memory: lane m holds row m, four channels per column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Consecutive fp32 columns of this warp's 32 tensor-memory lanes.
// tmem_get starts the load; tmem_wait ends it.
__device__ __forceinline__ void tmem_get(uint32_t t, float (&v)[16]) {
  __syncwarp();  // the loads and stores of tensor memory are the whole warp's
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_get(uint32_t t, float (&v)[4]) {
  __syncwarp();
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(t)
               : "memory");
}
__device__ __forceinline__ void tmem_get(uint32_t t, float (&v)[8]) {
  __syncwarp();
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t)
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[8]) {
  __syncwarp();
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(t)
               : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_get(uint32_t t, float (&v)[32]) {
  __syncwarp();
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_put(uint32_t t, const float (&v)[16]) {
  __syncwarp();
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[16]) {
  tmem_put(t, v);
  tmem_put_wait();
}
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[32]) {
  __syncwarp();
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(t)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kCount>
__device__ __forceinline__ void tmem_wait(float (&v)[kCount]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kCount; ++i) asm volatile("" : "+f"(v[i]));  // no use of v moves above the wait
}
template <int kCount>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[kCount]) {
  tmem_get(t, v);
  tmem_wait(v);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 values as an f16 pair (a in the low half).
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Two fp32 values as e4m3 (a in the low byte; finite values saturate), and back.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 e4m3_floats(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  float2 f;
  asm("{\n\t.reg .f16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Barrier `id` over `n` threads; the second form also says whether any thread
// brought a true `p`.
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool bar_any(int id, int n, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(p))
      : "memory");
  return any != 0;
}

// Largest value of the warp's lanes that is a number (-infinity if none).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return fmaxf(r, -INFINITY);
}

__device__ __forceinline__ void store_pair(uint16_t* p, uint32_t pair, bool wide) {
  if (wide) {
    *reinterpret_cast<uint32_t*>(p) = pair;
  } else {
    p[0] = static_cast<uint16_t>(pair);
    p[1] = static_cast<uint16_t>(pair >> 16);
  }
}

// Sums of kCount values over the warp's 32 lanes; lane i gets the sum of
// value i % kCount (a butterfly that halves the values at each step).
template <int kCount>
__device__ __forceinline__ float warp_sums(float (&v)[kCount]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= kCount) {
#pragma unroll
      for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const bool up = lane & o;
        const float keep = up ? v[i + o] : v[i];
        const float give = up ? v[i] : v[i + o];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
  }
  return v[0];
}

// Row number to token (division by multiplication, after Granlund and
// Montgomery: the multiplier is floor(2^(31+l) / group) + 1, l = ceil(log2 group)).
__device__ __forceinline__ int32_t token_of(const AttnArgs& a, int32_t row) {
  return a.group == 1 ? row : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(row), a.group_mul) >> a.group_shift);
}

// What the scheduler knows of one request.
struct Request {
  const int32_t* row;
  int32_t qbegin, n, base;
  bool ok;
};

__device__ __forceinline__ Request request_of(const AttnArgs& a, int32_t r) {
  Request q;
  q.qbegin = a.offsets ? a.offsets[r] : r;
  const int32_t end = a.offsets ? a.offsets[r + 1] : r + 1;
  q.base = a.kv_len[r];
  q.row = table_row(a.t, r);
  q.n = end - q.qbegin;
  q.ok = q.row && q.base >= 0 && q.qbegin >= 0 && q.qbegin <= end && end <= a.total_queries && q.n <= a.max_queries &&
         !(a.parents && q.n > SS_TREE_MAX_NODES) && static_cast<int64_t>(q.base) + q.n <= 0x7fffff00ll;
  if (__builtin_expect(!a.few_tiles, 0) && q.ok && q.n > 0) {
    // no fewer than the tiles of one head, which are counted in 31 bits
    const uint32_t all = min(q.base + q.n, a.table_end);
    const uint32_t keys = a.window > 0 ? min(all, a.window + 2u * kTile) + min(static_cast<uint32_t>(a.sinks), all) : all;
    const uint32_t blocks = (static_cast<uint32_t>(q.n * a.group - 1) >> (31 - __clz(a.block_rows))) + 1;
    q.ok = (static_cast<uint64_t>(blocks) * (keys / kTile + 3)) >> 31 == 0;
  }
  if (!q.ok) q.n = 0;
  return q;
}

// The statuses of this CTA's share of the requests: a thread per request, or
// with parents, which are looked at, a warp; from warp 3 on, as the first ones
// have the requests' tiles to count.
//
// A time-out wins over them, whatever the order of the CTAs: a CTA that gives
// up sets the workspace's word, and then exchanges the statuses for the
// time-out.  Either that comes after the exchange here, or what comes back here
// is the time-out, and the word is there to be seen.  (It stays until the
// workspace is zeroed: the joining's counts may be off.)
template <int kThreads>
__device__ __forceinline__ void write_statuses(const AttnArgs& a) {
  const int t = (threadIdx.x + kThreads - 96) % kThreads, lane = t & 31;
  const int64_t first = a.parents ? t >> 5 : t, width = a.parents ? kThreads / 32 : kThreads;
  const volatile int32_t* word = a.gave_up;
#pragma unroll 1
  for (int64_t r = blockIdx.x + first * gridDim.x; r < a.num_requests; r += width * gridDim.x) {
    const int32_t early = *word;  // on its way with the request's numbers
    const Request q = request_of(a, static_cast<int32_t>(r));
    bool bad = !q.ok;
    if (a.parents) {
#pragma unroll 1
      for (int32_t n = 1 + lane; n < q.n; n += 32) {
        const int32_t pa = a.parents[q.qbegin + n];
        bad |= pa < 0 || pa >= n;
      }
      bad = __any_sync(0xffffffffu, bad);
      if (lane != 0) continue;
    }
    const bool beyond = q.n > 0 && ((q.base + q.n - 1) >> a.c.page_shift) >= a.t.max_pages;
    const int32_t before = atomicExch(a.status + r, bad ? SS_ROW_BAD_PARAM : beyond ? SS_ROW_BAD_INDEX : SS_ROW_OK);
    bool gave_up = early != 0;
    if (before == SS_ROW_TIMEOUT) {
      __threadfence();
      gave_up = *word != 0;
    }
    if (gave_up && q.n > 0) atomicExch(a.status + r, SS_ROW_TIMEOUT);
  }
  __syncwarp();
}

// The keys of the block of rows that starts at row0: tiles over the first
// tokens (sinks) and tiles from the window's start on, in units of a page (or
// 128 slots of a larger one).
struct Span {
  int32_t nsink, sink_end, origin, end, tiles;
};

__device__ __forceinline__ Span span_of(const AttnArgs& a, const Request& q, int32_t row0) {
  Span s;
  const int32_t unit = min(1 << a.c.page_shift, kTile);
  const int32_t first = q.base + (a.parents ? 0 : token_of(a, row0));  // the lowest position of the block
  const int32_t low = (a.window > 0 && first >= a.window) ? first - a.window + 1 : 0;
  s.origin = low & ~(unit - 1);
  s.end = q.base + token_of(a, min(row0 + a.block_rows, q.n * a.group) - 1) + 1;
  // slots beyond the table are holes: no tiles for them, but one if nothing else is left
  if (s.end > a.table_end) s.end = max(a.table_end, s.origin + 1);
  s.sink_end = min(min(a.sinks, s.origin), a.table_end);
  s.nsink = (s.sink_end + kTile - 1) / kTile;
  s.tiles = s.nsink + (s.end - s.origin + kTile - 1) / kTile;
  return s;
}

// Sums of tiles end at 2^31 - 1.
__device__ __forceinline__ int32_t add_tiles(int32_t x, int32_t y) {
  return static_cast<int32_t>(min(static_cast<uint32_t>(x) + static_cast<uint32_t>(y), 0x7fffffffu));
}

// Tiles of one kv head of a request; the lanes of a warp share its blocks.
__device__ __forceinline__ int32_t request_tiles(const AttnArgs& a, const Request& q, int32_t block0, int32_t step) {
  int32_t sum = 0;
#pragma unroll 1
  for (int32_t row0 = block0 * a.block_rows; row0 < q.n * a.group; row0 += step * a.block_rows)
    sum += span_of(a, q, row0).tiles;
  return sum;
}

// The queries of an item over a 4-bit cache: row n as unit (hi + lo / 32), both
// e4m3, unit a power of two by the row's largest channel: q's 8 bits are 4 + 4,
// so this is exact but for channels below 2^-15 of the largest.  16 lanes per
// row, 8 channels each; a warp has 2 kEach rows in flight.
template <int kLive, int kEach>
__device__ __forceinline__ void convert_queries(const AttnArgs& a, const Item& it, uint8_t* q, float* qsum, float* unit,
                                                int warp, int warps) {
  const int lane = threadIdx.x & 31, ch = lane & 15;
  const int32_t row0 = it.row0, rows = it.rows, head = it.head, qbegin = it.qbegin;
#pragma unroll 1
  for (int n0 = warp * (2 * kEach) + (lane >> 4); n0 < kLive; n0 += warps * (2 * kEach)) {
    uint4 x[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int n = n0 + 2 * u, token = token_of(a, row0 + n);
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      if (n < rows && ch * 8 < a.c.dim)
        x[u] = *reinterpret_cast<const uint4*>(
            a.q + (static_cast<int64_t>(qbegin) + token) * a.q_token +
            (static_cast<int64_t>(head) * a.group + (row0 + n - token * a.group)) * a.q_head + ch * 16);
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int n = n0 + 2 * u;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float v[8], sum = 0.0f, top = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
        sum += v[2 * i] + v[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool finite = fabsf(v[i]) <= 3.4e38f;
        if (finite) top = fmaxf(top, fabsf(v[i]));
        else v[i] = __int_as_float(0x7fffffff);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o, 16);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, 16));
      }
      // top * scale is in [128, 256)
      const int e = max((__float_as_int(top) >> 23) & 0xff, 16);
      const float scale = __int_as_float((261 - e) << 23);
      uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
      // the unpacked keys' order of eight channels: 0 4 1 5, 2 6 3 7
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = (i & 1) + (i >> 1) * 2;  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
        const float p0 = v[c] * scale, p1 = v[c + 4] * scale;
        const uint32_t h = e4m3_pair(p0, p1);
        const float2 back = e4m3_floats(h);
        const uint32_t r = e4m3_pair((p0 - back.x) * 32.0f, (p1 - back.y) * 32.0f);
        hi[i >> 1] |= h << (16 * (i & 1));
        lo[i >> 1] |= r << (16 * (i & 1));
      }
      uint8_t* at = q + (((ch >> 1) ^ (n & 7)) << 4) + (ch & 1) * 8;  // kLive is a multiple of 8
      *reinterpret_cast<uint2*>(at + n * 128) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(at + (kLive + n) * 128) = make_uint2(lo[0], lo[1]);
      if (ch == 0) {
        qsum[n] = sum;
        unit[n] = __int_as_float((e - 7) << 23);
      }
    }
  }
}

// kAtLaunch: the registers per thread that the warpgroups share out again, or 0
// where they do not.  As a part of the kernel's name it lets the build hold what
// the compiler used against it.
template <int kLive, bool kPacked, int kHalves, int kAtLaunch>
__global__ void __launch_bounds__(Cfg<kLive, kPacked, kHalves>::kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_q, const AttnArgs a) {
  using F = Cfg<kLive, kPacked, kHalves>;
  constexpr int kRing = F::kRing, kKs = F::kKs, kVs = F::kVs, kNQ = F::kNQ, kCols = F::kCols, kN = F::kN, kNS = F::kNS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kfull[kKs], kempty[kKs], vfull[kVs], vempty[kVs], sfull[2], sempty[2], pfull[2], pdone[2], oempty[2],
      mfull[kNQ], qfull[kNQ], qempty[kNQ], qfree[F::kQBufs], rfull[F::kRawStages], rempty[F::kRawStages], written[2], drain[2];
  __shared__ Item items[kNQ];
  __shared__ __align__(16) int32_t row_pos[kNQ][kN];
  __shared__ __align__(16) uint64_t row_path[kNQ][kN];
  __shared__ int64_t row_out[kNQ][kN];
  __shared__ int64_t row_lse[kNQ][kN];
  __shared__ __align__(16) float row_qsum[kPacked ? kNQ : 1][kPacked ? kN : 4], row_unit[kPacked ? kNQ : 1][kPacked ? kN : 4];
  __shared__ uint8_t node_depth[kNQ][SS_TREE_MAX_NODES];
  __shared__ uint64_t node_sees[kNQ][SS_TREE_MAX_NODES];
  __shared__ uint32_t info[kInfo];
  __shared__ uint32_t k_pair[kPacked ? kPairs : 1][kPacked ? kTile : 1], v_pair[kPacked ? kPairs : 1][kPacked ? kTile : 1];
  constexpr int kRows = F::kStreams * kN;  // of the softmax's state
  __shared__ __align__(16) float nref[kRows], corr[kRows], shift[kRows], sums[kRows], csums[kRows];
  __shared__ float part[4][kRows];
  __shared__ uint32_t tmem_slot;
  __shared__ uint8_t v_bad[2][F::kGroups > 1 && !kPacked ? kTile : 1];  // keys whose values are not finite
  __shared__ int32_t s_dead, s_last, s_r0, s_before, s_tiles0, s_scan[32];

  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* pbuf = ring + kRing * F::kStage;
  uint8_t* qbuf = pbuf + F::kPBufs * F::kP;
  uint8_t* vring = ring + (kPacked ? 0 : kKs) * F::kStage;  // after K's slots
  uint8_t* raw = qbuf + F::kQBufs * F::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* dead = &s_dead;

  if (tid == 0) {
    // the self-test of the waits: one kind of barrier expects an arrival more
    const auto more = [&](int kind) { return a.stall == kind ? 1u : 0u; };
    for (int i = 0; i < kKs; ++i) {
      mbar_init(kfull + i, (kPacked ? 128 : 1) + more(SS_STALL_KEYS));
      mbar_init(kempty + i, 1);
    }
    for (int i = 0; i < kVs; ++i) {
      mbar_init(vfull + i, (kPacked ? 128 : 1) + more(SS_STALL_VALUES));
      mbar_init(vempty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1 + more(SS_STALL_SCORES));
      mbar_init(sempty + i, F::kPerTile);
      mbar_init(pfull + i, F::kPerTile + more(SS_STALL_WEIGHTS));
      mbar_init(pdone + i, 1);
      mbar_init(oempty + i, F::kSoft);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(mfull + i, 32 + more(SS_STALL_ITEMS));
      mbar_init(qfull + i, 32 + more(SS_STALL_QUERIES));
      mbar_init(qempty + i, 1 + F::kSoft / 32);
    }
    for (int i = 0; i < F::kQBufs; ++i) mbar_init(qfree + i, 1);
    if (kPacked)
      for (int i = 0; i < F::kRawStages; ++i) {
        mbar_init(rfull + i, 33 + more(SS_STALL_PACKED));  // the copies' bytes, and the lanes' own copies
        mbar_init(rempty + i, 256);
      }
    for (int i = 0; i < 2; ++i) mbar_init(written + i, F::kGroups > 1 ? F::kSoft - 128 : 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    s_dead = 0;
    s_r0 = s_before = 0;
    fence_barrier_init();
  }
  if (F::kGroups > 1 && !kPacked && tid < kTile) v_bad[0][tid] = v_bad[1][tid] = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(F::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  // ---- this CTA's part of the tiles
  // Tiles of each request, in the ring's memory before the ring is used: a
  // thread per request when a request is one block, else a warp.
  int32_t* weights = reinterpret_cast<int32_t*>(ring);
  if (a.max_queries * a.group <= kLive) {
#pragma unroll 1
    for (int32_t r = tid; r < a.num_requests; r += F::kThreads) {
      const Request q = request_of(a, r);
      weights[r] = request_tiles(a, q, 0, 1);
    }
  } else {
#pragma unroll 1
    for (int32_t r = warp; r < a.num_requests; r += F::kThreads / 32) {
      const Request q = request_of(a, r);
      const int32_t w = __reduce_add_sync(0xffffffffu, request_tiles(a, q, lane, 32));
      if (lane == 0) weights[r] = w;
    }
  }
  write_statuses<F::kThreads>(a);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int32_t chunk = (a.num_requests + F::kThreads - 1) / F::kThreads;  // consecutive requests per thread
  const int32_t r_from = min(a.num_requests, tid * chunk), r_to = min(a.num_requests, r_from + chunk);
  int32_t mine = 0;  // the requests' tiles for one head; sums end at 2^31 - 1
#pragma unroll 1
  for (int32_t r = r_from; r < r_to; ++r) mine = add_tiles(mine, weights[r]);
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = add_tiles(upto, y);
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  int32_t all_tiles = 0;
#pragma unroll
  for (int w = 0; w < F::kThreads / 32; ++w) {
    if (w == warp) upto = add_tiles(upto, all_tiles);
    all_tiles = add_tiles(all_tiles, s_scan[w]);
  }
  const bool too_many = all_tiles > a.most_tiles;
  if (too_many) all_tiles = 0;
  const int64_t total = static_cast<int64_t>(all_tiles) * a.c.heads;
  const int32_t ctas = static_cast<int32_t>(min(total, static_cast<int64_t>(gridDim.x)));  // each has a tile or more
  const int64_t lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
  const int32_t my_tiles = static_cast<int32_t>(blockIdx.x) < ctas ? static_cast<int32_t>(hi - lo) : 0;
  if (my_tiles > 0 && mine > 0) {
    const int64_t heads = a.c.heads;
    int32_t before = upto - mine;
    if (lo >= before * heads && lo < upto * heads) {
      int32_t r = r_from;
      while (lo >= (before + weights[r]) * heads) before += weights[r++];
      s_r0 = r;
      s_before = before;
      s_tiles0 = weights[r];
    }
  }
  proxy_fence();  // the weights' reads before the ring's copies
  __syncthreads();
  if (my_tiles == 0) {  // fewer tiles than CTAs, or more than can be walked
    if (too_many)
      for (int64_t r = blockIdx.x + static_cast<int64_t>(tid) * gridDim.x; r < a.num_requests;
           r += static_cast<int64_t>(F::kThreads) * gridDim.x)
        if (request_of(a, static_cast<int32_t>(r)).n > 0) a.status[r] = SS_ROW_LIMIT;
  } else if (warp < 4) {
    if constexpr (F::kSplit) regs_fewer<F::kRegs0>();
    if (warp == 0) {
    // ---------------------------------------------------- tensor copies --
    const int32_t unit_shift = min(a.c.page_shift, 7), units = kTile >> unit_shift;
    const int32_t tiles_all = __shfl_sync(0xffffffffu, my_tiles, 0);
    const uint32_t ring_a = smem_addr(ring);
    const uint32_t vring_a = ring_a + (kPacked ? 0 : kKs) * F::kStage;
    const uint32_t raw_a = ring_a + kRing * F::kStage + F::kPBufs * F::kP + F::kQBufs * F::kQ;
    int32_t at = 0, k = 0;  // tile, item
    bool ok = true;
    int32_t k_tiles = 0, v_tiles = 0;  // issued
    const auto wait = [&](uint64_t* bar, int32_t use) {
      if (ok) ok = __all_sync(0xffffffffu, wait_or_dead(bar, use & 1, dead));
    };
#pragma unroll 1
    while (at < tiles_all && ok) {
      const int b = k % kNQ;
      wait(mfull + b, k / kNQ);
      if (!ok) break;
      const Item& it = items[b];
      const auto same = [](int32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      const int32_t tiles = same(it.tiles), tile0 = same(it.tile0), nsink = same(it.nsink), sink_end = same(it.sink_end);
      const int32_t origin = same(it.origin), end = same(it.end), head = same(it.head);
      const int32_t* row = it.row;
      // 64 entries of the page table from the next tile's on, two per lane,
      // loaded a tile or more before their use: a load per tile, waited for,
      // would take longer than the tile
      const int32_t last = min((end - 1) >> a.c.page_shift, a.t.max_pages - 1);
      const auto entry = [&](int32_t e) { return e <= last ? row[e] : -1; };
      int32_t e0 = (origin + max(tile0 - nsink, 0) * kTile) >> a.c.page_shift;
      int32_t near = entry(e0 + lane), far = entry(e0 + 32 + lane);
#pragma unroll 1
      for (int32_t t = 0; t < tiles && ok; ++t, ++at) {
        const int32_t n = tile0 + t;
        const bool sink = n < nsink;
        const int32_t j0 = sink ? n * kTile : origin + (n - nsink) * kTile;
        const int32_t u = j0 + (lane << unit_shift);
        int32_t page = -1;
        if (sink) {
          if (lane < units && u < sink_end) page = page_of(a.t, a.c, row, u);
        } else {
          if ((j0 >> a.c.page_shift) - e0 >= 32) {
            e0 += 32;
            near = far;
            far = entry(e0 + 32 + lane);
          }
          const int32_t e = (u >> a.c.page_shift) - e0;
          const int32_t p0 = __shfl_sync(0xffffffffu, near, e & 31), p1 = __shfl_sync(0xffffffffu, far, e & 31);
          page = e < 32 ? p0 : p1;
          if (lane >= units || u >= end || page >= a.c.num_pages) page = -1;
        }
        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(info + at % kInfo) = there;
        const auto copies = [&](const CUtensorMap* map, uint32_t dst, uint64_t* bar) {  // of K or V, a lane per page
          if (lane < units) {
            const int32_t slot = u & ((1 << a.c.page_shift) - 1);
            // a page out of range is filled with zeros
#pragma unroll
            for (int h = 0; h < (kPacked ? 1 : kHalves); ++h)
              tma_4d(dst + h * 16384 + (lane << unit_shift) * (kPacked ? F::kRawRow : 128), map, h * 64, slot, head,
                     page < 0 ? a.c.num_pages : page, bar);
          }
        };
        if constexpr (kPacked) {
          const int s = at % F::kRawStages;
          wait(rempty + s, at / F::kRawStages + 1);
          if (!ok) break;
          const uint32_t dst = raw_a + s * F::kRaw;
          if (lane == 0) mbar_arrive_expect_tx(rfull + s, 2 * kTile * F::kRawRow);
          __syncwarp();
          copies(&tm_k, dst, rfull + s);
          copies(&tm_v, dst + kTile * F::kRawRow, rfull + s);
          // the (s, m) pairs, four slots per lane (a bulk copy per page and
          // array is too small to be worth one: 256 bytes for 64 slots)
          const int32_t p = __shfl_sync(0xffffffffu, page, (4 * lane) >> unit_shift);
          const int32_t slot = (j0 + 4 * lane) & ((1 << a.c.page_shift) - 1);
          const int64_t off = max(p, 0) * a.c.s_page_stride + head * a.c.s_head_stride + slot * 4;
          const uint32_t to = dst + 2 * kTile * F::kRawRow + lane * 16;
          async_load16(to, a.c.ks + off, p >= 0);
          async_load16(to + kTile * 4, a.c.vs + off, p >= 0);
          async_arrive(rfull + s);
        } else {
          const int ks = at % kKs, vs = at % kVs;
          wait(kempty + ks, at / kKs + 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(kfull + ks, F::kStage);
          __syncwarp();
          copies(&tm_k, ring_a + ks * F::kStage, kfull + ks);
          ++k_tiles;
          wait(vempty + vs, at / kVs + 1);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(vfull + vs, F::kStage);
          __syncwarp();
          copies(&tm_v, vring_a + vs * F::kStage, vfull + vs);
          ++v_tiles;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty + b);
      ++k;
    }
    // The copies in flight end before this warp does, also where other warps
    // have given up on them (else their users wait for them anyway).
    bool landed = true;
    if (kPacked) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int32_t i = max(0, at - F::kRawStages); i < at && landed; ++i)
        landed = wait_drained(rfull + i % F::kRawStages, (i / F::kRawStages) & 1);
    } else {
      for (int32_t i = max(0, k_tiles - kKs); i < k_tiles && landed; ++i)
        landed = wait_drained(kfull + i % kKs, (i / kKs) & 1);
      for (int32_t i = max(0, v_tiles - kVs); i < v_tiles && landed; ++i)
        landed = wait_drained(vfull + i % kVs, (i / kVs) & 1);
    }
  } else if (warp == 1) {
    // -------------------------------------------- first product, S^T = K Q^T --
    // The whole warp runs the loop on values that are the same in every lane
    // (so that descriptors stay in uniform registers); one lane issues.  An MMA
    // takes 64 clocks for 128 keys or channels however few rows there are, and
    // its warp waits that long to issue the next; the second product has a warp
    // of its own, so that one's waits pass under the other's MMAs.
    constexpr uint32_t kHi = desc_hi(1024, 2);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int32_t tiles_all = __shfl_sync(0xffffffffu, my_tiles, 0);
    const uint32_t ring_a = smem_addr(ring);
    const uint32_t q_a = ring_a + kRing * F::kStage + F::kPBufs * F::kP;
    const int k_steps = kPacked ? (a.c.dim + 31) / 32 : (a.c.dim + 15) / 16;
    bool ok = true;
    const auto wait = [&](uint64_t* bar, int32_t use) {
      if (ok) ok = __all_sync(0xffffffffu, wait_or_dead(bar, use & 1, dead));
    };
    int32_t at = 0;
#pragma unroll 1
    for (int32_t k = 0; at < tiles_all && ok; ++k) {
      const int qb = k % kNQ;
      wait(qfull + qb, k / kNQ);
      if (!ok) break;
      const int32_t tiles = __shfl_sync(0xffffffffu, items[qb].tiles, 0);
      const uint32_t qa = desc_lo(q_a + k % F::kQBufs * F::kQ, 16);
#pragma unroll 1
      for (int32_t t = 0; t < tiles; ++t, ++at) {
        const int b = at & 1;
        const int32_t s = at % kKs;
        wait(kfull + s, at / kKs);
        wait(sempty + b, (at >> 1) + 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if constexpr (kPacked) {
#pragma unroll
            for (int kk = 0; kk < 2 * kHalves; ++kk)
              if (kk < k_steps)
                umma_ts(tm + b * kNS, tm + F::kKCol + s * F::kKCols + kk * 8, desc(qa + kk * 2, kHi), instr_desc_e4m3<kNS>(),
                        kk > 0 ? 1u : 0u);
          } else {
            const uint32_t ka = desc_lo(ring_a + s * F::kStage, 16);
#pragma unroll
            for (int kk = 0; kk < 4 * kHalves; ++kk)
              if (kk < k_steps)
                umma(tm + b * kNS, desc(ka + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2, kHi),
                     desc(qa + (kk >> 2) * (kN * 128 >> 4) + (kk & 3) * 2, kHi), instr_desc<kN>(false), kk > 0 ? 1u : 0u);
          }
          umma_commit(kempty + s);
          umma_commit(sfull + b);
          if (t == tiles - 1) umma_commit(qfree + k % F::kQBufs);  // the queries are read
        }
        __syncwarp();
      }
    }
    // The MMAs in flight end before tensor memory is freed, also where the
    // softmax has given up (the lane that issued them commits).
    if (elect_one()) {
      umma_commit(&drain[0]);
      wait_drained(&drain[0], 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------- second product, O^T += V^T P^T --
    constexpr uint32_t kHiV = desc_hi(1024, 2), kHiP = desc_hi(8 * F::kPitch, kN >= 64 ? 2u : kN == 32 ? 4u : 6u);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int32_t tiles_all = __shfl_sync(0xffffffffu, my_tiles, 0);
    const uint32_t ring_a = smem_addr(ring);
    const uint32_t p_a = ring_a + kRing * F::kStage, v_a = ring_a + (kPacked ? 0 : kKs) * F::kStage;
    bool ok = true;
    const auto wait = [&](uint64_t* bar, int32_t use) {
      if (ok) ok = __all_sync(0xffffffffu, wait_or_dead(bar, use & 1, dead));
    };
    int32_t at = 0;
#pragma unroll 1
    for (int32_t k = 0; at < tiles_all && ok; ++k) {
      const int qb = k % kNQ;
      wait(mfull + qb, k / kNQ);
      if (!ok) break;
      const int32_t tiles = __shfl_sync(0xffffffffu, items[qb].tiles, 0);
      wait(oempty + (k & 1), (k >> 1) + 1);
#pragma unroll 1
      for (int32_t t = 0; t < tiles; ++t, ++at) {
        const int b = at & 1;
        const int32_t s = at % kVs;
        wait(vfull + s, at / kVs);
        wait(pfull + b, at >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + F::kOCol + ((k & 1) * F::kStreams + (F::kStreams == 2 ? b : 0)) * kN;
        const uint32_t va = desc_lo(v_a + s * F::kStage, kHalves == 2 ? 16384 : 0);
        const uint32_t pa = desc_lo(p_a + b % F::kPBufs * F::kP, kTile * 128);
        if (elect_one()) {
#pragma unroll F::kUnrollPV
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma(d, desc(va + kk * (16 * 128 >> 4), kHiV), desc(pa + kk * (16 * F::kPitch >> 4), kHiP), instr_desc<kN, kPacked>(true),
                 (t >= F::kStreams || kk > 0) ? 1u : 0u);
          umma_commit(vempty + s);
          umma_commit(pdone + b);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(&drain[1]);
      wait_drained(&drain[1], 0);
    }
    __syncwarp();
  } else if (warp == 3) {
    // --------------------------------------------- the items' queries --
    int32_t r = s_r0, left = my_tiles;
    Request q = request_of(a, r);
    const int64_t before = static_cast<int64_t>(s_before) * a.c.heads;  // tiles before request r
    const int32_t w = s_tiles0;
    int32_t head = static_cast<int32_t>((lo - before) / w);
    int32_t skip = static_cast<int32_t>((lo - before) - static_cast<int64_t>(head) * w);  // tiles of the head passed
    int64_t start = before + static_cast<int64_t>(head) * w;  // the item's first tile
    int32_t row0 = 0;
#pragma unroll 1
    for (;; row0 += 32 * kLive) {  // the block that holds it: 32 blocks at a time
      const int32_t mine_row = row0 + lane * kLive;
      const int32_t n = mine_row < q.n * a.group ? span_of(a, q, mine_row).tiles : 0;
      int32_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, skip < sum);
      const int at = past ? __ffs(past) - 1 : 31;
      const int32_t passed = __shfl_sync(0xffffffffu, past ? sum - n : sum, at);
      skip -= passed;
      start += passed;
      if (past) {
        row0 += at * kLive;
        break;
      }
    }
    Span s = span_of(a, q, row0);
    int32_t q_items = 0;  // whose queries are issued
    int32_t tree_of = -1, node_deep[2];
    uint64_t node_path[2];
#pragma unroll 1
    for (int32_t k = 0; left > 0; ++k) {
      const int b = k % kNQ;
      if (!__all_sync(0xffffffffu, wait_item(qempty + b, ((k / kNQ) & 1) ^ 1u, dead))) break;
      const int32_t rows = min(kLive, q.n * a.group - row0), take = min(left, s.tiles - skip);
      if (lane == 0) {
        Item it;
        it.r = r;
        it.head = head;
        it.row0 = row0;
        it.rows = rows;
        it.tiles = take;
        it.tile0 = skip;
        it.all = s.tiles;
        it.nsink = s.nsink;
        it.sink_end = s.sink_end;
        it.origin = s.origin;
        it.end = s.end;
        it.base = q.base;
        it.qbegin = q.qbegin;
        it.cta0 = static_cast<int32_t>(((start + 1) * ctas - 1) / total);
        it.cta1 = static_cast<int32_t>(((start + s.tiles) * ctas - 1) / total);
        it.piece = (start + skip == lo) ? 0 : 1;
        it.pad = 0;
        it.row = q.row;
        items[b] = it;
      }
      if (a.parents) {
        // the request's tree: lane i walks up from nodes i and i + 32, all at once
        if (tree_of != r) {
          tree_of = r;
          int32_t up[2], pa[2];
          const auto parent_of = [&](int32_t n) {
            const int32_t p = (n > 0 && n < q.n) ? a.parents[q.qbegin + n] : 0;
            return (p < 0 || p >= n) ? 0 : p;
          };
          pa[0] = parent_of(lane);
          pa[1] = parent_of(lane + 32);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            up[h] = lane + 32 * h;
            node_path[h] = 1ull << up[h];
            node_deep[h] = 0;
          }
#pragma unroll 1
          while (__any_sync(0xffffffffu, up[0] > 0 || up[1] > 0)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int32_t p0 = __shfl_sync(0xffffffffu, pa[0], up[h] & 31), p1 = __shfl_sync(0xffffffffu, pa[1], up[h] & 31);
              if (up[h] > 0) {
                up[h] = up[h] < 32 ? p0 : p1;
                node_path[h] |= 1ull << up[h];
                ++node_deep[h];
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          node_depth[b][lane + 32 * h] = static_cast<uint8_t>(node_deep[h]);
          node_sees[b][lane + 32 * h] = node_path[h];
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int n = lane; n < kN; n += 32) {
        const int32_t token = token_of(a, row0 + n), h = head * a.group + (row0 + n - token * a.group);
        const bool live = n < rows;
        // rows without a query: a position past every key, their result is not used
        row_pos[b][n] = live ? q.base + (a.parents ? node_depth[b][token] : token) : 0x7ffffffe;
        if (a.parents) row_path[b][n] = live ? node_sees[b][token] : ~0ull;
        const int64_t t = static_cast<int64_t>(q.qbegin) + token;
        row_out[b][n] = t * a.out_token + h * a.out_head;
        row_lse[b][n] = t * a.num_heads + h;
      }
      mbar_arrive(mfull + b);
      __syncwarp();
      const int qb = k % F::kQBufs;
      if (!__all_sync(0xffffffffu, wait_item(qfree + qb, ((k / F::kQBufs) & 1) ^ 1u, dead))) break;
      if constexpr (!kPacked) {
        // by tensor copies: the block's tokens times the group's heads in one
        // box where blocks start at tokens, else row by row
        uint8_t* dst = qbuf + qb * F::kQ;
        const bool boxes = kLive % a.group == 0;
        if (lane == 0) mbar_expect_tx(qfull + b, static_cast<uint32_t>((boxes ? kLive : rows) * 128 * kHalves));
        __syncwarp();
        if (boxes) {
          if (lane < kHalves)
            tma_3d(dst + lane * (kN * 128), &tm_q, lane * 64, head * a.group, q.qbegin + token_of(a, row0), qfull + b);
        } else {
#pragma unroll 1
          for (int n = lane; n < rows; n += 32) {
            const int32_t token = token_of(a, row0 + n), h = head * a.group + (row0 + n - token * a.group);
#pragma unroll
            for (int x = 0; x < kHalves; ++x)
              tma_3d(dst + x * (kN * 128) + n * 128, &tm_q, x * 64, h, q.qbegin + token, qfull + b);
          }
        }
      } else {
        if (k > 0) {
          convert_queries<kLive, 4>(a, items[b], qbuf + qb * F::kQ, row_qsum[b], row_unit[b], 0, 1);
          proxy_fence();
        } else {
          bar_sync(6, F::kSoft + 32);  // the softmax warps have done it
        }
      }
      mbar_arrive(qfull + b);
      q_items = k + 1;
      // the next item
      left -= take;
      if (left == 0) break;
      start += s.tiles;
      skip = 0;
      row0 += kLive;
      if (row0 >= q.n * a.group) {
        row0 = 0;
        if (++head == a.c.heads) {
          head = 0;
          do {
            q = request_of(a, ++r);
          } while (q.n == 0);
        }
      }
      s = span_of(a, q, row0);
    }
    if constexpr (!kPacked) {  // their copies end before this warp does
      bool landed = true;
      for (int32_t i = max(0, q_items - kNQ); i < q_items && landed; ++i) landed = wait_drained(qfull + i % kNQ, (i / kNQ) & 1);
    }
  }
  } else if (!kPacked || warp < 4 + F::kSoft / 32) {
    if constexpr (F::kSplit) regs_more<F::kRegsSoft>();
    // ---------------------------------------------------------- softmax --
    const int st = tid - 128, wg = st >> 7, lt = st & 127, wq = warp & 3;
    const int stream = F::kStreams == 2 ? wg : 0;
    const int c0 = F::kStreams == 2 ? 0 : wg * kCols;             // this warpgroup's rows
    const int h0 = stream * kN + c0;                              // their state
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;  // this warp's tensor-memory lanes
    const int bar = 1 + wg;                                       // its barrier
    const int32_t unit_shift = min(a.c.page_shift, 7);
    const uint32_t every = static_cast<uint32_t>((1ull << (kTile >> unit_shift)) - 1);
    const bool tree = a.parents != nullptr;
    // two channels per store where the rows of out allow it
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 3) == 0 && ((a.out_token | a.out_head) & 1) == 0;
    constexpr uint32_t kSwz = kN >= 64 ? 0x70u : kN == 32 ? 0x30u : 0x10u;  // P's swizzle
    int32_t done = 0;  // tiles of the items before
    uint32_t uses[2] = {0, 0};  // of written
    for (int32_t k = 0; done < my_tiles; ++k) {
      const int b = k % kNQ;
      if constexpr (kPacked)
        if (k == 0) {  // the first item's queries, for which everyone waits, by all of these warps
          constexpr int kWarps = F::kSoft / 32, kEach = kLive >= 8 * kWarps ? 4 : kLive >= 4 * kWarps ? 2 : 1;
          // (given up: there is no item to read; the barrier all the same)
          if (__all_sync(0xffffffffu, wait_or_dead(mfull, 0, dead)))
            convert_queries<kLive, kEach>(a, items[0], qbuf, row_qsum[0], row_unit[0], st >> 5, kWarps);
          proxy_fence();
          bar_sync(6, F::kSoft + 32);
        }
      // The rows' references start at 0: before the barrier, behind which every
      // warp reads them (the last item's readers have passed barriers since).
      if (lt < kCols) nref[h0 + lt] = 0.0f;
      // (4 bits: the rows' sums and units come with the queries)
      const bool in = wait_or_dead((kPacked ? qfull : mfull) + b, (k / kNQ) & 1, dead);
      if (bar_any(5, F::kSoft, !in)) break;  // the same decision for every softmax thread
      const Item it = items[b];
      float l[kCols], cs[kPacked ? kCols : 1];
#pragma unroll
      for (int n = 0; n < kCols; ++n) l[n] = 0.0f;
      if (kPacked)
#pragma unroll
        for (int n = 0; n < kCols; ++n) cs[n] = 0.0f;
      bool unset = true;  // thread i of the warpgroup: row i has seen no key yet
      bool fresh = true;  // some row has not
      const uint32_t o_item = tmem + F::kOCol + (k & 1) * F::kStreams * kN + lanes, o_base = o_item + h0;
      const int32_t first_pos = it.base + (tree ? 0 : token_of(a, it.row0));
      const int32_t last_pos = it.base + token_of(a, it.row0 + it.rows - 1);  // of a tree: at most
      const int32_t first_off = it.row0 - token_of(a, it.row0) * a.group;     // rows of the first token in blocks before
#pragma unroll 1
      for (int32_t t = F::kStreams == 2 ? (done ^ stream) & 1 : 0; t < it.tiles; t += F::kStreams) {
        const int32_t at = done + t;
        const int sb = at & 1;
        const int32_t n = it.tile0 + t;
        const bool sink = n < it.nsink;
        const int32_t j0 = sink ? n * kTile : it.origin + (n - it.nsink) * kTile;
        if (F::kPBufs == 2 && at >= 2)  // and P's buffer is free, V's slot has moved on to this tile
          wait_both(sfull + sb, (at >> 1) & 1, pdone + sb, ((at - 2) >> 1) & 1, dead);
        else
          wait_or_dead(sfull + sb, (at >> 1) & 1, dead);
        tc_fence_after();
        constexpr int kPart = !kPacked ? 8 : kCols < 16 ? kCols : 16;
        float x[kCols], low[kPart];
        tmem_get(tmem + sb * kNS + c0 + lanes, x);
        if constexpr (kPacked) tmem_get(tmem + sb * kNS + kLive + c0 + lanes, low);
        // (Where the wait has given up the copies' warp may write it now: the
        // threads need not agree on it, and nothing that they do together
        // depends on it.)
        const uint32_t there = *reinterpret_cast<volatile uint32_t*>(info + at % kInfo);
        // does some row miss some key of the tile?
        const bool masked = sink || there != every || j0 + kTile - 1 > (tree ? it.base - 1 : first_pos) ||
                            (a.window > 0 && j0 <= last_pos - a.window);
        float ka = a.scale_log2, kb = 0.0f, sv = 0.0f, wv = 0.0f;
        float big = 0.0f;  // log2 of the key's values, rounded up: 0 where it does not matter
        bool poison = false;
        if (kPacked) {  // the tensor cores multiplied n / 512 and n - 8
          const uint32_t kp = k_pair[at % kPairs][lt], vp = v_pair[at % kPairs][lt];
          ka = a.scale_log2 * 512.0f * bf16_lo(kp);
          kb = a.scale_log2 * bf16_hi(kp);
          sv = bf16_lo(vp);
          wv = __fmaf_rn(8.0f, sv, bf16_hi(vp));
          poison = !(fabsf(wv) <= 3.0e38f);  // as below; a step that is not finite makes wv so
          if (poison) sv = wv = 0.0f;
          // at most 2^big are s and |m + 8 s| / 16; 2^-80 stands for a row of zeros
          const float top = fmaxf(sv, fabsf(wv) * 0.0625f);
          big = static_cast<float>(max((__float_as_int(top) >> 23) - 126, -80));
        }
        uint32_t vis = 0xffffffffu;  // the rows that see this thread's key
        int32_t from = 0, node = -1;
        uint32_t span = 0x7fffffffu;
        const auto sees = [&](int c) {
          return static_cast<uint32_t>(row_pos[b][c] - from) <= span && (node < 0 || ((row_path[b][c] >> node) & 1ull) != 0);
        };
        if (masked) {
          const int32_t j = j0 + lt;
          const bool here = ((there >> (lt >> unit_shift)) & 1u) && j < (sink ? it.sink_end : it.end);
          const bool draft = tree && here && j >= it.base;
          const int32_t place = draft ? it.base + node_depth[b][j - it.base] : j;
          // a row at position pos sees the key when 0 <= pos - place <= span
          const bool always = a.window == 0 || place < a.sinks;
          span = always ? 0x7fffffffu : static_cast<uint32_t>(a.window) - 1u;
          from = here ? place : 0x7fffffff;
          if (draft) node = j - it.base;
          vis = 0;
          if (!tree) {
            // the rows are in the order of their positions: a range sees the key
            const int32_t e = place - first_pos;  // in tokens from the block's first
            const int32_t f = always ? kLive : static_cast<int32_t>(min(static_cast<int64_t>(e) + a.window,
                                                                       static_cast<int64_t>(kLive)));
            const int32_t lo_row = min(max(e, 0), kLive) * a.group - first_off - c0;
            const int32_t hi_row = max(f, 0) * a.group - first_off - c0;
            const auto below = [](int32_t n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u; };
            if (here) vis = below(hi_row) & ~below(lo_row);
          } else {
#pragma unroll 1
          for (int i = 0; i < kCols; i += 4) {
            const int4 p4 = *reinterpret_cast<const int4*>(&row_pos[b][c0 + i]);
            vis |= (static_cast<uint32_t>(static_cast<uint32_t>(p4.x - from) <= span) << i) |
                   (static_cast<uint32_t>(static_cast<uint32_t>(p4.y - from) <= span) << (i + 1)) |
                   (static_cast<uint32_t>(static_cast<uint32_t>(p4.z - from) <= span) << (i + 2)) |
                   (static_cast<uint32_t>(static_cast<uint32_t>(p4.w - from) <= span) << (i + 3));
          }
          if (draft) {
            const uint32_t* word = reinterpret_cast<const uint32_t*>(&row_path[b][c0]) + ((j - it.base) >> 5);
            uint32_t on = 0;
#pragma unroll 4
            for (int i = 0; i < kCols; ++i) on |= ((word[2 * i] >> ((j - it.base) & 31)) & 1u) << i;
            vis &= on;
          }
          }
          if (!kPacked) {
            // A value that is not finite must not meet a weight of 0: the row
            // of such a key, where not every query sees it, becomes 0 in
            // shared memory, and the queries that do see it get a weight of NaN.
            // Each warpgroup looks at its part of the channels.
            constexpr int kScan = 8 * kHalves / F::kGroups;
            const int32_t s = at % kVs;
            wait_or_dead(vfull + s, (at / kVs) & 1, dead);
            const bool all = here && !draft && j <= first_pos && (always || j > last_pos - a.window);
            if (!all) {
              uint4* v = reinterpret_cast<uint4*>(vring + s * F::kStage + lt * 128);
              uint32_t acc = 0;  // 0 times each channel, added up: NaN as soon as one is not finite
#pragma unroll 4
              for (int c = wg * kScan; c < (wg + 1) * kScan; ++c) {
                const uint4 x = v[(c >> 3) * 1024 + ((c & 7) ^ (lt & 7))];
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(y[e]), "r"(0u));
              }
              poison = (acc & 0x7fff7fffu) != 0;
              if (F::kGroups > 1 && poison) v_bad[sb][lt] = 1;
            }
          }
        }
        // x_nj - r_n of this key, every row
        tmem_wait(x);
        if constexpr (kPacked) {
#pragma unroll
          for (int i0 = 0; i0 < kCols; i0 += kPart) {
            if (i0 > 0) tmem_get(tmem + sb * kNS + kLive + c0 + i0 + lanes, low);
            tmem_wait(low);
#pragma unroll
            for (int i = 0; i < kPart; i += 2)
              split(fma_2(two(low[i], low[i + 1]), two(0.03125f, 0.03125f), two(x[i0 + i], x[i0 + i + 1])), x[i0 + i], x[i0 + i + 1]);
          }
        }
        tc_fence_before();
        mbar_arrive(sempty + sb);
#pragma unroll
        for (int i = 0; i < kCols; i += 4) {
          const float4 r4 = *reinterpret_cast<const float4*>(nref + h0 + i);
          uint64_t y[2] = {two(r4.x, r4.y), two(r4.z, r4.w)}, z[2] = {two(x[i], x[i + 1]), two(x[i + 2], x[i + 3])};
          if (kPacked) {
            const float4 q4 = *reinterpret_cast<const float4*>(&row_qsum[b][c0 + i]);
            const float4 u4 = *reinterpret_cast<const float4*>(&row_unit[b][c0 + i]);
            y[0] = fma_2(two(kb, kb), two(q4.x, q4.y), y[0]);
            y[1] = fma_2(two(kb, kb), two(q4.z, q4.w), y[1]);
            z[0] = mul_2(z[0], two(u4.x, u4.y));
            z[1] = mul_2(z[1], two(u4.z, u4.w));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) split(fma_2(z[e], two(ka, ka), y[e]), x[i + 2 * e], x[i + 2 * e + 1]);
        }
        float least = INFINITY;
        if (!kPacked && fresh)
#pragma unroll
          for (int i = 0; i < kCols; ++i) least = fminf(least, ((vis >> i) & 1u) ? x[i] : INFINITY);
        if (masked)
#pragma unroll
          for (int i = 0; i < kCols; ++i) x[i] = ((vis >> i) & 1u) ? x[i] : -INFINITY;
        float most[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < kCols; ++i) most[i & 3] = fmaxf(most[i & 3], x[i]);
        bool pass = bar_any(bar, 128, fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) + big > kSlack<kPacked> ||
                                      (!kPacked && fresh && least < -kDeep));
        if (kPacked) pass |= fresh;  // a row's first keys set its reference
        if (!kPacked && fresh && !pass) {
          // the rows that see a key here may keep the reference 0 (whatever
          // the tile's mask, the barriers are the same: after a wait that gave
          // up the warps need not agree on it)
          const uint32_t any = __reduce_or_sync(0xffffffffu, vis);
          if (lane == 0) part[wq][h0] = __uint_as_float(any);
          bar_sync(bar, 128);
          const uint32_t seen = (__float_as_uint(part[0][h0]) | __float_as_uint(part[1][h0])) |
                                (__float_as_uint(part[2][h0]) | __float_as_uint(part[3][h0]));
          unset = unset && ((seen >> (lt & 31)) & 1u) == 0;
          fresh = bar_any(bar, 128, lt < kCols && c0 + lt < it.rows && unset);
        }
        if (pass) {
          // some row's score passes its reference by too much (or the row has
          // no reference yet; bf16: and its scores are far below 0): the new
          // reference is the row's largest score of the tile (4 bits: kTop below)
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            const float m = warp_max(x[i] + big);  // a NaN counts as nothing
            if (lane == i) part[wq][h0 + i] = m;
          }
          bar_sync(bar, 128);
          if (lt < kCols) {
            const int c = h0 + lt;
            const float m = fmaxf(fmaxf(part[0][c], part[1][c]), fmaxf(part[2][c], part[3][c]));
            // by the row's own scores alone, so that what other rows see changes no bit of it
            const bool move = m > kSlack<kPacked> || (unset && m > -INFINITY && (kPacked || m < -kDeep));
            const float by = kPacked ? m - kTop : m;
            corr[c] = !move ? 1.0f : unset ? 0.0f : ex2(-by);  // 2^(old reference - new)
            shift[c] = move ? by : 0.0f;
            if (move) nref[c] -= by;
            unset = unset && !(m > -INFINITY);
          }
          // is there a row left that has seen nothing?
          fresh = bar_any(bar, 128, lt < kCols && c0 + lt < it.rows && unset);
          bool change = false;
#pragma unroll
          for (int i = 0; i < kCols; ++i) {
            const float g = corr[h0 + i];
            change |= g != 1.0f;
            l[i] *= g;
            if (kPacked) cs[i] *= g;
            x[i] -= shift[h0 + i];
          }
          if (change && t >= F::kStreams) {
            // the accumulator's last tile (of two streams: waited for above)
            if (F::kStreams == 1) wait_or_dead(pdone + ((at - 1) & 1), ((at - 1) >> 1) & 1, dead);
            tc_fence_after();
#pragma unroll 1
            for (int i0 = 0; i0 < kCols; i0 += 8) {
              float o[8];
              tmem_ld(o_base + i0, o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= corr[h0 + i0 + i];
              tmem_st(o_base + i0, o);
            }
          }
        }
        if (F::kPBufs == 1 && at >= 1) wait_or_dead(pdone + ((at - 1) & 1), ((at - 1) >> 1) & 1, dead);  // P's buffer is free
        // powers, sums, and P^T [key][row], swizzled as the MMA reads it
        uint8_t* pb = pbuf + sb % F::kPBufs * F::kP + (c0 >> 6) * (kTile * 128);
#pragma unroll
        for (int i8 = 0; i8 < kCols / 8; ++i8) {
          uint32_t o4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i8 * 8 + e * 2;
            float p[2] = {ex2(x[i]), ex2(x[i + 1])};
            const uint64_t p2 = two(p[0], p[1]);
            split(add_2(two(l[i], l[i + 1]), p2), l[i], l[i + 1]);
            if constexpr (kPacked) {
              split(fma_2(p2, two(wv, wv), two(cs[i], cs[i + 1])), cs[i], cs[i + 1]);
              split(mul_2(p2, two(sv, sv)), p[0], p[1]);
            }
            o4[e] = kPacked ? f16_pair(p[0], p[1]) : bf16_pair(p[0], p[1]);
          }
          const uint32_t off = lt * F::kPitch + ((c0 & 63) + i8 * 8) * 2;
          *reinterpret_cast<uint4*>(pb + (off ^ ((off >> 3) & kSwz))) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
        }
        if (!kPacked && F::kGroups > 1 && masked) {
          // warpgroup 0 hears what the others found, and writes into their
          // weights once they are there
          poison = false;
          if (wg != 0) {
            mbar_arrive(&written[sb]);
          } else {
            wait_or_dead(&written[sb], uses[sb] & 1, dead);
            poison = v_bad[sb][lt] != 0;
          }
          uses[sb] += 1;
        }
        if (poison) {
          if (!kPacked) {
            if (F::kGroups > 1) v_bad[sb][lt] = 0;
            uint4* v = reinterpret_cast<uint4*>(vring + at % kVs * F::kStage + lt * 128);
#pragma unroll 1
            for (int c = 0; c < 8 * kHalves; ++c) v[(c >> 3) * 1024 + (c & 7)] = make_uint4(0u, 0u, 0u, 0u);
          }
          const int from = kPacked ? c0 : 0, upto = kPacked ? c0 + kCols : kLive;
#pragma unroll 1
          for (int c = from; c < upto; ++c) {
            const bool see = kPacked ? ((vis >> (c - c0)) & 1u) != 0 : sees(c);
            const uint32_t off = lt * F::kPitch + (c & 63) * 2;
            uint8_t* p = pbuf + sb % F::kPBufs * F::kP + (c >> 6) * (kTile * 128);
            if (see) *reinterpret_cast<uint16_t*>(p + (off ^ ((off >> 3) & kSwz))) = 0x7fffu;
          }
        }
        proxy_fence();
        tc_fence_before();
        mbar_arrive(pfull + sb);
      }
      // ---- the item's end: sums over the keys, then the rows
      done += it.tiles;
      const int32_t mine = F::kStreams == 2 ? done - 1 - ((done - 1 - stream) & 1) : done - 1;  // this stream's last tile
      const bool any = mine >= done - it.tiles;
      if (any) wait_or_dead(pdone + (mine & 1), (mine >> 1) & 1, dead);
      tc_fence_after();
      const auto over_keys = [&](auto& v) {  // thread i: the sum of row i over the warpgroup's keys
        const float w = warp_sums<kCols>(v);
        if (lane < kCols) part[wq][h0 + lane] = w;
        bar_sync(bar, 128);
        return lt < kCols ? (part[0][h0 + lt] + part[1][h0 + lt]) + (part[2][h0 + lt] + part[3][h0 + lt]) : 0.0f;
      };
      float sum = over_keys(l), csum = 0.0f;
      if constexpr (kPacked) {
        bar_sync(bar, 128);
        csum = over_keys(cs);
      }
      const int32_t rows = it.rows;            // live rows
      const int ch = wq * 32 + lane;           // this lane's channel
      const bool whole = it.tiles == it.all;
      float* piece = a.pieces + (static_cast<int64_t>(blockIdx.x) * 2 + it.piece) * kSlotFloats;
      if constexpr (F::kStreams == 1) {
        if (lt < kCols) {
          sums[c0 + lt] = !whole ? 1.0f : sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
          csums[c0 + lt] = csum * sums[c0 + lt];
        }
        bar_sync(bar, 128);
      } else {
        // both streams' sums at the larger reference; a stream that saw nothing
        // of a row has sum 0 there (or NaN from a NaN score, which stays)
        if (lt < kCols) {
          part[0][h0 + lt] = unset ? kUnset : nref[h0 + lt];
          part[1][h0 + lt] = sum;
          part[2][h0 + lt] = csum;
        }
        tc_fence_before();  // each warpgroup reads both accumulators
        bar_sync(5, F::kSoft);
        tc_fence_after();
        if (st < kCols) {
          const float n0 = part[0][st], n1 = part[0][kN + st], s0 = part[1][st], s1 = part[1][kN + st];
          const float top = fminf(n0, n1);
          const float g0 = n0 == kUnset ? (s0 == 0.0f ? 0.0f : 1.0f) : ex2(top - n0);
          const float g1 = n1 == kUnset ? (s1 == 0.0f ? 0.0f : 1.0f) : ex2(top - n1);
          sum = __fmaf_rn(g0, s0, g1 * s1);
          const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
          nref[st] = top;
          sums[st] = g0 * inv;
          sums[kN + st] = g1 * inv;
          csums[st] = __fmaf_rn(g0, part[2][st], g1 * part[2][kN + st]) * inv;
          unset = top == kUnset;
        }
        bar_sync(5, F::kSoft);
      }
      // this warpgroup's rows of the result, scaled
      constexpr int kOut = kCols / F::kStreams;
      const int r0 = F::kStreams == 2 ? wg * kOut : c0;
      if (wq * 32 < kHalves * 64 && r0 < rows) {
        // eight rows at a time, in a loop: the code is fetched once per item
        constexpr int kStep = kOut < 8 ? kOut : 8;
#pragma unroll 1
        for (int i0 = r0; i0 < min(r0 + kOut, rows); i0 += kStep) {
          float o[kStep];
          tmem_ld(o_item + i0, o);
#pragma unroll
          for (int i = 0; i < kStep; ++i) o[i] = F::kStreams == 2 && sums[i0 + i] == 0.0f ? 0.0f : o[i] * sums[i0 + i];
          if constexpr (F::kStreams == 2) {
            float o1[kStep];
            tmem_ld(o_item + kN + i0, o1);
#pragma unroll
            for (int i = 0; i < kStep; ++i)
              if (sums[kN + i0 + i] != 0.0f) o[i] = __fmaf_rn(o1[i], sums[kN + i0 + i], o[i]);
          }
          if (kPacked)
#pragma unroll
            for (int i = 0; i < kStep; ++i) o[i] += csums[i0 + i];
          if (whole) {
            // even lanes take two channels of the even row, odd lanes of the odd one
            const bool odd = lane & 1;
            const bool in = (ch & ~1) < a.c.dim;
#pragma unroll
            for (int i = 0; i < kStep; i += 2) {
              const int c = i0 + i + odd;
              const float other = __shfl_xor_sync(0xffffffffu, odd ? o[i] : o[i + 1], 1);
              const uint32_t pair = odd ? bf16_pair(other, o[i + 1]) : bf16_pair(o[i], other);
              if (c < rows && in) store_pair(a.out + row_out[b][c] + (ch & ~1), pair, wide);
            }
          } else {
#pragma unroll
            for (int i = 0; i < kStep; ++i)
              if (i0 + i < rows) __stcg(piece + (i0 + i) * 128 + ch, o[i]);
          }
        }
      }
      if (stream == 0 && lt < kCols && c0 + lt < rows) {
        const int c = c0 + lt;
        if (!whole) {
          __stcg(piece + 128 * 128 + 2 * c, unset ? kUnset : nref[c]);
          __stcg(piece + 128 * 128 + 2 * c + 1, sum);
        } else if (a.lse) {
          a.lse[row_lse[b][c]] = sum == 0.0f ? -INFINITY : 0.69314718055994531f * (log2f(sum) - nref[c]);
        }
      }
      tc_fence_before();
      mbar_arrive(oempty + (k & 1));
      if (!whole) {
        __threadfence();
        bar_sync(5, F::kSoft);
        const int32_t parts = it.cta1 - it.cta0 + 1;
        if (st == 0) {
          const int32_t before = atomicAdd(a.counters + it.cta0, 1);
          s_last = before == parts - 1;
          if (s_last) a.counters[it.cta0] = 0;
        }
        bar_sync(5, F::kSoft);
        if (s_last) {
          // ---- the last CTA of the item joins the pieces, in the CTAs' order:
          // piece p is CTA cta0 + p's first, but for the first CTA, whose
          // second piece it is unless the item starts where the CTA starts
          __threadfence();
          const int64_t item_start = (it.piece == 0 ? lo : hi - it.tiles) - it.tile0;
          const int32_t first_piece = item_start == total * it.cta0 / ctas ? 0 : 1;
          const float* base = a.pieces + static_cast<int64_t>(it.cta0) * 2 * kSlotFloats;
          const auto piece_at = [&](int32_t p) {
            return base + (static_cast<int64_t>(p) * 2 + (p == 0 ? first_piece : 0)) * kSlotFloats;
          };
          // a warp takes kJoin rows at once: what one row costs is the latency
          // of its loads
          constexpr int kWarps = F::kSoft / 32, kJoin = kLive >= 4 * kWarps ? 4 : kLive > kWarps ? 2 : 1;
#pragma unroll 1
          for (int cj = (st >> 5) * kJoin; cj < rows; cj += kWarps * kJoin) {
            float top[kJoin], total_sum[kJoin];
            float4 acc[kJoin];
#pragma unroll
            for (int u = 0; u < kJoin; ++u) {
              top[u] = -INFINITY;  // the largest reference
              total_sum[u] = 0.0f;
              acc[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll 1
            for (int32_t p0 = 0; p0 < parts; p0 += 32) {
              float2 rl[kJoin];  // lane i: piece p0 + i's reference and sum
              float g[kJoin];
              const float* pc = piece_at(min(p0 + lane, parts - 1)) + 128 * 128;
#pragma unroll
              for (int u = 0; u < kJoin; ++u)
                rl[u] = __ldcg(reinterpret_cast<const float2*>(pc + 2 * min(cj + u, rows - 1)));
#pragma unroll
              for (int u = 0; u < kJoin; ++u) {
                const bool set = p0 + lane < parts && rl[u].x != kUnset;
                float m = set ? -rl[u].x : -INFINITY;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                m = fmaxf(m, top[u]);
                if (p0 > 0) {
                  const float f = top[u] == -INFINITY ? 1.0f : ex2(top[u] - m);
                  total_sum[u] *= f;
                  acc[u].x *= f;
                  acc[u].y *= f;
                  acc[u].z *= f;
                  acc[u].w *= f;
                }
                top[u] = m;
                // a piece in which the row saw nothing has sum 0 (or NaN from a NaN score, which stays)
                g[u] = set ? ex2(-rl[u].x - m) : rl[u].y == 0.0f ? 0.0f : 1.0f;
              }
              const int32_t m = min(32, parts - p0);
#pragma unroll 2
              for (int32_t i = 0; i < m; ++i) {
                const float* po = piece_at(p0 + i) + lane * 4;
                float4 v[kJoin];
#pragma unroll
                for (int u = 0; u < kJoin; ++u) v[u] = __ldcg(reinterpret_cast<const float4*>(po + min(cj + u, rows - 1) * 128));
#pragma unroll
                for (int u = 0; u < kJoin; ++u) {
                  const float gi = __shfl_sync(0xffffffffu, g[u], i), li = __shfl_sync(0xffffffffu, rl[u].y, i);
                  total_sum[u] = __fmaf_rn(gi, li, total_sum[u]);
                  if (gi != 0.0f) {
                    acc[u].x = __fmaf_rn(gi, v[u].x, acc[u].x);
                    acc[u].y = __fmaf_rn(gi, v[u].y, acc[u].y);
                    acc[u].z = __fmaf_rn(gi, v[u].z, acc[u].z);
                    acc[u].w = __fmaf_rn(gi, v[u].w, acc[u].w);
                  }
                }
              }
            }
#pragma unroll
            for (int u = 0; u < kJoin; ++u) {
              const int c = cj + u;
              if (c >= rows) break;
              const float inv = total_sum[u] == 0.0f ? 0.0f : __fdividef(1.0f, total_sum[u]);
              if (lane * 4 < a.c.dim) {
                uint16_t* o = a.out + row_out[b][c] + lane * 4;
                store_pair(o, bf16_pair(acc[u].x * inv, acc[u].y * inv), wide);
                store_pair(o + 2, bf16_pair(acc[u].z * inv, acc[u].w * inv), wide);
              }
              if (lane == 0 && a.lse)
                a.lse[row_lse[b][c]] = total_sum[u] == 0.0f ? -INFINITY : 0.69314718055994531f * (log2f(total_sum[u]) + top[u]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty + b);
    }
  } else if constexpr (kPacked) {
    if constexpr (F::kSplit) regs_fewer<F::kRegsUnpack>();
    // --------------------------------------------------------- unpacking --
    // A thread per key; one warpgroup the K tiles, the others the V tiles.
    // A byte n = 0..15 is the e4m3 number n / 512 (0..7 its subnormals, 8..15
    // the first binade), so K only takes its bits apart; it goes to tensor
    // memory (a key's lane is the thread's), which spares shared memory a write
    // and the MMAs a read of the tile.  V becomes n - 8 in f16, whose 11
    // bits for the weights halve the error (references: kSlack), and as an
    // M-major operand it is in shared memory.
    const int key = (tid - 128 - F::kSoft) & 127, turn = ((tid - 128 - F::kSoft) >> 7) - 1;
    const bool is_v = turn >= 0;
#pragma unroll 1
    for (int32_t at = is_v ? turn : 0; at < my_tiles; at += is_v ? F::kVGroups : 1) {
      const int32_t rs = at % F::kRawStages;
      if (!__all_sync(0xffffffffu, wait_or_dead(rfull + rs, (at / F::kRawStages) & 1, dead))) break;
      const uint8_t* src = raw + rs * F::kRaw + (is_v ? kTile * F::kRawRow : 0);
      const uint32_t* pairs = reinterpret_cast<const uint32_t*>(raw + rs * F::kRaw + 2 * kTile * F::kRawRow) + key;
      const auto packed = [&](int c) {  // 16 bytes: 32 channels
        const uint32_t off = key * F::kRawRow + c * 16;
        return *reinterpret_cast<const uint4*>(src + (off ^ ((off >> 3) & (kHalves == 2 ? 0x30u : 0x10u))));
      };
      constexpr bool kAhead = F::kUnrollV > 1;  // the loads before the wait
      uint4 w4[2 * kHalves];
      if constexpr (kAhead)
#pragma unroll
        for (int c = 0; c < 2 * kHalves; ++c) w4[c] = packed(c);
      if (is_v) {
        const int32_t s = at % kVs;
        if (!__all_sync(0xffffffffu, wait_or_dead(vempty + s, ((at / kVs) & 1) ^ 1u, dead))) break;
        uint8_t* dst = vring + s * F::kStage + key * 128;
#pragma unroll F::kUnrollV
        for (int c = 0; c < 2 * kHalves; ++c) {
          const uint4 x4 = kAhead ? w4[c] : packed(c);
          const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // 1024 + n in f16 is 0x6400 | n; minus 1032 leaves n - 8 exactly
              uint32_t y;  // (w >> 4 i) & 0x000f000f | 0x64006400 in one instruction after the shift
              asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(w[e] >> (4 * i)), "r"(0x000f000fu), "r"(0x64006400u));
              asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(y), "r"(0x64086408u));
            }
            const int x = c * 4 + e;  // 8 channels
            *reinterpret_cast<uint4*>(dst + (x >> 3) * 16384 + (((x & 7) ^ (key & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        proxy_fence();
        mbar_arrive(vfull + s);
      } else {
        if (!__all_sync(0xffffffffu, wait_or_dead(kempty + (at & 1), ((at >> 1) & 1) ^ 1u, dead))) break;
        tc_fence_after();
        k_pair[at % kPairs][key] = pairs[0];
        v_pair[at % kPairs][key] = pairs[kTile];
        const uint32_t dst = tmem + F::kKCol + (at & 1) * F::kKCols + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll
        for (int c = 0; c < kHalves; ++c) {
          const uint4 w0 = kAhead ? w4[2 * c] : packed(2 * c), w1 = kAhead ? w4[2 * c + 1] : packed(2 * c + 1);
          const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          float o[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[2 * e] = __uint_as_float(w[e] & 0x0f0f0f0fu);
            o[2 * e + 1] = __uint_as_float((w[e] >> 4) & 0x0f0f0f0fu);
          }
          tmem_put(dst + c * 16, o);
        }
        tmem_put_wait();
        tc_fence_before();
        mbar_arrive(kfull + (at & 1));
      }
      mbar_arrive(rempty + rs);
    }
  }
  __syncthreads();
  // Given up: every request with tiles of this CTA (by a thread of the softmax,
  // whose warps have registers for it).
  if (s_dead && my_tiles > 0 && tid == 128) {
    *reinterpret_cast<volatile int32_t*>(a.gave_up) = 1;
    __threadfence();
    int64_t upto = s_before;  // tiles of one head before and in the requests
#pragma unroll 1
    for (int32_t r = s_r0; r < a.num_requests && upto * a.c.heads < hi; ++r) {
      const Request q = request_of(a, r);
      upto += request_tiles(a, q, 0, 1);
      if (q.n > 0) atomicExch(a.status + r, SS_ROW_TIMEOUT);
    }
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::kTmem) : "memory");
  }
}

template <int kLive, bool kPacked, int kHalves>
ss_status launch(const AttnArgs& a, cudaStream_t s) {
  using F = Cfg<kLive, kPacked, kHalves>;
  const auto kernel = attn_kernel<kLive, kPacked, kHalves, F::kSplit ? F::kRegs : 0>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  CUtensorMap mk, mv, mq{};
  const int unit = 1 << (a.c.page_shift < 7 ? a.c.page_shift : 7);
  if (!make_cache_map(&mk, a.c.k, a.c, unit) || !make_cache_map(&mv, a.c.v, a.c, unit)) return SS_ERR_UNSUPPORTED;
  if (!kPacked && !make_query_map(&mq, a, kLive)) return SS_ERR_UNSUPPORTED;
  // what does not change from call to call, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  static std::atomic<int> grids[kMaxDevices];
  int grid = (e == cudaSuccess && dev < kMaxDevices) ? grids[dev].load(std::memory_order_relaxed) : 0;
  if (e == cudaSuccess && grid == 0) {
    cudaFuncAttributes at{};
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, fn);
    if (e != cudaSuccess) return finish(e);
    // the warpgroups' shares of registers are of what the launch brings (a
    // build in which they are not fails: build.py)
    if (F::kSplit && at.numRegs != F::kRegs) return SS_ERR_UNSUPPORTED;
    grid = sms < kMaxCtas ? sms : kMaxCtas;
    if (dev < kMaxDevices) grids[dev].store(grid, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) kernel<<<grid, F::kThreads, F::kSmem, s>>>(mk, mv, mq, a);
  return finish(e);
}

#endif  // __CUDACC__

}  // namespace ssa
