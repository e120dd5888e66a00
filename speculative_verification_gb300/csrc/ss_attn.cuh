// ss_attn.cuh -- attention of a step's new tokens over the paged cache, on the
// tensor cores (ss_attn_bf16.cu and ss_attn_int4.cu instantiate it).
//
// The mathematics.  For a row n (one query of one head) and the keys j it
// sees, x_nj = scale log2(e) q_n.k_j, with a reference r_n (below):
//   p_nj = 2^(x_nj - r_n),  out_n = sum_j p_nj v_j / sum_j p_nj,
//   lse_n = ln 2 (r_n + log2 sum_j p_nj).
// Any r_n gives the same result; it only has to keep the powers in range.  The
// running maximum is the usual choice; here r_n moves only when some x_nj
// passes it by more than 8, so the accumulated sums are rescaled a few times
// per row instead of at every tile and a tile needs no maximum over its keys
// at all (p <= 2^8 stays exact enough in fp32 and bf16 alike, as both are
// relative).
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
// 4 bits.  A row stands for s n + m, n = 0..15.  n - 8 is exact in bf16, so
// the tensor cores multiply the exact integers, and s and m enter in fp32:
//   q.k = s_k (q.(n - 8)) + (m_k + 8 s_k) sum(q)
//   sum_j p v = sum_j (p s_v) (n - 8) + sum_j p (m_v + 8 s_v),
// the first in fp32 on the thread that owns the key, the second by rounding
// p s_v to bf16 instead of p, plus one fp32 sum per row.
//
// Roundings: P (or p s_v) to bf16, the result to bf16; everything else is
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
// page table), 1 tcgen05.mma, 2-3 the next item's queries and masks, then the
// softmax warps (128 threads per 64 rows or fewer) and for 4 bits four warps
// that unpack.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss.h"
#include "ss_cache.h"
#include "ss_ptx.cuh"

namespace ssa {
using namespace ss;

constexpr int kTile = 128;                // keys per tile
constexpr int kMaxCtas = 256;             // the workspace's limit on the grid
constexpr uint32_t kPolls = 1u << 20;     // bounded waits
constexpr int kInfo = 16;                 // tiles whose page masks are kept
constexpr int kPairs = 8;                 // tiles whose (s, m) pairs are kept
constexpr float kUnset = 3.0e38f;         // minus the reference of a row that has seen nothing
constexpr int kSlotFloats = 128 * 130;    // one piece: up to 128 rows of 128 channels, r and l

struct AttnArgs {
  CacheView c;
  TableView t;
  int32_t num_requests, num_heads, group, max_queries, total_queries;
  int32_t block_rows;  // rows of an item (the kernel's kN)
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
  int32_t* status;
  int32_t* counters;  // [kMaxCtas], zero between calls
  float* pieces;      // [kMaxCtas][2][kSlotFloats]
};

ss_status launch_bf16(const AttnArgs& a, cudaStream_t s);
ss_status launch_int4(const AttnArgs& a, cudaStream_t s);

// Rank-4 tensor map (channel bytes, slot, head, page) of K or V.
bool make_cache_map(CUtensorMap* m, void* base, const CacheView& c, int box_slots);

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

template <int kN, bool kPacked, int kHalves>
struct Cfg {
  static constexpr int kGroups = kN >= 64 ? 2 : 1;           // softmax warpgroups
  static constexpr int kCols = kN / kGroups;                 // rows per softmax thread
  static constexpr int kSub = kCols < 32 ? kCols : 32;       // handled at once
  static constexpr int kSoft = 128 * kGroups;
  static constexpr int kUnpack = kPacked ? 128 : 0;
  static constexpr int kThreads = 128 + kSoft + kUnpack;
  static constexpr int kStage = kHalves * 16384;             // 128 keys x 64 channels x 2 bytes per half
  static constexpr int kQ = kHalves * kN * 128;
  static constexpr int kNQ = kN >= 128 || (kPacked && kN >= 64) ? 1 : 2;
  static constexpr int kPitch = kN >= 64 ? 128 : kN * 2;     // bytes per key of a P block
  static constexpr int kP = kTile * kN * 2;
  static constexpr int kRawRow = 32 * kHalves;               // packed bytes per key
  static constexpr int kRaw = kPacked ? 2 * kTile * kRawRow + 2 * kTile * 4 : 0;
  static constexpr int kRawStages = kPacked ? (kN >= 64 ? 3 : 4) : 1;
  static constexpr int kMeta = kNQ * (static_cast<int>(sizeof(Item)) + kN * 16 + 64) + kN * 4 * 11 + 2048 +
                               (kPacked ? 2 * kPairs * kTile * 4 : 0);
  static constexpr int kBudget = 232448 - 1024 - kNQ * kQ - 2 * kP - kRawStages * kRaw - kMeta;
  static constexpr int kRing = kBudget / kStage < 8 ? kBudget / kStage : 8;
  static constexpr int kSmem = 1024 + kRing * kStage + kNQ * kQ + 2 * kP + kRawStages * kRaw;
  static constexpr uint32_t kTmem = 4 * kN;                  // columns: S x 2, O x 2
  static_assert(kRing >= 3, "K, the next K and V are held at once");
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A wait that gives up: after kPolls polls, or at once when another wait of
// the CTA has given up before.  The caller goes on (single-role warps stop);
// nothing it computes then is used.
__device__ __forceinline__ bool wait_or_dead(uint64_t* bar, uint32_t parity, volatile int32_t* dead) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
  }
  *dead = 1;
  return false;
}

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t w,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// Shared-memory matrix descriptor: start, leading and stride byte offsets,
// version 1, swizzle layout (2: 128 bytes, 4: 64, 6: 32).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(layout) << 61);
}

// Instruction descriptor of kind::f16: fp32 accumulator, bf16 A and B, M = 128;
// `mn`: both operands M-/N-major instead of K-major.
template <int kN>
__device__ __forceinline__ constexpr uint32_t instr_desc(bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? (3u << 15) : 0u) | (static_cast<uint32_t>(kN >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
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
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[16]) {
  __syncwarp();  // the loads and stores of tensor memory are the whole warp's
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[32]) {
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
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[16]) {
  __syncwarp();
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// Order-preserving signed integer of a float that is not NaN, and back.
__device__ __forceinline__ int32_t order_int(float f) {
  const int32_t i = __float_as_int(f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

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
  if (!q.ok) q.n = 0;
  return q;
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
  const int32_t first = q.base + (a.parents ? 0 : row0 / a.group);  // the lowest position of the block
  const int32_t low = (a.window > 0 && first >= a.window) ? first - a.window + 1 : 0;
  s.origin = low & ~(unit - 1);
  s.end = q.base + (min(row0 + a.block_rows, q.n * a.group) - 1) / a.group + 1;
  s.sink_end = min(a.sinks, s.origin);
  s.nsink = (s.sink_end + kTile - 1) / kTile;
  s.tiles = s.nsink + (s.end - s.origin + kTile - 1) / kTile;
  return s;
}

__device__ __forceinline__ int32_t request_tiles(const AttnArgs& a, const Request& q) {
  int32_t sum = 0;
  for (int32_t row0 = 0; row0 < q.n * a.group; row0 += a.block_rows) sum += span_of(a, q, row0).tiles;
  return sum;
}

template <int kN, bool kPacked, int kHalves>
__global__ void __launch_bounds__(Cfg<kN, kPacked, kHalves>::kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a) {
  using F = Cfg<kN, kPacked, kHalves>;
  constexpr int kRing = F::kRing, kNQ = F::kNQ, kSub = F::kSub, kCols = F::kCols;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kRing], empty[kRing], sfull[2], sempty[2], pfull[2], pdone[2], oempty[2],
      qfull[kNQ], qempty[kNQ], rfull[F::kRawStages], rempty[F::kRawStages], looked, drain;
  __shared__ Item items[kNQ];
  __shared__ int32_t row_pos[kNQ][kN];
  __shared__ uint64_t row_path[kNQ][kN];
  __shared__ float row_qsum[kPacked ? kNQ : 1][kPacked ? kN : 1];
  __shared__ uint8_t node_depth[kNQ][SS_TREE_MAX_NODES];
  __shared__ uint32_t info[kInfo];
  __shared__ uint32_t k_pair[kPacked ? kPairs : 1][kPacked ? kTile : 1], v_pair[kPacked ? kPairs : 1][kPacked ? kTile : 1];
  __shared__ __align__(16) float nref[kN], corr[kN], sums[kN], csums[kN];
  __shared__ float part[4][kN];
  __shared__ uint32_t tmem_slot;
  __shared__ int32_t s_dead, s_last, s_chunk0, s_chunk1, s_scan[32];
  __shared__ int32_t s_before;

  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* pbuf = ring + kRing * F::kStage;
  uint8_t* qbuf = pbuf + 2 * F::kP;
  uint8_t* raw = qbuf + kNQ * F::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int32_t* dead = &s_dead;

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(full + i, kPacked ? 128 : 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(sempty + i, F::kSoft);
      mbar_init(pfull + i, F::kSoft);
      mbar_init(pdone + i, 1);
      mbar_init(oempty + i, F::kSoft);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(qfull + i, 64);
      mbar_init(qempty + i, 1 + F::kSoft / 32);
    }
    if (kPacked)
      for (int i = 0; i < F::kRawStages; ++i) {
        mbar_init(rfull + i, 1);
        mbar_init(rempty + i, 128);
      }
    mbar_init(&looked, F::kSoft);
    mbar_init(&drain, 1);
    s_dead = 0;
    s_chunk0 = s_chunk1 = -1;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                 "r"(F::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  // this CTA's part of the tiles: thread t weighs the requests of its chunk
  const int32_t chunk = (a.num_requests + F::kThreads - 1) / F::kThreads;
  int32_t mine = 0;
  for (int32_t i = 0; i < chunk; ++i) {
    const int32_t r = tid * chunk + i;
    if (r < a.num_requests) {
      const Request q = request_of(a, r);
      mine += request_tiles(a, q);
      if (blockIdx.x == 0) {
        int32_t st = q.ok ? SS_ROW_OK : SS_ROW_BAD_PARAM;
        if (q.ok && q.n > 0 && ((q.base + q.n - 1) >> a.c.page_shift) >= a.t.max_pages) st = SS_ROW_BAD_INDEX;
        if (q.ok && a.parents)
          for (int32_t n = 1; n < q.n; ++n) {
            const int32_t pa = a.parents[q.qbegin + n];
            if (pa < 0 || pa >= n) st = SS_ROW_BAD_PARAM;
          }
        a.status[r] = st;
      }
    }
  }
  int32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  int32_t all_tiles = 0;
  for (int w = 0; w < F::kThreads / 32; ++w) {
    if (w == warp) upto += all_tiles;
    all_tiles += s_scan[w];
  }
  const int64_t total = static_cast<int64_t>(all_tiles) * a.c.heads;
  const int32_t ctas = static_cast<int32_t>(min(total, static_cast<int64_t>(gridDim.x)));  // each has a tile or more
  const int64_t lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
  const int32_t my_tiles = static_cast<int32_t>(blockIdx.x) < ctas ? static_cast<int32_t>(hi - lo) : 0;
  if (my_tiles > 0) {
    const int64_t from = static_cast<int64_t>(upto - mine) * a.c.heads, to = static_cast<int64_t>(upto) * a.c.heads;
    if (lo >= from && lo < to) {
      s_chunk0 = tid;
      s_before = upto - mine;
    }
    if (hi - 1 >= from && hi - 1 < to) s_chunk1 = tid;
  }
  __syncthreads();
  // The ring's order within an item whose first tile is the CTA's tile f and
  // that has m tiles: K0, K1, V0, K2, V1, .., K(m-1), V(m-2), V(m-1), as the
  // MMAs take them.
  const auto k_seq = [](int32_t f, int32_t t) { return 2 * f + (t == 0 ? 0 : 2 * t - 1); };
  const auto v_seq = [](int32_t f, int32_t m, int32_t t) { return 2 * f + (t == m - 1 ? 2 * t + 1 : 2 * t + 2); };

  if (my_tiles == 0) {
    // fewer tiles than CTAs
  } else if (warp == 0) {
    // ---------------------------------------------------- tensor copies --
    const int32_t unit_shift = min(a.c.page_shift, 7), units = kTile >> unit_shift;
    int32_t at = 0, k = 0;  // tile, item
    int32_t page_k = 0, slot_k = 0;
    bool ok = true;
    int32_t last_seq = -1;
    const auto issue = [&](const CUtensorMap* map, int32_t seq, int32_t page, int32_t slot, int32_t head) {
      const int s = seq % kRing;
      if (ok) ok = wait_or_dead(empty + s, ((seq / kRing) & 1) ^ 1u, dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) mbar_arrive_expect_tx(full + s, F::kStage);
      __syncwarp();
      if (lane < units)
        for (int h = 0; h < kHalves; ++h)
          tma_4d(ring + s * F::kStage + h * 16384 + (lane << unit_shift) * 128, map, h * 64, slot, head, page, full + s);
      last_seq = seq;
    };
    while (at < my_tiles && ok) {
      const int b = k % kNQ;
      ok = wait_or_dead(qfull + b, (k / kNQ) & 1, dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Item it = items[b];
      const int32_t f = at;
      for (int32_t t = 0; t < it.tiles && ok; ++t, ++at) {
        const int32_t n = it.tile0 + t;
        const bool sink = n < it.nsink;
        const int32_t u = (sink ? n * kTile : it.origin + (n - it.nsink) * kTile) + (lane << unit_shift);
        int32_t page = -1;
        if (lane < units && u < (sink ? it.sink_end : it.end)) page = page_of(a.t, a.c, it.row, u);
        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
        const int32_t slot = u & ((1 << a.c.page_shift) - 1);
        if (kPacked) {
          const int s = at % F::kRawStages;
          ok = wait_or_dead(rempty + s, ((at / F::kRawStages) & 1) ^ 1u, dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* dst = raw + s * F::kRaw;
          if (lane == 0) {
            *reinterpret_cast<volatile uint32_t*>(info + at % kInfo) = there;
            mbar_arrive_expect_tx(rfull + s, 2 * kTile * F::kRawRow + 2 * __popc(there) * (4 << unit_shift));
          }
          __syncwarp();
          if (lane < units) {
            const int32_t pg = page < 0 ? a.c.num_pages : page;  // out of range: filled with zeros
            tma_4d(dst + (lane << unit_shift) * F::kRawRow, &tm_k, 0, slot, it.head, pg, rfull + s);
            tma_4d(dst + kTile * F::kRawRow + (lane << unit_shift) * F::kRawRow, &tm_v, 0, slot, it.head, pg, rfull + s);
            if (page >= 0) {
              const int64_t off = page * a.c.s_page_stride + it.head * a.c.s_head_stride + slot * 4;
              uint8_t* pair = dst + 2 * kTile * F::kRawRow + (lane << unit_shift) * 4;
              bulk_load(pair, a.c.ks + off, 4u << unit_shift, rfull + s);
              bulk_load(pair + kTile * 4, a.c.vs + off, 4u << unit_shift, rfull + s);
            }
          }
        } else {
          if (lane == 0) *reinterpret_cast<volatile uint32_t*>(info + at % kInfo) = there;
          const int32_t pg = page < 0 ? a.c.num_pages : page;
          issue(&tm_k, k_seq(f, t), pg, slot, it.head);
          if (t > 0) issue(&tm_v, v_seq(f, it.tiles, t - 1), page_k, slot_k, it.head);
          page_k = pg;
          slot_k = slot;
        }
      }
      if (!kPacked && ok) issue(&tm_v, v_seq(f, it.tiles, it.tiles - 1), page_k, slot_k, it.head);
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty + b);
      ++k;
    }
    if (!ok) {
      // given up: wait (bounded) for the copies in flight before leaving
      if (kPacked) {
        for (int32_t i = max(0, at - F::kRawStages); i < at; ++i)
          mbar_wait_bounded(rfull + i % F::kRawStages, (i / F::kRawStages) & 1, 1u << 16);
      } else {
        for (int32_t i = max(0, last_seq - kRing + 1); i <= last_seq; ++i)
          mbar_wait_bounded(full + i % kRing, (i / kRing) & 1, 1u << 16);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMAs --
    if (lane == 0) {
      constexpr uint32_t kIdS = instr_desc<kN>(false), kIdO = instr_desc<kN>(true);
      constexpr uint32_t kPLayout = kN >= 64 ? 2u : kN == 32 ? 4u : 6u;
      const int k_steps = (a.c.dim + 15) / 16;
      bool ok = true;
      const auto second = [&](int32_t i, int32_t seq, bool first, int32_t item) {  // O^T += V^T P^T of tile i
        const int b = i & 1;
        const int32_t s = seq % kRing;
        ok = ok && wait_or_dead(pfull + b, (i >> 1) & 1, dead);
        ok = ok && wait_or_dead(full + s, (seq / kRing) & 1, dead);
        if (first) ok = ok && wait_or_dead(oempty + (item & 1), ((item >> 1) & 1) ^ 1u, dead);
        if (!ok) return;
        tc_fence_after();
        const uint32_t va = smem_addr(ring + s * F::kStage), pa = smem_addr(pbuf + b * F::kP);
        const uint32_t d = tmem + 2 * kN + (item & 1) * kN;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma(d, smem_desc(va + kk * 16 * 128, kHalves == 2 ? 16384 : 0, 1024, 2),
               smem_desc(pa + kk * 16 * F::kPitch, kTile * 128, 8 * F::kPitch, kPLayout), kIdO, (!first || kk > 0) ? 1u : 0u);
        umma_commit(empty + s);
        umma_commit(pdone + b);
      };
      int32_t at = 0, k = 0;
      bool prev_first = false;
      int32_t prev_item = 0, prev_seq = 0;
      while (at < my_tiles && ok) {
        const int qb = k % kNQ;
        if (kNQ == 1 && at > 0) second(at - 1, prev_seq, prev_first, prev_item);  // else the next item's queries cannot come
        ok = ok && wait_or_dead(qfull + qb, (k / kNQ) & 1, dead);
        if (!ok) break;
        const int32_t tiles = items[qb].tiles, f = at;
        const uint32_t qa = smem_addr(qbuf + qb * F::kQ);
        for (int32_t t = 0; t < tiles && ok; ++t, ++at) {
          const int b = at & 1;
          const int32_t seq = k_seq(f, t), s = seq % kRing;
          ok = ok && wait_or_dead(full + s, (seq / kRing) & 1, dead);
          ok = ok && wait_or_dead(sempty + b, ((at >> 1) & 1) ^ 1u, dead);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ka = smem_addr(ring + s * F::kStage);
          for (int kk = 0; kk < k_steps; ++kk)
            umma(tmem + b * kN, smem_desc(ka + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024, 2),
                 smem_desc(qa + (kk >> 2) * (kN * 128) + (kk & 3) * 32, 16, 1024, 2), kIdS, kk > 0 ? 1u : 0u);
          umma_commit(empty + s);
          umma_commit(sfull + b);
          if (at > 0 && !(kNQ == 1 && t == 0)) second(at - 1, prev_seq, prev_first, prev_item);
          prev_seq = v_seq(f, tiles, t);
          prev_first = t == 0;
          prev_item = k;
        }
        ++k;
      }
      if (ok) second(my_tiles - 1, prev_seq, prev_first, prev_item);
      if (!ok) {  // given up: the MMAs in flight end before tensor memory is freed
        umma_commit(&drain);
        mbar_wait_bounded(&drain, 0, 1u << 16);
      }
    }
  } else if (warp < 4) {
    // --------------------------------------------- the items' queries --
    const int lt = tid - 64;
    int32_t r = s_chunk0 * chunk, left = my_tiles;
    Request q = request_of(a, r);
    int32_t w = request_tiles(a, q);
    int64_t before = static_cast<int64_t>(s_before) * a.c.heads;  // tiles before request r
    while (lo >= before + static_cast<int64_t>(w) * a.c.heads) {
      before += static_cast<int64_t>(w) * a.c.heads;
      q = request_of(a, ++r);
      w = request_tiles(a, q);
    }
    int32_t head = static_cast<int32_t>((lo - before) / w);
    int32_t skip = static_cast<int32_t>((lo - before) - static_cast<int64_t>(head) * w);  // tiles of the head passed
    int32_t row0 = 0;
    Span s = span_of(a, q, 0);
    int64_t start = before + static_cast<int64_t>(head) * w;  // the item's first tile
    while (skip >= s.tiles) {
      skip -= s.tiles;
      start += s.tiles;
      row0 += kN;
      s = span_of(a, q, row0);
    }
    for (int32_t k = 0; left > 0; ++k) {
      const int b = k % kNQ;
      if (!__all_sync(0xffffffffu, wait_or_dead(qempty + b, ((k / kNQ) & 1) ^ 1u, dead))) break;
      const int32_t rows = min(kN, q.n * a.group - row0), take = min(left, s.tiles - skip);
      if (lt == 0) {
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
      for (int n = lt; n < kN; n += 64) {
        const int32_t token = (row0 + n) / a.group;
        int32_t depth = token;
        uint64_t path = 0;
        if (a.parents && n < rows) {
          depth = 0;
          path = 1ull << token;
          for (int32_t u = token; u > 0; ++depth) {
            const int32_t pa = a.parents[q.qbegin + u];
            u = (pa < 0 || pa >= u) ? 0 : pa;
            path |= 1ull << u;
          }
        }
        // rows without a query: a position past every key, their result is not used
        row_pos[b][n] = n < rows ? q.base + depth : 0x7fffffff;
        row_path[b][n] = n < rows ? path : ~0ull;
      }
      if (a.parents && lt < q.n) {
        int32_t depth = 0;
        for (int32_t u = lt; u > 0; ++depth) {
          const int32_t pa = a.parents[q.qbegin + u];
          u = (pa < 0 || pa >= u) ? 0 : pa;
        }
        node_depth[b][lt] = static_cast<uint8_t>(depth);
      }
      // 16 lanes per row, 8 channels each
      for (int n = lt >> 4; n < kN; n += 4) {
        const int ch = lt & 15, token = (row0 + n) / a.group;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (n < rows && ch * 8 < a.c.dim)
          x = *reinterpret_cast<const uint4*>(
              a.q + (static_cast<int64_t>(q.qbegin) + token) * a.q_token +
              (static_cast<int64_t>(head) * a.group + (row0 + n - token * a.group)) * a.q_head + ch * 16);
        if (ch < 8 * kHalves)
          *reinterpret_cast<uint4*>(qbuf + b * F::kQ + (ch >> 3) * (kN * 128) + n * 128 + (((ch & 7) ^ (n & 7)) << 4)) = x;
        if (kPacked) {
          float sum = ((bf16_lo(x.x) + bf16_hi(x.x)) + (bf16_lo(x.y) + bf16_hi(x.y))) +
                      ((bf16_lo(x.z) + bf16_hi(x.z)) + (bf16_lo(x.w) + bf16_hi(x.w)));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, 16);
          if (ch == 0) row_qsum[b][n] = sum;
        }
      }
      proxy_fence();
      mbar_arrive(qfull + b);
      // the next item
      left -= take;
      if (left == 0) break;
      start += s.tiles;
      skip = 0;
      row0 += kN;
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
  } else if (!kPacked || tid < 128 + F::kSoft) {
    // ---------------------------------------------------------- softmax --
    const int st = tid - 128, wg = st >> 7, lt = st & 127, wq = warp & 3;
    const int col0 = wg * kCols;                            // this warpgroup's rows
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;  // this warp's tensor-memory lanes
    const int bar = 1 + wg;                                 // its barrier
    int32_t at = 0;
    uint32_t looks = 0;
    for (int32_t k = 0; at < my_tiles; ++k) {
      const int b = k % kNQ;
      const bool in = wait_or_dead(qfull + b, (k / kNQ) & 1, dead);
      if (bar_any(5, F::kSoft, !in)) break;  // the same decision for every softmax thread
      const Item it = items[b];
      float l[kCols], cs[kPacked ? kCols : 1];
#pragma unroll
      for (int n = 0; n < kCols; ++n) l[n] = 0.0f;
      if (kPacked)
#pragma unroll
        for (int n = 0; n < kCols; ++n) cs[n] = 0.0f;
      if (lt < kCols) nref[col0 + lt] = kUnset;
      const uint32_t o_base = tmem + 2 * kN + (k & 1) * kN + col0 + lanes;
      const bool tree = a.parents != nullptr;
      const int32_t f = at;
      const int32_t first_pos = it.base + (tree ? 0 : it.row0 / a.group);
      const int32_t last_pos = it.base + (it.row0 + it.rows - 1) / a.group;  // of a tree: at most
      for (int32_t t = 0; t < it.tiles; ++t, ++at) {
        const int sb = at & 1;
        const int32_t n = it.tile0 + t;
        const bool sink = n < it.nsink;
        const int32_t j0 = sink ? n * kTile : it.origin + (n - it.nsink) * kTile;
        wait_or_dead(sfull + sb, (at >> 1) & 1, dead);
        tc_fence_after();
        const uint32_t there = *reinterpret_cast<volatile uint32_t*>(info + at % kInfo);
        const int32_t unit_shift = min(a.c.page_shift, 7);
        const uint32_t every = (kTile >> unit_shift) == 16 ? 0xffffu : (1u << (kTile >> unit_shift)) - 1u;
        // does some row miss some key of the tile?
        const bool masked = sink || there != every || j0 + kTile - 1 > (tree ? it.base - 1 : first_pos) ||
                            (a.window > 0 && j0 <= last_pos - a.window);
        float ka = a.scale_log2, kb = 0.0f, sv = 0.0f, wv = 0.0f;
        if (kPacked) {
          const uint32_t kp = k_pair[at % kPairs][lt];
          const float s = bf16_lo(kp);
          ka = a.scale_log2 * s;
          kb = a.scale_log2 * __fmaf_rn(8.0f, s, bf16_hi(kp));
        }
        bool seen_key = true, poison = false;
        int32_t j = 0, place = 0;
        if (masked) {
          j = j0 + lt;
          place = j;
          seen_key = ((there >> (lt >> unit_shift)) & 1u) && j < (sink ? it.sink_end : it.end);
          if (tree && seen_key && j >= it.base) place = it.base + node_depth[b][j - it.base];
          if (!kPacked) {
            // A value that is not finite must not meet a weight of 0: such a
            // key's row becomes 0, and the rows that see it NaN by its weight.
            const int32_t seq = v_seq(f, it.tiles, t), s = seq % kRing;
            wait_or_dead(full + s, (seq / kRing) & 1, dead);
            uint4* v = reinterpret_cast<uint4*>(ring + s * F::kStage + lt * 128);
            uint32_t bad = 0;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 x = v[h * 1024 + (c ^ (lt & 7))];
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  bad |= ((y[e] & 0x7f80u) == 0x7f80u) | ((y[e] & 0x7f800000u) == 0x7f800000u);
              }
            poison = bad != 0;
            if (F::kGroups > 1) {  // both warpgroups have looked
              mbar_arrive(&looked);
              wait_or_dead(&looked, looks++ & 1, dead);
            }
            if (poison && wg == 0) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int c = 0; c < 8; ++c) v[h * 1024 + c] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
#pragma unroll
        for (int sub = 0; sub < kCols / kSub; ++sub) {
          const int c0 = col0 + sub * kSub;
          float x[kSub];
          tmem_ld(tmem + sb * kN + c0 + lanes, x);
          if (sub == kCols / kSub - 1) {
            tc_fence_before();
            mbar_arrive(sempty + sb);
          }
          float mul = ka;
          if (kPacked) {
            mul = 1.0f;
#pragma unroll
            for (int i = 0; i < kSub; ++i) x[i] = __fmaf_rn(x[i], ka, kb * row_qsum[b][c0 + i]);
          }
          uint32_t vis = 0xffffffffu;
          if (masked) {
            vis = 0;
#pragma unroll 4
            for (int i = 0; i < kSub; ++i) {
              const int32_t pos = row_pos[b][c0 + i];
              bool see = tree && j >= it.base ? seen_key && ((row_path[b][c0 + i] >> (j - it.base)) & 1ull) != 0
                                              : seen_key && j <= pos;
              see = see && (a.window == 0 || place > pos - a.window || place < a.sinks);
              vis |= static_cast<uint32_t>(see) << i;
            }
#pragma unroll
            for (int i = 0; i < kSub; ++i) x[i] = ((vis >> i) & 1u) ? x[i] * mul : -INFINITY;
            mul = 1.0f;
          }
          // does some row's score pass its reference by more than 8?
          bool pass = true;
          if (t > 0) {
            float most = -INFINITY;
#pragma unroll
            for (int i = 0; i < kSub; ++i) most = fmaxf(most, __fmaf_rn(x[i], mul, nref[c0 + i]));
            pass = most > 8.0f;
          }
          if (bar_any(bar, 128, pass)) {
            // new references: the largest score of the tile where it passes
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              const float y = fmaxf(x[i] * mul, -INFINITY);  // a NaN counts as nothing
              const float m = order_float(__reduce_max_sync(0xffffffffu, order_int(y)));
              if (lane == (i & 31)) part[wq][c0 + i] = m;
            }
            bar_sync(bar, 128);
            if (lt < kSub) {
              const int c = c0 + lt;
              const float m = fmaxf(fmaxf(part[0][c], part[1][c]), fmaxf(part[2][c], part[3][c]));
              const float old = nref[c];
              float f = 1.0f;
              if (m + old > 8.0f) {
                nref[c] = -m;
                f = old == kUnset ? 0.0f : ex2(-m - old);  // 2^(old reference - new)
              }
              corr[c] = f;
            }
            bar_sync(bar, 128);
            bool change = false;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
              const float f = corr[c0 + i];
              change |= f != 1.0f;
              l[sub * kSub + i] *= f;
              if (kPacked) cs[sub * kSub + i] *= f;
            }
            if (change && t > 0) {
              wait_or_dead(pdone + ((at - 1) & 1), ((at - 1) >> 1) & 1, dead);
              tc_fence_after();
              float o[kSub];
              tmem_ld(o_base + sub * kSub, o);
#pragma unroll
              for (int i = 0; i < kSub; ++i) o[i] *= corr[c0 + i];
              tmem_st(o_base + sub * kSub, o);
              tc_fence_before();
            }
          }
          if (sub == 0 && at >= 2) wait_or_dead(pdone + sb, ((at - 2) >> 1) & 1, dead);  // P's buffer is free
          if (kPacked && sub == 0) {
            const int32_t seq = v_seq(f, it.tiles, t), s = seq % kRing;
            wait_or_dead(full + s, (seq / kRing) & 1, dead);  // V is unpacked, so its pairs are there
            const uint32_t vp = v_pair[at % kPairs][lt];
            sv = bf16_lo(vp);
            wv = __fmaf_rn(8.0f, sv, bf16_hi(vp));
          }
          // powers, sums, and P^T [key][row], swizzled as the MMA reads it
          uint8_t* pb = pbuf + sb * F::kP + (kN == 128 ? wg * (kTile * 128) : 0);
          const int in_block = (kN == 128 ? 0 : col0) + sub * kSub;
#pragma unroll
          for (int i8 = 0; i8 < kSub / 8; ++i8) {
            uint32_t o4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float p[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int i = i8 * 8 + e * 2 + h, c = sub * kSub + i;
                p[h] = ex2(__fmaf_rn(x[i], mul, nref[c0 + i]));
                if (!kPacked && masked && poison && ((vis >> i) & 1u)) p[h] = __int_as_float(0x7fffffff);
                l[c] += p[h];
                if (kPacked) {
                  if (masked && !((vis >> i) & 1u)) {
                    p[h] = 0.0f;  // the pair may hold anything
                  } else {
                    cs[c] = __fmaf_rn(p[h], wv, cs[c]);
                    p[h] *= sv;
                  }
                }
              }
              o4[e] = bf16_pair(p[0], p[1]);
            }
            const uint32_t off = lt * F::kPitch + (in_block + i8 * 8) * 2;
            const uint32_t swz = kN >= 64 ? 0x70u : kN == 32 ? 0x30u : 0x10u;
            *reinterpret_cast<uint4*>(pb + (off ^ ((off >> 3) & swz))) = make_uint4(o4[0], o4[1], o4[2], o4[3]);
          }
        }
        proxy_fence();
        tc_fence_before();
        mbar_arrive(pfull + sb);
      }
      // ---- the item's end: sums over the keys, then the rows
      wait_or_dead(pdone + ((at - 1) & 1), ((at - 1) >> 1) & 1, dead);
      tc_fence_after();
#pragma unroll
      for (int sub = 0; sub < kCols / kSub; ++sub) {
        float y[kSub];
#pragma unroll
        for (int i = 0; i < kSub; ++i) y[i] = l[sub * kSub + i];
        const float s = warp_sums<kSub>(y);
        if (lane < kSub) part[wq][col0 + sub * kSub + lane] = s;
      }
      bar_sync(bar, 128);
      if (lt < kCols) sums[col0 + lt] = (part[0][col0 + lt] + part[1][col0 + lt]) + (part[2][col0 + lt] + part[3][col0 + lt]);
      if (kPacked) {
        bar_sync(bar, 128);
#pragma unroll
        for (int sub = 0; sub < kCols / kSub; ++sub) {
          float y[kSub];
#pragma unroll
          for (int i = 0; i < kSub; ++i) y[i] = cs[sub * kSub + i];
          const float s = warp_sums<kSub>(y);
          if (lane < kSub) part[wq][col0 + sub * kSub + lane] = s;
        }
        bar_sync(bar, 128);
        if (lt < kCols)
          csums[col0 + lt] = (part[0][col0 + lt] + part[1][col0 + lt]) + (part[2][col0 + lt] + part[3][col0 + lt]);
      }
      bar_sync(bar, 128);
      const int32_t rows = it.rows;            // live rows
      const int ch = wq * 32 + lane;           // this lane's channel
      const bool whole = it.tiles == it.all;
      const auto place_of = [&](int32_t c, int64_t& token, int32_t& head) {  // of row c of the block
        const int32_t t = (it.row0 + c) / a.group;
        token = static_cast<int64_t>(it.qbegin) + t;
        head = it.head * a.group + (it.row0 + c - t * a.group);
      };
      int64_t token;
      int32_t head;
      float* piece = a.pieces + (static_cast<int64_t>(blockIdx.x) * 2 + it.piece) * kSlotFloats;
      if (wq * 32 < kHalves * 64) {
#pragma unroll 1
        for (int sub = 0; sub < kCols / kSub; ++sub) {
          const int c0 = col0 + sub * kSub;
          if (c0 >= rows) break;
          float o[kSub];
          tmem_ld(o_base + sub * kSub, o);
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            const int c = c0 + i;
            if (kPacked) o[i] += csums[c];
            if (c >= rows) continue;
            if (whole) {
              const float s = sums[c], y = s == 0.0f ? 0.0f : __fdividef(o[i], s);
              place_of(c, token, head);
              if (ch < a.c.dim)
                a.out[token * a.out_token + head * a.out_head + ch] = static_cast<uint16_t>(bf16_pair(y, 0.0f));
            } else {
              __stcg(piece + c * 128 + ch, o[i]);
            }
          }
        }
      }
      if (lt < kCols && col0 + lt < rows) {
        const int c = col0 + lt;
        if (!whole) {
          __stcg(piece + 128 * 128 + 2 * c, nref[c]);
          __stcg(piece + 128 * 128 + 2 * c + 1, sums[c]);
        } else if (a.lse) {
          place_of(c, token, head);
          a.lse[token * a.num_heads + head] =
              sums[c] == 0.0f ? -INFINITY : 0.69314718055994531f * (log2f(sums[c]) - nref[c]);
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
          // ---- the last CTA of the item joins the pieces, in the CTAs' order
          __threadfence();
          // piece p is CTA cta0 + p's first one, but the first CTA's, which may be its second
          const int64_t s0 = total * it.cta0 / ctas;  // the first CTA's first tile
          const int64_t item_start = (it.piece == 0 ? lo : hi - it.tiles) - it.tile0;
          const int32_t first_piece = item_start == s0 ? 0 : 1;
          const float* base = a.pieces + static_cast<int64_t>(it.cta0) * 2 * kSlotFloats;
          for (int c = (st >> 5); c < rows; c += F::kSoft / 32) {
            place_of(c, token, head);
            float top = -INFINITY;  // the largest reference
            for (int32_t p = lane; p < parts; p += 32) {
              const float* pc = base + (static_cast<int64_t>(p) * 2 + (p == 0 ? first_piece : 0)) * kSlotFloats;
              const float nr = __ldcg(pc + 128 * 128 + 2 * c);
              top = fmaxf(top, nr == kUnset ? -INFINITY : -nr);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
            for (int32_t p0 = 0; p0 < parts; p0 += 32) {
              const int32_t p = p0 + lane;
              float f = 0.0f, ls = 0.0f;
              if (p < parts) {
                const float* pc = base + (static_cast<int64_t>(p) * 2 + (p == 0 ? first_piece : 0)) * kSlotFloats;
                const float nr = __ldcg(pc + 128 * 128 + 2 * c);
                ls = __ldcg(pc + 128 * 128 + 2 * c + 1);
                // a piece in which the row saw nothing has sum 0 (or NaN from a NaN score, which stays)
                f = nr == kUnset ? (ls == 0.0f ? 0.0f : 1.0f) : ex2(-nr - top);
              }
              const int32_t m = min(32, parts - p0);
#pragma unroll 4
              for (int32_t i = 0; i < m; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i), li = __shfl_sync(0xffffffffu, ls, i);
                const int32_t pp = p0 + i;
                const float4 v = __ldcg(reinterpret_cast<const float4*>(
                    base + (static_cast<int64_t>(pp) * 2 + (pp == 0 ? first_piece : 0)) * kSlotFloats + c * 128 + lane * 4));
                sum = __fmaf_rn(fi, li, sum);
                if (fi != 0.0f || li != 0.0f) {
                  acc.x = __fmaf_rn(fi, v.x, acc.x);
                  acc.y = __fmaf_rn(fi, v.y, acc.y);
                  acc.z = __fmaf_rn(fi, v.z, acc.z);
                  acc.w = __fmaf_rn(fi, v.w, acc.w);
                }
              }
            }
            const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
            if (lane * 4 < a.c.dim) {
              uint16_t* o = a.out + token * a.out_token + head * a.out_head + lane * 4;
              const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = static_cast<uint16_t>(bf16_pair(y[e], 0.0f));
            }
            if (lane == 0 && a.lse)
              a.lse[token * a.num_heads + head] =
                  sum == 0.0f ? -INFINITY : 0.69314718055994531f * (log2f(sum) + top);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty + b);
    }
  } else if (kPacked) {
    // --------------------------------------------------------- unpacking --
    const int key = tid - 128 - F::kSoft;
    bool ok = true;
    const auto unpack = [&](int32_t tile, bool is_v, int32_t seq) {
      const int rs = tile % F::kRawStages, s = seq % kRing;
      if (!is_v) ok = ok && wait_or_dead(rfull + rs, (tile / F::kRawStages) & 1, dead);
      ok = ok && wait_or_dead(empty + s, ((seq / kRing) & 1) ^ 1u, dead);
      if (!ok) return;
      const uint8_t* src = raw + rs * F::kRaw + (is_v ? kTile * F::kRawRow : 0);
      const uint32_t pair = reinterpret_cast<const uint32_t*>(raw + rs * F::kRaw + 2 * kTile * F::kRawRow)[(is_v ? kTile : 0) + key];
      (is_v ? v_pair : k_pair)[tile % kPairs][key] = pair;
      uint8_t* dst = ring + s * F::kStage + key * 128;
#pragma unroll
      for (int c = 0; c < 2 * kHalves; ++c) {  // 16 packed bytes: 32 channels
        const uint32_t off = key * F::kRawRow + c * 16;
        const uint4 w4 = *reinterpret_cast<const uint4*>(src + (off ^ ((off >> 3) & (kHalves == 2 ? 0x30u : 0x10u))));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // 128 + n in bf16 is 0x4300 | n; minus 136 leaves n - 8 exactly
            uint32_t y = ((w[e] >> (4 * i)) & 0x000f000fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(y), "r"(0x43084308u));
          }
          const int chunk = c * 4 + e;  // 8 channels
          *reinterpret_cast<uint4*>(dst + (chunk >> 3) * 16384 + (((chunk & 7) ^ (key & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      proxy_fence();
      mbar_arrive(full + s);
      if (is_v) mbar_arrive(rempty + rs);
    };
    int32_t at = 0;
    for (int32_t k = 0; at < my_tiles && ok; ++k) {
      ok = wait_or_dead(qfull + k % kNQ, (k / kNQ) & 1, dead);
      if (!ok) break;
      const int32_t tiles = items[k % kNQ].tiles, f = at;
      for (int32_t t = 0; t < tiles; ++t) {
        unpack(f + t, false, k_seq(f, t));
        if (t > 0) unpack(f + t - 1, true, v_seq(f, tiles, t - 1));
      }
      unpack(f + tiles - 1, true, v_seq(f, tiles, tiles - 1));
      at += tiles;
    }
  }
  __syncthreads();
  if (s_dead && my_tiles > 0) {
    const int32_t r0 = s_chunk0 * chunk, r1 = min(a.num_requests, (s_chunk1 + 1) * chunk);
    for (int32_t r = r0 + tid; r < r1; r += F::kThreads) a.status[r] = SS_ROW_TIMEOUT;
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::kTmem) : "memory");
  }
}

template <int kN, bool kPacked, int kHalves>
ss_status launch(const AttnArgs& a, cudaStream_t s) {
  using F = Cfg<kN, kPacked, kHalves>;
  const void* fn = reinterpret_cast<const void*>(&attn_kernel<kN, kPacked, kHalves>);
  CUtensorMap mk, mv;
  const int unit = 1 << (a.c.page_shift < 7 ? a.c.page_shift : 7);
  if (!make_cache_map(&mk, a.c.k, a.c, unit) || !make_cache_map(&mv, a.c.v, a.c, unit)) return SS_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
  if (e == cudaSuccess) {
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    attn_kernel<kN, kPacked, kHalves><<<grid, F::kThreads, F::kSmem, s>>>(mk, mv, a);
  }
  return finish(e);
}

#endif  // __CUDACC__

}  // namespace ssa
