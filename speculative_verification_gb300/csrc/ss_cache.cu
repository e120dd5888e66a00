// ss_cache.cu -- the paged key/value cache: writing and reading rows (bf16 or
// 4 bits), and the pages' bookkeeping (reserve, fork, compact, trim).
//
// A row is one token's keys or values of one head.  All of it moves bytes and
// computes next to nothing, so the floor of every call is its bytes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss.h"
#include "ss_cache.h"
#include "ss_nvtx.h"

namespace ssc {
using namespace ss;

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;                     // a row is at most 16 lanes of 8 channels
constexpr int kGroups = kThreads / kRowLanes;     // rows in flight per CTA
constexpr int kMostCtas = 4 * 152;                // per request
constexpr uint32_t kNaN2 = 0x7fc07fc0u;           // a bf16 pair of NaNs

struct AppendArgs {
  CacheView c;
  TableView t;
  int32_t max_tokens, total_tokens;
  const int32_t* offsets;
  const int32_t* kv_len;
  uint8_t* k;
  uint8_t* v;
  int64_t token_stride, head_stride;  // bytes
  int32_t* status;
};

// Row number to token and head (division by multiplication: the multiplier is
// floor(2^(31+l) / d) + 1, l = ceil(log2 d), after Granlund and Montgomery).
struct FastDiv {
  uint32_t d, mul, shift;
};
static FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1u << l) < d) ++l;
  return {d, static_cast<uint32_t>((1ull << (31 + l)) / d + 1), l ? l - 1 : 0};
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) {
  return f.d == 1 ? n : __umulhi(n, f.mul) >> f.shift;
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // bf16 pairs; a NaN stays
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight channels of a row, quantised: the row's low value and step come from
// the 16 lanes of the row, as the pair (min x, min -x), so that one shuffle and
// one instruction join two lanes.
//
// round((x - m) / s) without a division per channel: with y = x - m and
// q = y * (1 / s), the remainder y - q s is exact in fp32 (q is off by a few
// units at most and s has 8 bits), and q + (y - q s) / s is the quotient to
// within 2^-20 of its last place before the one rounding.  A quotient that is
// no half differs from every half by more than 1.003 times half a unit (y has
// 24 bits, s has 8), so it is not rounded onto one: adding 1.5 * 2^23 then
// leaves the integer, ties to even, in the low bits.
__device__ __forceinline__ uint32_t quantise8(const uint4 x, bool live, uint32_t lanes, uint32_t& pair) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint32_t mn = min2(min2(w[0], w[1]), min2(w[2], w[3]));
  const uint32_t mx = max2(max2(w[0], w[1]), max2(w[2], w[3])) ^ 0x80008000u;
  uint32_t both = min2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
  if (!live) both = 0x7f807f80u;
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) both = min2(both, __shfl_xor_sync(lanes, both, o, kRowLanes));
  float lo = bf16_lo(both);
  const float range = __fsub_rn(-bf16_hi(both), lo);
  if (!(range < __int_as_float(0x7f800000))) {  // a NaN, an infinity or too wide
    pair = kNaN2;
    return 0;
  }
  // the smallest bf16 that is not below range / 15: then 15 steps reach the
  // highest channel (the division as above)
  constexpr float kTiny = 1.0e-28f, kUp = 18446744073709551616.0f;
  float step = range * (1.0f / 15.0f);
  step = __fmaf_rn(__fmaf_rn(-step, 15.0f, range), 1.0f / 15.0f, step);
  if (range < kTiny) step = __fdiv_rn(range, 15.0f);
  step = __uint_as_float((__float_as_uint(step) + 0xffffu) & 0xffff0000u);
  pair = (__float_as_uint(step) >> 16) | __float_as_uint(lo);  // lo is one of the row's bf16
  if (step == 0.0f) return 0;
  if (range < kTiny) {  // keep 1 / step and the remainders in the normal range: all of it times 2^64
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(0x5f805f80u));
    lo *= kUp;
    step *= kUp;
  }
  const float inv = __fdividef(1.0f, step);
  const uint64_t low2 = two(-lo, -lo), inv2 = two(inv, inv), step2 = two(-step, -step);
  constexpr uint32_t kRound = 0x4b400000u;  // 1.5 * 2^23
  uint32_t out = 0u - 0x11111111u * kRound;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t y = add_2(two(bf16_lo(w[i]), bf16_hi(w[i])), low2), q = mul_2(y, inv2);
    const uint64_t t = add_2(fma_2(fma_2(q, step2, y), inv2, q), two(__uint_as_float(kRound), __uint_as_float(kRound)));
    out += (static_cast<uint32_t>(t) << (4 * i)) + (static_cast<uint32_t>(t >> 32) << (16 + 4 * i));
  }
  return out;
}

__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint32_t pair) {
  const float s = bf16_lo(pair), m = bf16_hi(pair);
  const uint64_t s2 = two(s, s), m2 = two(m, m), off = two(-8388608.0f, -8388608.0f);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 2^23 + n, minus 2^23: no conversion
    const uint64_t n = add_2(two(__uint_as_float(((w >> (4 * i)) & 15u) | 0x4b000000u),
                                 __uint_as_float(((w >> (16 + 4 * i)) & 15u) | 0x4b000000u)), off);
    const uint64_t v = fma_2(n, s2, m2);
    float a, b;
    split(v, a, b);
    o[i] = bf16_pair(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A row is (token, K or V, head): 16 lanes of 16 bytes on the bf16 side.  16
// lanes take kEach consecutive rows of one token (four where the heads are
// even), so a token's page is looked up once for them and their loads are in
// flight together; CTA (x, r) takes kGroups * kEach rows of request r, then a
// grid's width further.  4 x 2-6k tokens, 8 heads of 128 channels: 4 bits in
// 32.6 us (67 with a division per channel), out in 21.6 (4.4 TB/s), both bound
// by instructions first (72 % of the issue slots: rounding or unpacking, and
// the addresses), out also by the loads' latency; bf16, 32 x 1-8 tokens: 4.4
// us, the latency of lengths, table and rows one after the other.
template <bool kPacked, bool kRead, int kEach>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const AppendArgs a, const FastDiv by_token) {
  const int r = blockIdx.y;
  const int32_t begin = a.offsets ? a.offsets[r] : r;
  const int32_t end = a.offsets ? a.offsets[r + 1] : r + 1;
  const int32_t base = a.kv_len[r];
  const int32_t* row = table_row(a.t, r);
  const int32_t n = end - begin;
  const bool ok = row && base >= 0 && begin >= 0 && begin <= end && end <= a.total_tokens && n <= a.max_tokens;
  if (!ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) a.status[r] = SS_ROW_BAD_PARAM;
    return;
  }
  const int lane = threadIdx.x % kRowLanes, group = threadIdx.x / kRowLanes;
  const bool live = lane * 8 < a.c.dim;
  const uint32_t lanes = 0xffffu << (threadIdx.x & 16);
  const uint32_t total = 2u * static_cast<uint32_t>(n) * static_cast<uint32_t>(a.c.heads);
  for (uint32_t i = (blockIdx.x * kGroups + group) * kEach; i < total; i += gridDim.x * (kGroups * kEach)) {
    const uint32_t token = divide(i, by_token), first = i - token * by_token.d;
    const int64_t slot = static_cast<int64_t>(base) + token;
    const int32_t in_page = static_cast<int32_t>(slot) & ((1 << a.c.page_shift) - 1);
    const int32_t page = page_of(a.t, a.c, row, slot);
    const int64_t in_flat = (begin + static_cast<int64_t>(token)) * a.token_stride + lane * 16;
    const int64_t in_cell = max(page, 0) * a.c.page_stride + in_page * a.c.slot_stride + lane * (kPacked ? 4 : 16);
    const int64_t in_scale = max(page, 0) * a.c.s_page_stride + in_page * 4;
    const auto flat = [&](int u) {
      const int32_t head = first + u;
      return head < a.c.heads ? a.k + in_flat + head * a.head_stride : a.v + in_flat + (head - a.c.heads) * a.head_stride;
    };
    const auto cell = [&](int u) {
      const int32_t head = first + u;
      return head < a.c.heads ? a.c.k + in_cell + head * a.c.head_stride
                              : a.c.v + in_cell + (head - a.c.heads) * a.c.head_stride;
    };
    const auto scale = [&](int u) {
      const int32_t head = first + u;
      return reinterpret_cast<uint32_t*>(head < a.c.heads ? a.c.ks + in_scale + head * a.c.s_head_stride
                                                          : a.c.vs + in_scale + (head - a.c.heads) * a.c.s_head_stride);
    };
    uint4 x[kEach];
    uint32_t word[kEach], pair[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      word[u] = pair[u] = 0;
      if (!live || page < 0) continue;
      if (!kRead) {
        x[u] = *reinterpret_cast<const uint4*>(flat(u));
      } else if (kPacked) {
        word[u] = *reinterpret_cast<const uint32_t*>(cell(u));
        pair[u] = *scale(u);
      } else {
        x[u] = *reinterpret_cast<const uint4*>(cell(u));
      }
    }
    if (!kRead && page < 0) continue;  // the same for the row's 16 lanes
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (kRead) {  // (a step and a low value of 0 give the zeros of a hole)
        if (live) *reinterpret_cast<uint4*>(flat(u)) = kPacked ? dequantise8(word[u], pair[u]) : x[u];
      } else if (kPacked) {
        const uint32_t w = quantise8(x[u], live, lanes, pair[u]);
        if (live) *reinterpret_cast<uint32_t*>(cell(u)) = w;
        if (lane == 0) *scale(u) = pair[u];
      } else if (live) {
        *reinterpret_cast<uint4*>(cell(u)) = x[u];
      }
    }
  }
  if (blockIdx.x == 0) {  // the status: does every slot have a page?
    int missing = 0;
    const int64_t last = (static_cast<int64_t>(base) + n - 1) >> a.c.page_shift;
    if (n > 0)
      for (int64_t e = (base >> a.c.page_shift) + threadIdx.x; e <= last; e += kThreads)
        missing |= e >= a.t.max_pages || row[e] < 0 || row[e] >= a.c.num_pages;
    missing = __syncthreads_or(missing);
    if (threadIdx.x == 0) a.status[r] = missing ? SS_ROW_BAD_INDEX : SS_ROW_OK;
  }
}

static ss_status rows_call(const ss_append_args* args, bool read, cudaStream_t s) {
  if (!args || !check_cache(args->cache) || !check_table(args->pool)) return SS_ERR_INVALID_ARG;
  const ss_append_args& A = *args;
  if (A.layer < 0 || A.layer >= A.cache->num_layers || A.num_requests < 0 || A.num_requests > 65535 ||
      A.max_tokens < 0 || A.total_tokens < 0)
    return SS_ERR_INVALID_ARG;
  if (!A.token_offsets && A.total_tokens < A.num_requests) return SS_ERR_INVALID_ARG;
  if (A.num_requests == 0) return SS_OK;
  if (!A.kv_len || !A.out_status || (A.total_tokens > 0 && (!A.k || !A.v)) || !aligned16(A.k) || !aligned16(A.v) || (A.token_stride & 7) != 0 ||
      (A.head_stride & 7) != 0)
    return SS_ERR_INVALID_ARG;
  AppendArgs a{};
  a.c = view_of(A.cache, A.layer);
  a.t = table_of(A.pool, A.table_rows);
  a.max_tokens = A.token_offsets ? A.max_tokens : 1;
  a.total_tokens = A.total_tokens;
  a.offsets = A.token_offsets;
  a.kv_len = A.kv_len;
  a.k = static_cast<uint8_t*>(A.k);
  a.v = static_cast<uint8_t*>(A.v);
  a.token_stride = A.token_stride * 2;
  a.head_stride = A.head_stride * 2;
  a.status = A.out_status;
  const int64_t rows = 2ll * a.max_tokens * a.c.heads;
  if (rows >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
  // No more CTAs per request than fill the GPU; they loop over the rest of its
  // rows (4 bits, 4 x 2-6k tokens: 32 us, 35 with a CTA for every 64 rows).
  const bool even = (a.c.heads & 1) == 0;
  const int64_t each = kGroups * (even ? 4 : 2), want = (rows + each - 1) / each;
  const dim3 grid(static_cast<unsigned>(want < 1 ? 1 : want > kMostCtas ? kMostCtas : want), A.num_requests);
  const FastDiv by_token = fast_div(2u * a.c.heads);
  const bool packed = a.c.format == SS_CACHE_INT4;
  const auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a, by_token); };
  if (even) launch(packed ? (read ? rows_kernel<true, true, 4> : rows_kernel<true, false, 4>)
                          : (read ? rows_kernel<false, true, 4> : rows_kernel<false, false, 4>));
  else launch(packed ? (read ? rows_kernel<true, true, 2> : rows_kernel<true, false, 2>)
                     : (read ? rows_kernel<false, true, 2> : rows_kernel<false, false, 2>));
  return finish(cudaSuccess);
}

// ------------------------------------------------------------- the pages --

constexpr int kBook = 1024;  // threads of the bookkeeping kernels (one CTA: their order is the calls' order)

struct PoolView {
  int32_t num_rows, max_pages;
  int64_t stride;
  int32_t* table;
  int32_t num_pages, page_shift;
  int32_t* refs;
  int32_t* free_pages;
  int32_t* free_count;
};

// Inclusive sum over the CTA's kBook threads; `ws` has kBook / 32 words.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T* ws) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) ws[wid] = x;
  __syncthreads();
  if (wid == 0) {
    T y = ws[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    ws[lane] = y;
  }
  __syncthreads();
  return x + (wid ? ws[wid - 1] : 0);
}

__device__ __forceinline__ int32_t free_now(const PoolView& p) {
  return max(0, min(*p.free_count, p.num_pages));
}

__device__ __forceinline__ bool is_hole(const PoolView& p, int32_t page) { return page < 0 || page >= p.num_pages; }

// The k-th page from the top of the stack of `have` pages (bad contents: -1).
__device__ __forceinline__ int32_t take(const PoolView& p, int32_t have, int32_t k) {
  const int32_t page = p.free_pages[have - 1 - k];
  if (page < 0 || page >= p.num_pages) return -1;
  p.refs[page] = 1;
  return page;
}

// A warp per request counts its holes, one scan over the requests gives each
// its place in the stack, the warps fill the holes.  What the requests want in
// all passes 2^31 where the table does: summed in 64 bits.
__global__ void __launch_bounds__(kBook) reserve_kernel(const PoolView p, int32_t n, const int32_t* rows,
                                                        const int32_t* from, const int32_t* to, int32_t* status) {
  __shared__ int32_t s_need[kBook], s_place[kBook], ws[kBook / 32], s_given;
  __shared__ int64_t ws64[kBook / 32], s_used;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t have = free_now(p);
  const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
  int64_t used = 0;   // pages wanted by the chunks before
  int32_t taken = 0;  // and given
  for (int32_t c = 0; c < n; c += kBook) {
    const int32_t m = min(kBook, n - c);
    for (int32_t i = wid; i < m; i += kBook / 32) {
      const int32_t row = rows ? rows[c + i] : c + i, a = from[c + i], b = to[c + i];
      int32_t need = -1;  // invalid
      if (row >= 0 && row < p.num_rows && a >= 0 && a <= b && b <= most) {
        need = 0;
        const int32_t last = b > 0 ? ((b - 1) >> p.page_shift) + 1 : 0;
        for (int32_t e = (a >> p.page_shift) + lane; e < last; e += 32) need += is_hole(p, p.table[row * p.stride + e]);
        need = (a < b) ? __reduce_add_sync(0xffffffffu, need) : 0;
      }
      if (lane == 0) s_need[i] = need;
    }
    __syncthreads();
    const int32_t need = (threadIdx.x < m) ? max(0, s_need[threadIdx.x]) : 0;
    const int64_t upto = used + block_scan(static_cast<int64_t>(need), ws64);
    const bool fits = upto <= have;
    if (threadIdx.x < m) s_place[threadIdx.x] = (need > 0 && fits) ? static_cast<int32_t>(upto) - need : -1;
    if (threadIdx.x < m)
      status[c + threadIdx.x] = s_need[threadIdx.x] < 0 ? SS_ROW_BAD_PARAM
                                : need == 0 || fits     ? SS_ROW_OK
                                                        : SS_ROW_LIMIT;
    const int32_t given = block_scan(fits ? need : 0, ws);
    if (threadIdx.x == kBook - 1) {
      s_used = upto;
      s_given = given;
    }
    __syncthreads();
    used = s_used;
    taken += s_given;
    for (int32_t i = wid; i < m; i += kBook / 32) {
      int32_t at = s_place[i];
      if (at < 0) continue;
      const int32_t row = rows ? rows[c + i] : c + i, a = from[c + i], b = to[c + i];
      const int32_t last = b > 0 ? ((b - 1) >> p.page_shift) + 1 : 0;
      for (int32_t e0 = a >> p.page_shift; e0 < last; e0 += 32) {
        int32_t* cell = p.table + row * p.stride + e0 + lane;
        const bool hole = e0 + lane < last && is_hole(p, *cell);
        const uint32_t holes = __ballot_sync(0xffffffffu, hole);
        if (hole) *cell = take(p, have, at + __popc(holes & ((1u << lane) - 1u)));
        at += __popc(holes);
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.free_count = have - taken;
}

// The children's table rows; the partly filled last pages are copied by
// fork_copy_kernel, which finds them in the rows written here.
__global__ void __launch_bounds__(kBook) fork_kernel(const PoolView p, int32_t n, const int32_t* parent,
                                                     const int32_t* child, const int32_t* length, int32_t* status) {
  __shared__ int32_t s_state[kBook], ws[kBook / 32], s_used, s_given;
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t have = free_now(p);
  const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
  const int32_t in_page = (1 << p.page_shift) - 1;
  int32_t used = 0, taken = 0;
  for (int32_t c = 0; c < n; c += kBook) {
    const int32_t m = min(kBook, n - c);
    for (int32_t i = wid; i < m; i += kBook / 32) {
      const int32_t pa = parent[c + i], ch = child[c + i], len = length[c + i];
      int32_t state = -1;  // invalid, else whether a page is needed
      if (pa >= 0 && pa < p.num_rows && ch >= 0 && ch < p.num_rows && len >= 0 && len <= most) {
        bool held = false;
        for (int32_t e = lane; e < p.max_pages; e += 32) held |= p.table[ch * p.stride + e] >= 0;
        if (!__any_sync(0xffffffffu, held)) {
          state = 0;
          if (len & in_page) {
            const int32_t e = p.table[pa * p.stride + (len >> p.page_shift)];
            state = e >= 0 && e < p.num_pages;
          }
        }
      }
      if (lane == 0) s_state[i] = state;
    }
    __syncthreads();
    const int32_t need = (threadIdx.x < m) ? max(0, s_state[threadIdx.x]) : 0;
    const int32_t upto = used + block_scan(need, ws);
    const bool fits = upto <= have;
    const int32_t given = block_scan(fits ? need : 0, ws);
    if (threadIdx.x == kBook - 1) {
      s_used = upto;
      s_given = given;
    }
    if (threadIdx.x < m) {
      const int32_t state = s_state[threadIdx.x];
      status[c + threadIdx.x] = state < 0 ? SS_ROW_BAD_PARAM : need && !fits ? SS_ROW_LIMIT : SS_ROW_OK;
      // what the warps do: -2 nothing, -1 share only, k: and take the k-th page
      s_state[threadIdx.x] = (state < 0 || (need && !fits)) ? -2 : need ? upto - 1 : -1;
    }
    __syncthreads();
    used = s_used;
    taken += s_given;
    for (int32_t i = wid; i < m; i += kBook / 32) {
      const int32_t todo = s_state[i];
      if (todo == -2) continue;
      const int32_t* src = p.table + parent[c + i] * p.stride;
      int32_t* dst = p.table + child[c + i] * p.stride;
      const int32_t full = length[c + i] >> p.page_shift;
      for (int32_t e = lane; e < p.max_pages; e += 32) {
        int32_t page = -1;
        if (e < full) {
          page = src[e];
          if (page < 0 || page >= p.num_pages) page = -1;
          else atomicAdd(p.refs + page, 1);
        } else if (e == full && todo >= 0) {
          page = take(p, have, todo);
        }
        dst[e] = page;
      }
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.free_count = have - taken;
}

// Bound by HBM: 64 children, 32 layers, half-filled pages of 64 slots, 57 us
// (66 with one load in flight per thread).
// CTA (i, 2 * layer + K or V): the used slots of the last page of child i.
__global__ void __launch_bounds__(kThreads) fork_copy_kernel(const PoolView p, const CacheView c, const int32_t* parent,
                                                             const int32_t* child, const int32_t* length,
                                                             const int32_t* status) {
  const int i = blockIdx.x, layer = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  if (status[i] != SS_ROW_OK) return;
  const int32_t len = length[i], slots = len & ((1 << c.page_shift) - 1), e = len >> c.page_shift;
  if (slots == 0) return;
  const int32_t src = p.table[parent[i] * p.stride + e], dst = p.table[child[i] * p.stride + e];
  if (src < 0 || src >= c.num_pages || dst < 0 || dst >= c.num_pages) return;
  const int32_t chunks = (c.format == SS_CACHE_INT4 ? c.dim / 2 : c.dim * 2) / 16;
  const uint8_t* from = (is_v ? c.v : c.k) + layer * c.layer_stride + src * c.page_stride;
  uint8_t* to = (is_v ? c.v : c.k) + layer * c.layer_stride + dst * c.page_stride;
  const int32_t per_head = slots * chunks, total = per_head * c.heads;
  for (int32_t x0 = threadIdx.x; x0 < total; x0 += 4 * kThreads) {
    int64_t at[4];
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int32_t x = x0 + u * kThreads;
      if (x >= total) continue;
      const int32_t head = x / per_head, y = x - head * per_head, slot = y / chunks, chunk = y - slot * chunks;
      at[u] = head * c.head_stride + slot * c.slot_stride + chunk * 16;
      v[u] = *reinterpret_cast<const uint4*>(from + at[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (x0 + u * kThreads < total) *reinterpret_cast<uint4*>(to + at[u]) = v[u];
  }
  if (c.format == SS_CACHE_INT4) {
    const uint8_t* sf = (is_v ? c.vs : c.ks) + layer * c.s_layer_stride + src * c.s_page_stride;
    uint8_t* st = (is_v ? c.vs : c.ks) + layer * c.s_layer_stride + dst * c.s_page_stride;
    for (int32_t x = threadIdx.x; x < slots * c.heads; x += kThreads) {
      const int64_t at = (x / slots) * c.s_head_stride + (x % slots) * 4;
      *reinterpret_cast<uint32_t*>(st + at) = *reinterpret_cast<const uint32_t*>(sf + at);
    }
  }
}

struct CompactArgs {
  CacheView c;
  TableView t;
  const int32_t* kv_len;
  const int32_t* path;
  int32_t path_stride;
  const int32_t* accepted;
  const int32_t* verified;
  int32_t* new_len;
  int32_t* status;
};

constexpr int kPath = 64;  // accepted nodes whose places are held in shared memory at once

// CTA (i, layer): thread t moves the same 16 bytes of every accepted row, in
// the path's order: node j's place kv_len + 1 + j is at or before its source
// kv_len + path[j] (the path is increasing and starts at 1 or more) and before
// every later source, so no row is overwritten before it is read.  64 requests, 32
// layers, up to 7 accepted rows: 13 us, the latency of path, table and rows.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  __shared__ int64_t s_from[kPath], s_to[kPath], s_sfrom[kPath], s_sto[kPath];
  const int i = blockIdx.x, layer = blockIdx.y;
  const CacheView& c = a.c;
  const int32_t base = a.kv_len[i], count = a.accepted[i], verified = a.verified ? a.verified[i] : SS_ROW_OK;
  const int32_t* row = table_row(a.t, i);
  const int32_t* path = a.path + static_cast<int64_t>(i) * a.path_stride;
  int32_t st = SS_ROW_OK;
  if (verified != SS_ROW_OK) st = verified;
  else if (!row || base < 0 || count < 0 || count > a.path_stride || base > 0x7ffffffe - count) st = SS_ROW_BAD_PARAM;
  int bad = 0;
  if (st == SS_ROW_OK)
    for (int32_t j = threadIdx.x; j < count; j += kThreads) {
      const int32_t node = path[j];
      bad |= node <= (j ? path[j - 1] : 0) || page_of(a.t, c, row, static_cast<int64_t>(base) + max(node, 0)) < 0 ||
             page_of(a.t, c, row, static_cast<int64_t>(base) + 1 + j) < 0;
    }
  if (__syncthreads_or(bad)) st = SS_ROW_BAD_INDEX;
  if (layer == 0 && threadIdx.x == 0) {
    a.new_len[i] = (st == SS_ROW_OK) ? base + 1 + count : base;
    a.status[i] = st;
  }
  if (st != SS_ROW_OK) return;
  const int32_t chunks = (c.format == SS_CACHE_INT4 ? c.dim / 2 : c.dim * 2) / 16;
  const int32_t per = chunks * c.heads, in_page = (1 << c.page_shift) - 1;
  for (int32_t j0 = 0; j0 < count; j0 += kPath) {
    const int32_t m = min(kPath, count - j0);
    __syncthreads();
    if (threadIdx.x < m) {
      const int32_t j = j0 + threadIdx.x;
      const int64_t src = static_cast<int64_t>(base) + path[j], dst = static_cast<int64_t>(base) + 1 + j;
      const int64_t sp = page_of(a.t, c, row, src), dp = page_of(a.t, c, row, dst);
      s_from[threadIdx.x] = src == dst ? -1 : sp * c.page_stride + (src & in_page) * c.slot_stride;
      s_to[threadIdx.x] = dp * c.page_stride + (dst & in_page) * c.slot_stride;
      s_sfrom[threadIdx.x] = sp * c.s_page_stride + (src & in_page) * 4;
      s_sto[threadIdx.x] = dp * c.s_page_stride + (dst & in_page) * 4;
    }
    __syncthreads();
    for (int32_t x = threadIdx.x; x < 2 * per; x += kThreads) {
      const int32_t y = x < per ? x : x - per, head = y / chunks, chunk = y - head * chunks;
      uint8_t* at = (x < per ? c.k : c.v) + layer * c.layer_stride + head * c.head_stride + chunk * 16;
      for (int32_t j8 = 0; j8 < m; j8 += 8) {  // read, then written: no later source lies before these places
        uint4 v[8];
#pragma unroll
        for (int32_t u = 0; u < 8; ++u)
          if (j8 + u < m && s_from[j8 + u] >= 0) v[u] = *reinterpret_cast<const uint4*>(at + s_from[j8 + u]);
#pragma unroll
        for (int32_t u = 0; u < 8; ++u)
          if (j8 + u < m && s_from[j8 + u] >= 0) *reinterpret_cast<uint4*>(at + s_to[j8 + u]) = v[u];
      }
    }
    if (c.format == SS_CACHE_INT4)
      for (int32_t x = threadIdx.x; x < 2 * c.heads; x += kThreads) {
        const int32_t head = x < c.heads ? x : x - c.heads;
        uint8_t* at = (x < c.heads ? c.ks : c.vs) + layer * c.s_layer_stride + head * c.s_head_stride;
        for (int32_t j = 0; j < m; ++j)
          if (s_from[j] >= 0)
            *reinterpret_cast<uint32_t*>(at + s_sto[j]) = *reinterpret_cast<const uint32_t*>(at + s_sfrom[j]);
      }
  }
}

// The usual sizes, up to kBook * kFew entries in all: the four passes of
// trim_kernel with the entries in registers, thread t holding consecutive ones
// from the last entry of the last request on.  64 rows of 96 entries take
// 10.3 us instead of 12.7, 80 rows of 33 take 7.1 instead of 12.
constexpr int kFew = 8;
__device__ void trim_few(const PoolView& p, int32_t n, const int32_t* rows, const int32_t* length, int32_t window,
                         int32_t sinks, int32_t* status) {
  __shared__ int32_t ws[kBook / 32];
  const int32_t t = threadIdx.x, have = free_now(p), total = n * p.max_pages;
  const int32_t per = (total + kBook - 1) / kBook, size = 1 << p.page_shift;
  for (int32_t i = t; i < n; i += kBook) {
    const int32_t row = rows ? rows[i] : i;
    status[i] = row < 0 || row >= p.num_rows || length[i] < 0 ? SS_ROW_BAD_PARAM : SS_ROW_OK;
  }
  int32_t page[kFew];
  int32_t* cell[kFew];
#pragma unroll
  for (int u = 0; u < kFew; ++u) {
    page[u] = -1;
    const int32_t lin = total - 1 - (t * per + u);
    if (u >= per || lin < 0) continue;
    const int32_t i = lin / p.max_pages, e = lin - i * p.max_pages;
    const int32_t row = rows ? rows[i] : i;
    const int64_t len = length[i], first = static_cast<int64_t>(e) << p.page_shift;
    if (row < 0 || row >= p.num_rows || len < 0) continue;
    if (first < len && (first < sinks || window == 0 || first + size > len - window)) continue;  // kept
    cell[u] = p.table + row * p.stride + e;
    page[u] = *cell[u];
  }
  __syncthreads();  // the statuses are there
#pragma unroll
  for (int u = 0; u < kFew; ++u) {
    if (u >= per || page[u] < 0) continue;
    *cell[u] = -1;
    bool bad = page[u] >= p.num_pages;
    if (!bad && atomicSub(p.refs + page[u], 1) <= 0) {
      atomicAdd(p.refs + page[u], 1);
      bad = true;
    }
    if (bad) {
      status[(total - 1 - (t * per + u)) / p.max_pages] = SS_ROW_BAD_INDEX;
      page[u] = -1;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kFew; ++u)
    if (u < per && page[u] >= 0 && *reinterpret_cast<volatile int32_t*>(p.refs + page[u]) <= 0)
      atomicMin(p.refs + page[u], -1 - (total - 1 - (t * per + u)));
  __syncthreads();
  int32_t wins = 0;
#pragma unroll
  for (int u = 0; u < kFew; ++u) {
    const bool win = u < per && page[u] >= 0 &&
                     *reinterpret_cast<volatile int32_t*>(p.refs + page[u]) == -1 - (total - 1 - (t * per + u));
    if (!win) page[u] = -1;
    wins += win;
  }
  const int32_t upto = block_scan(wins, ws);
  int32_t place = have + upto - wins;
#pragma unroll
  for (int u = 0; u < kFew; ++u)
    if (u < per && page[u] >= 0) {
      if (place < p.num_pages) p.free_pages[place] = page[u];
      p.refs[page[u]] = 0;
      ++place;
    }
  if (t == kBook - 1) *p.free_count = min(have + upto, p.num_pages);
}

// One CTA, a warp per table row, passes over the rows:
//   1. every dropped entry takes one from its page's count;
//   2. an entry whose page's count is now 0 bids for giving it back: the
//      largest (request, entry) number wins, kept as a negative count;
//   3. the winners are counted per row, a scan from the last row to the first
//      gives each its place on the stack, and the entries become holes.
// So the stack's order depends on the call's arguments alone.
__global__ void __launch_bounds__(kBook) trim_kernel(const PoolView p, int32_t n, const int32_t* rows,
                                                     const int32_t* length, int32_t window, int32_t sinks,
                                                     int32_t* status) {
  __shared__ int32_t s_count[kBook], s_place[kBook], ws[kBook / 32], s_total;
  if (static_cast<int64_t>(n) * p.max_pages <= kBook * kFew) {
    trim_few(p, n, rows, length, window, sinks, status);
    return;
  }
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t have = free_now(p);
  const int32_t size = 1 << p.page_shift;
  const auto row_of = [&](int32_t i) -> int32_t* {
    const int32_t row = rows ? rows[i] : i;
    return (row < 0 || row >= p.num_rows || length[i] < 0) ? nullptr : p.table + row * p.stride;
  };
  const auto dropped = [&](int32_t e, int64_t len) {
    const int64_t first = static_cast<int64_t>(e) << p.page_shift;
    return !(first < len && (first < sinks || window == 0 || first + size > len - window));
  };
  const auto bid = [&](int32_t i, int32_t e) { return -1 - (i * p.max_pages + e); };
  for (int32_t i = wid; i < n; i += kBook / 32) {
    int32_t* row = row_of(i);
    bool bad = false;
    if (row) {
      const int32_t len = length[i];
      for (int32_t e = lane; e < p.max_pages; e += 32) {
        const int32_t page = row[e];
        if (page < 0 || !dropped(e, len)) continue;
        if (page >= p.num_pages) {
          bad = true;
          row[e] = -1;
        } else if (atomicSub(p.refs + page, 1) <= 0) {
          atomicAdd(p.refs + page, 1);
          bad = true;
          row[e] = -1;
        }
      }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) status[i] = !row ? SS_ROW_BAD_PARAM : bad ? SS_ROW_BAD_INDEX : SS_ROW_OK;
  }
  __syncthreads();
  for (int32_t i = wid; i < n; i += kBook / 32) {
    const int32_t* row = row_of(i);
    if (!row) continue;
    const int32_t len = length[i];
    for (int32_t e = lane; e < p.max_pages; e += 32)
      if (row[e] >= 0 && dropped(e, len)) {
        int32_t* ref = p.refs + row[e];
        if (*reinterpret_cast<volatile int32_t*>(ref) <= 0) atomicMin(ref, bid(i, e));
      }
  }
  __syncthreads();
  int32_t given = 0;
  for (int32_t c = (n - 1) / kBook * kBook; c >= 0; c -= kBook) {  // the last requests first
    const int32_t m = min(kBook, n - c);
    if (threadIdx.x < kBook) s_count[threadIdx.x] = 0;
    __syncthreads();
    for (int32_t i = wid; i < m; i += kBook / 32) {
      const int32_t* row = row_of(c + i);
      int32_t wins = 0;
      if (row) {
        const int32_t len = length[c + i];
        for (int32_t e = lane; e < p.max_pages; e += 32)
          if (row[e] >= 0 && dropped(e, len))
            wins += *reinterpret_cast<volatile int32_t*>(p.refs + row[e]) == bid(c + i, e);
      }
      wins = __reduce_add_sync(0xffffffffu, wins);
      if (lane == 0) s_count[m - 1 - i] = wins;
    }
    __syncthreads();
    const int32_t upto = block_scan(s_count[threadIdx.x], ws);
    s_place[threadIdx.x] = have + given + upto;  // one past the place of the row's first winner
    if (threadIdx.x == kBook - 1) s_total = upto;
    __syncthreads();
    for (int32_t i = wid; i < m; i += kBook / 32) {
      int32_t* row = row_of(c + i);
      if (!row) continue;
      int32_t at = s_place[m - 1 - i];
      const int32_t len = length[c + i];
      for (int32_t e0 = 0; e0 < p.max_pages; e0 += 32) {
        const int32_t e = e0 + lane;
        const bool out = e < p.max_pages && row[e] >= 0 && dropped(e, len);
        const int32_t page = out ? row[e] : 0;
        const bool win = out && *reinterpret_cast<volatile int32_t*>(p.refs + page) == bid(c + i, e);
        const uint32_t wins = __ballot_sync(0xffffffffu, win);
        if (win) {
          const int32_t place = at - 1 - __popc(wins & ((1u << lane) - 1u));
          if (place < p.num_pages) p.free_pages[place] = page;
          p.refs[page] = 0;
        }
        if (out) row[e] = -1;
        at -= __popc(wins);
      }
    }
    given += s_total;
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.free_count = min(have + given, p.num_pages);
}

static bool pool_view(const ss_page_pool* p, PoolView* v) {
  if (!check_table(p) || p->num_pages < 1 || p->page_size < 8 || p->page_size > 1024 ||
      (p->page_size & (p->page_size - 1)) != 0 || !p->ref_count || !p->free_pages || !p->free_count)
    return false;
  *v = PoolView{};
  v->num_rows = p->num_rows;
  v->max_pages = p->max_pages;
  v->stride = p->row_stride;
  v->table = p->page_table;
  v->num_pages = p->num_pages;
  while ((1 << v->page_shift) < p->page_size) ++v->page_shift;
  v->refs = p->ref_count;
  v->free_pages = p->free_pages;
  v->free_count = p->free_count;
  return true;
}

}  // namespace ssc

extern "C" {

ss_status ss_cache_append(const ss_append_args* args, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_cache_append");
  return ssc::rows_call(args, false, reinterpret_cast<cudaStream_t>(stream));
}

ss_status ss_cache_read(const ss_append_args* args, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_cache_read");
  return ssc::rows_call(args, true, reinterpret_cast<cudaStream_t>(stream));
}

ss_status ss_pages_reserve(const ss_page_pool* pool, int32_t n, const int32_t* table_rows, const int32_t* from_len,
                           const int32_t* to_len, int32_t* out_status, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_pages_reserve");
  using namespace ssc;
  PoolView p;
  if (!pool_view(pool, &p) || n < 0) return SS_ERR_INVALID_ARG;
  if (n == 0) return SS_OK;
  if (!from_len || !to_len || !out_status) return SS_ERR_INVALID_ARG;
  reserve_kernel<<<1, kBook, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, n, table_rows, from_len, to_len,
                                                                          out_status);
  return finish(cudaSuccess);
}

ss_status ss_pages_fork(const ss_page_pool* pool, const ss_kv_cache* cache, int32_t n, const int32_t* parent,
                        const int32_t* child, const int32_t* length, int32_t* out_status, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_pages_fork");
  using namespace ssc;
  PoolView p;
  if (!pool_view(pool, &p) || !check_cache(cache) || cache->page_size != pool->page_size ||
      cache->num_pages != pool->num_pages || cache->num_layers > 32767 || n < 0)
    return SS_ERR_INVALID_ARG;
  if (n == 0) return SS_OK;
  if (!parent || !child || !length || !out_status) return SS_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  fork_kernel<<<1, kBook, 0, s>>>(p, n, parent, child, length, out_status);
  fork_copy_kernel<<<dim3(n, 2 * cache->num_layers), kThreads, 0, s>>>(p, view_of(cache, 0), parent, child, length,
                                                                      out_status);
  return finish(cudaSuccess);
}

ss_status ss_pages_compact(const ss_page_pool* pool, const ss_kv_cache* cache, int32_t n, const int32_t* table_rows,
                           const int32_t* kv_len, const int32_t* path, int32_t path_stride,
                           const int32_t* num_accepted, const int32_t* verify_status, int32_t* new_len,
                           int32_t* out_status, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_pages_compact");
  using namespace ssc;
  if (!check_table(pool) || !check_cache(cache) || cache->page_size != pool->page_size || cache->num_layers > 65535 ||
      n < 0 || path_stride < 0)
    return SS_ERR_INVALID_ARG;
  if (n == 0) return SS_OK;
  if (!kv_len || !path || !num_accepted || !new_len || new_len == kv_len || !out_status) return SS_ERR_INVALID_ARG;
  CompactArgs a{};
  a.c = view_of(cache, 0);
  a.t = table_of(pool, table_rows);
  a.kv_len = kv_len;
  a.path = path;
  a.path_stride = path_stride;
  a.accepted = num_accepted;
  a.verified = verify_status;
  a.new_len = new_len;
  a.status = out_status;
  compact_kernel<<<dim3(n, cache->num_layers), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return finish(cudaSuccess);
}

ss_status ss_pages_trim(const ss_page_pool* pool, int32_t n, const int32_t* table_rows, const int32_t* length,
                        int32_t window, int32_t sinks, int32_t* out_status, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_pages_trim");
  using namespace ssc;
  PoolView p;
  if (!pool_view(pool, &p) || n < 0 || window < 0 || sinks < 0) return SS_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n) * p.max_pages >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
  if (n == 0) return SS_OK;
  if (!length || !out_status) return SS_ERR_INVALID_ARG;
  trim_kernel<<<1, kBook, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, n, table_rows, length, window, sinks,
                                                                      out_status);
  return finish(cudaSuccess);
}

}  // extern "C"
