// ss_cache.cu -- the paged key/value cache: writing and reading rows (bf16 or
// 4 bits; 8 bits are read here, and written by ss_rope.cu), and the pages'
// bookkeeping (reserve, fork, compact, trim).
//
// A row is one token's keys or values of one head.  All of it moves bytes and
// computes next to nothing, so the floor of every call is its bytes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss.h"
#include "ss_cache.h"
#include "ss_nvtx.h"
#include "ss_rows.cuh"

namespace ssc {
using namespace ss;

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / kRowLanes;     // rows in flight per CTA
constexpr int kMostCtas = 4 * 152;                // per request

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

// A row is (token, K or V, head): 16 lanes of 16 bytes on the bf16 side.  16
// lanes take kEach consecutive rows of one token (four where the heads are
// even), so a token's page is looked up once for them and their loads are in
// flight together; CTA (x, r) takes kGroups * kEach rows of request r, then a
// grid's width further.  4 x 2-6k tokens, 8 heads of 128 channels: 4 bits in
// 32.6 us (67 with a division per channel), out in 21.6 (4.4 TB/s), both bound
// by instructions first (72 % of the issue slots: rounding or unpacking, and
// the addresses), out also by the loads' latency; 8 bits out in 18.9 (7.0 TB/s with
// what L2 holds); bf16, 32 x 1-8 tokens: 4.4 us, the latency of lengths, table and
// rows one after the other.
template <int kFormat, bool kRead, int kEach>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(const AppendArgs a, const FastDiv by_token) {
  constexpr bool kPacked = kFormat == SS_CACHE_INT4, kBytes = kFormat == SS_CACHE_FP8;
  static_assert(!kBytes || kRead, "8 bits are written block by block");
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
    const int64_t in_cell = max(page, 0) * a.c.page_stride + in_page * a.c.slot_stride + lane * (kPacked ? 4 : kBytes ? 8 : 16);
    const int64_t in_scale = max(page, 0) * a.c.s_page_stride + (kBytes ? in_page >> a.c.block_shift : in_page) * 4;
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
    if constexpr (kBytes) {
      // (bound by instructions: the rows of K, or of V, a step apart)
      const bool is_v = first >= static_cast<uint32_t>(a.c.heads);
      if (is_v || first + kEach <= static_cast<uint32_t>(a.c.heads)) {
        const int32_t head = is_v ? first - a.c.heads : first;
        const uint8_t* from = (is_v ? a.c.v : a.c.k) + in_cell + head * a.c.head_stride;
        const uint8_t* scales = (is_v ? a.c.vs : a.c.ks) + in_scale + head * a.c.s_head_stride;
        uint8_t* to = (is_v ? a.v : a.k) + in_flat + head * a.head_stride;
        uint2 w[kEach];
        float s[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          w[u] = make_uint2(0u, 0u);
          s[u] = 0.0f;
          if (live && page >= 0) {
            w[u] = *reinterpret_cast<const uint2*>(from + u * a.c.head_stride);
            s[u] = *reinterpret_cast<const float*>(scales + u * a.c.s_head_stride);
          }
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
          const uint4 y = read8(w[u], s[u]);
          if (live) *reinterpret_cast<uint4*>(to + u * a.head_stride) = y;
        }
        continue;
      }
    }
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
      } else if (kBytes) {
        const uint2 w = *reinterpret_cast<const uint2*>(cell(u));
        x[u].x = w.x;
        x[u].y = w.y;
        pair[u] = *scale(u);
      } else {
        x[u] = *reinterpret_cast<const uint4*>(cell(u));
      }
    }
    if (!kRead && page < 0) continue;  // the same for the row's 16 lanes
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (kRead) {  // (a step and a low value, or a scale, of 0 give the zeros of a hole)
        if (kBytes) x[u] = read8(make_uint2(x[u].x, x[u].y), __uint_as_float(pair[u]));
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

ss_status check_append(const ss_append_args* args) {
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
  if (2ll * (A.token_offsets ? A.max_tokens : 1) * A.cache->num_kv_heads >= (1ll << 31)) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

static ss_status rows_call(const ss_append_args* args, bool read, cudaStream_t s) {
  const ss_status checked = check_append(args);
  if (checked != SS_OK || args->num_requests == 0) return checked;
  const ss_append_args& A = *args;
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
  // No more CTAs per request than fill the GPU; they loop over the rest of its
  // rows (4 bits, 4 x 2-6k tokens: 32 us, 35 with a CTA for every 64 rows).
  const bool even = (a.c.heads & 1) == 0;
  const int64_t each = kGroups * (even ? 4 : 2), want = (rows + each - 1) / each;
  const dim3 grid(static_cast<unsigned>(want < 1 ? 1 : want > kMostCtas ? kMostCtas : want), A.num_requests);
  const FastDiv by_token = fast_div(2u * a.c.heads);
  const auto launch = [&](auto four, auto two) { (even ? four : two)<<<grid, kThreads, 0, s>>>(a, by_token); };
  constexpr int kBf16 = SS_CACHE_BF16, kInt4 = SS_CACHE_INT4, kFp8 = SS_CACHE_FP8;
  if (a.c.format == SS_CACHE_FP8) launch(rows_kernel<kFp8, true, 4>, rows_kernel<kFp8, true, 2>);
  else if (a.c.format == SS_CACHE_INT4 && read) launch(rows_kernel<kInt4, true, 4>, rows_kernel<kInt4, true, 2>);
  else if (a.c.format == SS_CACHE_INT4) launch(rows_kernel<kInt4, false, 4>, rows_kernel<kInt4, false, 2>);
  else if (read) launch(rows_kernel<kBf16, true, 4>, rows_kernel<kBf16, true, 2>);
  else launch(rows_kernel<kBf16, false, 4>, rows_kernel<kBf16, false, 2>);
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
  const int32_t chunks = row_bytes(c.format, c.dim) / 16;
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
  if (c.format != SS_CACHE_BF16) {
    const int32_t scales = c.format == SS_CACHE_INT4 ? slots : ((slots - 1) >> c.block_shift) + 1;
    const uint8_t* sf = (is_v ? c.vs : c.ks) + layer * c.s_layer_stride + src * c.s_page_stride;
    uint8_t* st = (is_v ? c.vs : c.ks) + layer * c.s_layer_stride + dst * c.s_page_stride;
    for (int32_t x = threadIdx.x; x < scales * c.heads; x += kThreads) {
      const int64_t at = (x / scales) * c.s_head_stride + (x % scales) * 4;
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

// What compact does for a request, which every CTA of it finds by itself.
__device__ __forceinline__ int32_t compact_status(const CompactArgs& a, int i, const int32_t* row, const int32_t* path,
                                                  int32_t base, int32_t count) {
  const int32_t verified = a.verified ? a.verified[i] : SS_ROW_OK;
  int32_t st = SS_ROW_OK;
  if (verified != SS_ROW_OK) st = verified;
  else if (!row || base < 0 || count < 0 || count > a.path_stride || base > 0x7ffffffe - count) st = SS_ROW_BAD_PARAM;
  int bad = 0;
  if (st == SS_ROW_OK)
    for (int32_t j = threadIdx.x; j < count; j += kThreads) {
      const int32_t node = path[j];
      bad |= node <= (j ? path[j - 1] : 0) || page_of(a.t, a.c, row, static_cast<int64_t>(base) + max(node, 0)) < 0 ||
             page_of(a.t, a.c, row, static_cast<int64_t>(base) + 1 + j) < 0;
    }
  if (__syncthreads_or(bad)) st = SS_ROW_BAD_INDEX;
  if (blockIdx.y == 0 && threadIdx.x == 0) {
    a.new_len[i] = (st == SS_ROW_OK) ? base + 1 + count : base;
    a.status[i] = st;
  }
  return st;
}

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
  const int32_t base = a.kv_len[i], count = a.accepted[i];
  const int32_t* row = table_row(a.t, i);
  const int32_t* path = a.path + static_cast<int64_t>(i) * a.path_stride;
  if (compact_status(a, i, row, path, base, count) != SS_ROW_OK) return;
  const int32_t chunks = row_bytes(c.format, c.dim) / 16;
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

// 8 bits: a block into which rows move is encoded anew.  CTA (i, layer) takes
// the blocks from the first to the last; 16 lanes have one slot of a block (as
// in ss_rope.cu), kEach heads of K or V at a time.  Sources lie at or behind
// their places, so those of later blocks lie behind the block being written: a
// block's reads end at the barrier for its scales, before its writes and the
// next block's reads.  64 requests, 32 layers, up to 7 accepted rows: 69 us in a graph
// (bf16 9.7), 94 alone after a flush of L2: all rows of the blocks are read and
// written, block after block with a barrier for each four heads.
__global__ void __launch_bounds__(kThreads) compact_blocks_kernel(const CompactArgs a) {
  constexpr int kEach = 4;
  __shared__ uint32_t s_top[3][2 * kEach];
  const int i = blockIdx.x, layer = blockIdx.y;
  const CacheView& c = a.c;
  const int32_t base = a.kv_len[i], count = a.accepted[i];
  const int32_t* row = table_row(a.t, i);
  const int32_t* path = a.path + static_cast<int64_t>(i) * a.path_stride;
  if (compact_status(a, i, row, path, base, count) != SS_ROW_OK || count == 0) return;
  const int32_t size = 1 << c.block_shift, in_page = (1 << c.page_shift) - 1;
  const int lane = threadIdx.x % kRowLanes, group = threadIdx.x / kRowLanes;
  const int slot = group & (size - 1), side = group >> c.block_shift, sides = kGroups >> c.block_shift;
  const bool live = lane * 8 < c.dim;
  const int32_t units = 2 * c.heads;
  if (threadIdx.x < 3 * 2 * kEach) (&s_top[0][0])[threadIdx.x] = 0;
  __syncthreads();
  int turn = 0;
  const int64_t end = static_cast<int64_t>(base) + 1 + count;  // slots
  for (int64_t b = (static_cast<int64_t>(base) + 1) >> c.block_shift; b <= (end - 1) >> c.block_shift; ++b) {
    const int64_t at = (b << c.block_shift) + slot, j = at - base - 1;
    const int64_t from = j < 0 ? at : j < count ? static_cast<int64_t>(base) + path[j] : -1;  // -1: past the rows
    if (!__syncthreads_or(from >= 0 && from != at)) continue;
    const int32_t to_page = page_of(a.t, c, row, b << c.block_shift);
    const int32_t page = from < 0 ? -1 : page_of(a.t, c, row, from);
    const int64_t to = layer * c.layer_stride + to_page * c.page_stride + (at & in_page) * c.slot_stride + lane * 8;
    const int64_t src = layer * c.layer_stride + max(page, 0) * c.page_stride +
                        (max(from, int64_t{0}) & in_page) * c.slot_stride + lane * 8;
    const int64_t to_scale = layer * c.s_layer_stride + to_page * c.s_page_stride + ((at & in_page) >> c.block_shift) * 4;
    const int64_t src_scale = layer * c.s_layer_stride + max(page, 0) * c.s_page_stride +
                              ((max(from, int64_t{0}) & in_page) >> c.block_shift) * 4;
    for (int32_t u0 = side * kEach; u0 - side * kEach < units; u0 += sides * kEach, turn = turn == 2 ? 0 : turn + 1) {
      float x[kEach][8];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int32_t u = u0 + e, head = u < c.heads ? u : u - c.heads;
        const bool there = u < units && page >= 0;
        uint2 w = make_uint2(0u, 0u);
        float s = 0.0f;
        if (there && live) {
          w = *reinterpret_cast<const uint2*>((u < c.heads ? c.k : c.v) + src + head * c.head_stride);
          s = *reinterpret_cast<const float*>((u < c.heads ? c.ks : c.vs) + src_scale + head * c.s_head_stride);
        }
        decode8(w, s, x[e]);
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(finite_top(x[e])));
        if ((threadIdx.x & 31) == 0 && top != 0) atomicMax(&s_top[turn][side * kEach + e], top);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int32_t u = u0 + e, head = u < c.heads ? u : u - c.heads;
        const Scale8 f = scale8(__uint_as_float(s_top[turn][side * kEach + e]));
        if (u >= units || page < 0) continue;
        if (live) *reinterpret_cast<uint2*>((u < c.heads ? c.k : c.v) + to + head * c.head_stride) = encode8(x[e], f.inv);
        if (j == count - 1 || slot == size - 1)
          if (lane == 0) *reinterpret_cast<float*>((u < c.heads ? c.ks : c.vs) + to_scale + head * c.s_head_stride) = f.s;
      }
      // (the maxima of the batch before have been read before the barrier)
      if (threadIdx.x < 2 * kEach) s_top[turn == 0 ? 2 : turn - 1][threadIdx.x] = 0;
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
  if (args && args->cache && args->cache->format == SS_CACHE_FP8)
    return ssc::append_blocks(args, reinterpret_cast<cudaStream_t>(stream));
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
  const auto kernel = cache->format == SS_CACHE_FP8 ? compact_blocks_kernel : compact_kernel;
  kernel<<<dim3(n, cache->num_layers), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
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
