// ss_attn.cu -- attention of a step's new tokens over the paged cache: a
// sliding window with sinks, drafts in a row or in a tree, the cache in bf16
// or in 4 bits.
//
// One CTA per (query, head): 128 keys at a time, a thread per key for the
// scores, then a thread per channel for the values, with the running maximum
// and sum of the softmax.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ss.h"
#include "ss_cache.h"
#include "ss_nvtx.h"

namespace ssa {
using namespace ss;

constexpr int kThreads = 128;

struct AttnArgs {
  CacheView c;
  TableView t;
  int32_t num_requests, num_heads, group, max_queries, total_queries;
  const int32_t* offsets;
  const int32_t* kv_len;
  const int32_t* parents;
  const uint8_t* q;
  int64_t q_token, q_head;  // bytes
  uint16_t* out;
  int64_t out_token, out_head;  // elements
  float* lse;
  float scale;
  int32_t window, sinks;
  int32_t* status;
};

// Channel `ch` of a packed row.
__device__ __forceinline__ float unpack1(const uint8_t* row, int ch, uint32_t pair) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(row)[ch >> 3];
  const int i = ch & 7;
  return __fmaf_rn(static_cast<float>((w >> ((i & 1) * 16 + (i >> 1) * 4)) & 15u), bf16_lo(pair), bf16_hi(pair));
}

__global__ void __launch_bounds__(kThreads) attn_kernel(const AttnArgs a) {
  __shared__ float s_q[128], s_p[kThreads], s_red[4];
  __shared__ int32_t s_page[kThreads];
  __shared__ uint8_t s_depth[SS_TREE_MAX_NODES];
  const int r = blockIdx.z, head = blockIdx.y, qi = blockIdx.x, tid = threadIdx.x;
  const CacheView& c = a.c;
  const int32_t begin = a.offsets ? a.offsets[r] : r, end = a.offsets ? a.offsets[r + 1] : r + 1;
  const int32_t base = a.kv_len[r], n = end - begin;
  const int32_t* row = table_row(a.t, r);
  const bool tree = a.parents != nullptr;
  const bool ok = row && base >= 0 && begin >= 0 && begin <= end && end <= a.total_queries && n <= a.max_queries &&
                  !(tree && n > SS_TREE_MAX_NODES);
  if (qi == 0 && head == 0 && tid == 0) {
    int32_t st = ok ? SS_ROW_OK : SS_ROW_BAD_PARAM;
    if (ok) {
      if (n > 0 && ((static_cast<int64_t>(base) + n - 1) >> c.page_shift) >= a.t.max_pages) st = SS_ROW_BAD_INDEX;
      if (tree)
        for (int32_t i = 1; i < n; ++i)
          if (a.parents[begin + i] < 0 || a.parents[begin + i] >= i) st = SS_ROW_BAD_PARAM;
    }
    a.status[r] = st;
  }
  if (!ok || qi >= n) return;
  uint64_t path = 0;  // the nodes that this query sees
  int32_t pos = base + qi;
  if (tree) {
    int32_t up = qi, depth = 0;
    for (path = 1ull << qi; up > 0; ++depth) {
      const int32_t pa = a.parents[begin + up];
      up = (pa < 0 || pa >= up) ? 0 : pa;
      path |= 1ull << up;
    }
    pos = base + depth;
    if (tid < n) {
      int32_t d = 0;
      for (int32_t u = tid; u > 0; ++d) {
        const int32_t pa = a.parents[begin + u];
        u = (pa < 0 || pa >= u) ? 0 : pa;
      }
      s_depth[tid] = static_cast<uint8_t>(d);
    }
  }
  if (tid < c.dim) {
    const uint16_t w = reinterpret_cast<const uint16_t*>(a.q + (begin + static_cast<int64_t>(qi)) * a.q_token +
                                                         head * a.q_head)[tid];
    s_q[tid] = __uint_as_float(static_cast<uint32_t>(w) << 16);
  }
  __syncthreads();
  const int kvh = head / a.group;
  const bool packed = c.format == SS_CACHE_INT4;
  float top = -INFINITY, sum = 0.0f, acc = 0.0f;
  const int64_t upto = static_cast<int64_t>(base) + qi + 1;
  for (int64_t j0 = 0; j0 < upto; j0 += kThreads) {
    const int64_t j = j0 + tid;
    bool see = j < upto;
    int64_t place = j;
    if (see && tree && j >= base) {
      see = (path >> (j - base)) & 1;
      place = base + s_depth[j - base];
    }
    see = see && (a.window == 0 || place > static_cast<int64_t>(pos) - a.window || place < a.sinks);
    const int32_t page = see ? page_of(a.t, c, row, j) : -1;
    const int32_t slot = static_cast<int32_t>(j) & ((1 << c.page_shift) - 1);
    float s = -INFINITY;
    if (page >= 0) {
      const uint8_t* k = c.k + page * c.page_stride + kvh * c.head_stride + slot * c.slot_stride;
      float dot = 0.0f;
      if (packed) {
        const uint32_t pair = reinterpret_cast<const uint32_t*>(c.ks + page * c.s_page_stride + kvh * c.s_head_stride)[slot];
        for (int ch = 0; ch < c.dim; ++ch) dot = fmaf(s_q[ch], unpack1(k, ch, pair), dot);
      } else {
        for (int x = 0; x < c.dim / 2; ++x) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(k)[x];
          dot = fmaf(s_q[2 * x], bf16_lo(w), dot);
          dot = fmaf(s_q[2 * x + 1], bf16_hi(w), dot);
        }
      }
      s = dot * a.scale;
    }
    float m = s;
    bool nan = page >= 0 && isnan(s);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float next = fmaxf(top, m);
    const float ref = next == -INFINITY ? 0.0f : next;
    const float f = expf(top - ref);
    const float p = nan ? s : expf(s - ref);
    s_p[tid] = page >= 0 ? p : 0.0f;
    s_page[tid] = page;
    __syncthreads();
    acc *= f;
    sum *= f;
    top = next;
    const int32_t m_keys = static_cast<int32_t>(min(static_cast<int64_t>(kThreads), upto - j0));
    for (int x = 0; x < m_keys; ++x) {
      const int32_t pg = s_page[x];
      if (pg < 0) continue;
      sum += s_p[x];
      if (tid >= c.dim) continue;
      const int32_t sl = static_cast<int32_t>(j0 + x) & ((1 << c.page_shift) - 1);
      const uint8_t* v = c.v + pg * c.page_stride + kvh * c.head_stride + sl * c.slot_stride;
      float val;
      if (packed)
        val = unpack1(v, tid, reinterpret_cast<const uint32_t*>(c.vs + pg * c.s_page_stride + kvh * c.s_head_stride)[sl]);
      else
        val = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(v)[tid]) << 16);
      acc = fmaf(s_p[x], val, acc);
    }
    __syncthreads();
  }
  const int64_t t = begin + static_cast<int64_t>(qi);
  if (tid < c.dim) {
    const float o = sum == 0.0f ? 0.0f : acc / sum;
    a.out[t * a.out_token + head * a.out_head + tid] = static_cast<uint16_t>(bf16_pair(o, 0.0f));
  }
  if (tid == 0 && a.lse) a.lse[t * a.num_heads + head] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace ssa

extern "C" {

size_t ss_attention_workspace_size(void) { return 256; }

ss_status ss_cache_attention(const ss_attention_args* args, void* workspace, size_t workspace_bytes,
                             ss_stream_t stream) {
  SS_NVTX_RANGE("ss_cache_attention");
  using namespace ssa;
  if (!args || !check_cache(args->cache) || !check_table(args->pool)) return SS_ERR_INVALID_ARG;
  const ss_attention_args& A = *args;
  const int32_t kv_heads = A.cache->num_kv_heads;
  if (A.layer < 0 || A.layer >= A.cache->num_layers || A.num_requests < 0 || A.num_requests > 65535 ||
      A.max_queries < 0 || A.total_queries < 0 || A.num_heads < 1 || A.num_heads % kv_heads != 0 ||
      A.num_heads / kv_heads > 128 || A.window < 0 || A.sinks < 0 || !isfinite(A.scale))
    return SS_ERR_INVALID_ARG;
  if (!A.query_offsets && A.total_queries < A.num_requests) return SS_ERR_INVALID_ARG;
  if (A.num_requests == 0) return SS_OK;
  if (!A.kv_len || !A.out_status || !A.q || !A.out || !aligned16(A.q) || (A.q_token_stride & 7) != 0 ||
      (A.q_head_stride & 7) != 0 || (reinterpret_cast<uintptr_t>(A.out) & 1) != 0)
    return SS_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < ss_attention_workspace_size())
    return SS_ERR_WORKSPACE;
  AttnArgs a{};
  a.c = view_of(A.cache, A.layer);
  a.t = table_of(A.pool, A.table_rows);
  a.num_requests = A.num_requests;
  a.num_heads = A.num_heads;
  a.group = A.num_heads / kv_heads;
  a.max_queries = A.query_offsets ? A.max_queries : 1;
  a.total_queries = A.total_queries;
  a.offsets = A.query_offsets;
  a.kv_len = A.kv_len;
  a.parents = A.parents;
  a.q = static_cast<const uint8_t*>(A.q);
  a.q_token = A.q_token_stride * 2;
  a.q_head = A.q_head_stride * 2;
  a.out = static_cast<uint16_t*>(A.out);
  a.out_token = A.out_token_stride;
  a.out_head = A.out_head_stride;
  a.lse = A.lse;
  a.scale = A.scale;
  a.window = A.window;
  a.sinks = A.sinks;
  a.status = A.out_status;
  if (a.max_queries == 0) a.max_queries = 1;  // the statuses are written all the same
  attn_kernel<<<dim3(a.max_queries, a.num_heads, a.num_requests), kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return finish(cudaSuccess);
}

}  // extern "C"
