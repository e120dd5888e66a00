// ss_attn.cu -- attention of a step's new tokens over the paged cache: the
// entry point's checks and the choice of the kernel (ss_attn.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ss.h"
#include "ss_attn.cuh"
#include "ss_cache.h"
#include "ss_nvtx.h"

namespace ssa {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// bf16: boxes of 64 channels, the 128-byte swizzle, as the tensor cores read
// them.  4 bits: whole rows (32 or 64 bytes), the swizzle of that width, which
// spreads the rows that a warp unpacks over the shared-memory banks.  8 bits:
// whole rows (64 or 128 bytes), likewise, and K's are what the tensor cores read.
// Channels and pages out of range read as zero.
bool make_cache_map(CUtensorMap* m, void* base, const CacheView& c, int box_slots) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool packed = c.format == SS_CACHE_INT4, bytes = c.format == SS_CACHE_FP8;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(packed ? c.dim / 2 : c.dim), 1ull << c.page_shift,
                              static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.slot_stride), static_cast<cuuint64_t>(c.head_stride),
                                 static_cast<cuuint64_t>(c.page_stride)};
  const bool wide = c.dim > 64;
  const cuuint32_t box[4] = {packed ? (wide ? 64u : 32u) : bytes && wide ? 128u : 64u, static_cast<cuuint32_t>(box_slots), 1u, 1u};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, packed || bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            packed ? (wide ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B)
            : bytes && !wide ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_query_map(CUtensorMap* m, const AttnArgs& a, int rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool boxes = rows % a.group == 0;
  // the stride of a dimension of one entry is never used
  const int64_t head = a.num_heads > 1 ? a.q_head : 256, token = a.total_queries > 1 ? a.q_token : 256;
  // (no queries at all: a map that nothing is copied with, of an address that is there)
  void* base = a.total_queries > 0 ? const_cast<uint8_t*>(a.q) : a.c.k;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.dim), static_cast<cuuint64_t>(a.num_heads),
                              static_cast<cuuint64_t>(a.total_queries > 0 ? a.total_queries : 1)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head), static_cast<cuuint64_t>(token)};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(boxes ? a.group : 1),
                             static_cast<cuuint32_t>(boxes ? rows / a.group : 1)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ssa

extern "C" {

size_t ss_attention_workspace_size(void) {
  return ssa::kMaxCtas * sizeof(int32_t) + static_cast<size_t>(ssa::kMaxCtas) * 2 * ssa::kSlotFloats * sizeof(float) + 256;
}

static ss_status attention(const ss_attention_args* args, int32_t stall, void* workspace, size_t workspace_bytes,
                           ss_stream_t stream) {
  using namespace ssa;
  if (!args || !check_cache(args->cache) || !check_table(args->pool)) return SS_ERR_INVALID_ARG;
  const ss_attention_args& A = *args;
  const int32_t kv_heads = A.cache->num_kv_heads;
  if (A.layer < 0 || A.layer >= A.cache->num_layers || A.num_requests < 0 || A.num_requests > 16384 ||
      A.max_queries < 0 || A.total_queries < 0 || A.num_heads < 1 || A.num_heads % kv_heads != 0 ||
      A.num_heads / kv_heads > 128 || A.window < 0 || A.sinks < 0 || !isfinite(A.scale))
    return SS_ERR_INVALID_ARG;
  // a request's rows, and where the loops over 32 blocks of 128 of them end, are counted in 31 bits
  if (static_cast<int64_t>(A.max_queries) * A.num_heads > (1ll << 31) - 8192) return SS_ERR_INVALID_ARG;
  if (!A.query_offsets && A.total_queries < A.num_requests) return SS_ERR_INVALID_ARG;
  if (A.num_requests == 0) return SS_OK;
  if (!A.kv_len || !A.out_status || (A.total_queries > 0 && (!A.q || !A.out)) || !aligned16(A.q) || (A.q_token_stride & 7) != 0 ||
      (A.q_head_stride & 7) != 0 || (reinterpret_cast<uintptr_t>(A.out) & 1) != 0)
    return SS_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < ss_attention_workspace_size())
    return SS_ERR_WORKSPACE;
  AttnArgs a{};
  a.c = view_of(A.cache, A.layer);
  a.t = table_of(A.pool, A.table_rows);
  const int64_t slots = static_cast<int64_t>(A.pool->max_pages) << a.c.page_shift;
  a.table_end = static_cast<int32_t>(slots < 0x7fffffff ? slots : 0x7fffffff);
  a.num_requests = A.num_requests;
  a.num_heads = A.num_heads;
  a.group = A.num_heads / kv_heads;
  uint32_t log2 = 0;
  while ((1 << log2) < a.group) ++log2;
  a.group_mul = static_cast<uint32_t>((1ull << (31 + log2)) / a.group + 1);
  a.group_shift = log2 ? log2 - 1 : 0;
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
  a.scale_log2 = static_cast<float>(static_cast<double>(A.scale) * 1.4426950408889634);
  a.window = A.window;
  a.sinks = A.sinks;
  a.stall = stall;
  a.status = A.out_status;
  // Rows per item: the rows that a request can have, up to what the kernel
  // holds.  More rows per item read the cache fewer times; unused rows cost
  // tensor-core and softmax time (clocks a tile, bf16: 2550 for 8 rows, where the
  // copy bounds it, 2900 for 128; 4 bits: 1390 for 8, 2700 for 64).  8 bits, 64
  // rows against 32: 48 x 1-8 drafts 250 us, 293; 16 trees 125, 164; 2 x 4096
  // prompt 529, 797; a kernel of 128 spills its registers (670 and more).
  const int64_t rows = static_cast<int64_t>(a.max_queries) * a.group;
  const int32_t most = a.c.format == SS_CACHE_BF16 ? 128 : 64;
  a.block_rows = 8;
  while (a.block_rows < rows && a.block_rows < most) a.block_rows *= 2;
  // The most tiles that the table and the numbers of queries allow.
  const int64_t blocks = rows > 0 ? (rows - 1) / a.block_rows + 1 : 0;
  a.extra_tiles = a.c.format == SS_CACHE_FP8 ? kExtra8 : 0;
  a.few_tiles = blocks * (2ll * a.table_end / kTile + 3 + a.extra_tiles) < (1ll << 31) / a.num_requests;
  // (a CTA's share of the tiles of all heads fits 31 bits with 64 SMs or more)
  a.most_tiles = static_cast<int32_t>(kv_heads <= 64 ? 0x7ffffffell : (64ll << 31) / kv_heads);
  a.counters = static_cast<int32_t*>(workspace);
  a.pieces = reinterpret_cast<float*>(a.counters + kMaxCtas);
  a.gave_up = reinterpret_cast<int32_t*>(a.pieces + static_cast<size_t>(kMaxCtas) * 2 * kSlotFloats);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return a.c.format == SS_CACHE_FP8 ? launch_fp8(a, s) : a.c.format == SS_CACHE_INT4 ? launch_int4(a, s) : launch_bf16(a, s);
}

ss_status ss_cache_attention(const ss_attention_args* args, void* workspace, size_t workspace_bytes,
                             ss_stream_t stream) {
  SS_NVTX_RANGE("ss_cache_attention");
  return attention(args, 0, workspace, workspace_bytes, stream);
}

ss_status ss_selftest_attention_timeout(const ss_attention_args* args, int32_t stall, void* workspace,
                                        size_t workspace_bytes, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_selftest_attention_timeout");
  if (stall < SS_STALL_ITEMS || stall > SS_STALL_PACKED) return SS_ERR_INVALID_ARG;
  if (stall == SS_STALL_PACKED && args && args->cache && args->cache->format == SS_CACHE_BF16) return SS_ERR_UNSUPPORTED;
  return attention(args, stall, workspace, workspace_bytes, stream);
}

}  // extern "C"
