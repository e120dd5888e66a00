// ss_cache.h -- internal: the paged cache as the kernels see it, and the host
// checks of the structs that describe it.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss.h"

namespace ss {

void set_last_cuda_error(int32_t e);  // ss_kernel.cu: the value ss_last_cuda_error() reports

// ss_kv_cache with the layer's base pointers and the page size as a shift.
struct CacheView {
  int32_t format, num_pages, heads, dim, page_shift;
  int32_t block_shift;  // 8 bits: slots that share a scale
  uint8_t* k;
  uint8_t* v;
  int64_t layer_stride, page_stride, head_stride, slot_stride;
  uint8_t* ks;
  uint8_t* vs;
  int64_t s_layer_stride, s_page_stride, s_head_stride;
};

// The table rows of a call's requests.
struct TableView {
  const int32_t* entries;
  const int32_t* rows;  // [num_requests] or NULL
  int64_t stride;
  int32_t num_rows, max_pages;
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes of one row of one head (without its scales).
__host__ __device__ inline int32_t row_bytes(int32_t format, int32_t dim) {
  return format == SS_CACHE_INT4 ? dim / 2 : format == SS_CACHE_FP8 ? dim : 2 * dim;
}

inline bool check_cache(const ss_kv_cache* c) {
  if (!c) return false;
  if (c->format != SS_CACHE_BF16 && c->format != SS_CACHE_INT4 && c->format != SS_CACHE_FP8) return false;
  if (c->num_layers < 1 || c->num_pages < 1 || c->num_kv_heads < 1 || c->num_kv_heads > 65535) return false;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return false;
  const bool packed = c->format == SS_CACHE_INT4, bytes = c->format == SS_CACHE_FP8;
  const int32_t unit = packed ? 32 : bytes ? 16 : 8;
  if (c->head_dim < unit || c->head_dim > 128 || c->head_dim % unit != 0) return false;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return false;
  const int64_t row = row_bytes(c->format, c->head_dim);
  // a tensor copy's strides are multiples of 16 bytes below 2^40
  for (int64_t s : {c->layer_stride, c->page_stride, c->head_stride, c->slot_stride})
    if (s < row || (s & 15) != 0 || s >= (1ll << 40)) return false;
  if (packed) {
    if (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)) return false;
    for (int64_t s : {c->scale_layer_stride, c->scale_page_stride, c->scale_head_stride})
      if (s < 4ll * c->page_size || (s & 15) != 0 || s >= (1ll << 40)) return false;
  }
  if (bytes) {
    if (!c->k_scale || !c->v_scale || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) != 0)
      return false;
    const int64_t page = 4ll * (c->page_size < SS_FP8_BLOCK ? 1 : c->page_size / SS_FP8_BLOCK);
    for (int64_t s : {c->scale_layer_stride, c->scale_page_stride, c->scale_head_stride})
      if (s < page || (s & 3) != 0 || s >= (1ll << 40)) return false;
  }
  return true;
}

inline bool check_table(const ss_page_pool* p) {
  return p && p->page_table && p->num_rows >= 1 && p->max_pages >= 1 && p->row_stride >= p->max_pages;
}

inline CacheView view_of(const ss_kv_cache* c, int32_t layer) {
  CacheView v{};
  v.format = c->format;
  v.num_pages = c->num_pages;
  v.heads = c->num_kv_heads;
  v.dim = c->head_dim;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  v.k = static_cast<uint8_t*>(c->k) + layer * c->layer_stride;
  v.v = static_cast<uint8_t*>(c->v) + layer * c->layer_stride;
  v.layer_stride = c->layer_stride;
  v.page_stride = c->page_stride;
  v.head_stride = c->head_stride;
  v.slot_stride = c->slot_stride;
  v.block_shift = v.page_shift < 4 ? v.page_shift : 4;  // SS_FP8_BLOCK, or a page of 8
  if (c->format != SS_CACHE_BF16) {
    v.ks = static_cast<uint8_t*>(c->k_scale) + layer * c->scale_layer_stride;
    v.vs = static_cast<uint8_t*>(c->v_scale) + layer * c->scale_layer_stride;
    v.s_layer_stride = c->scale_layer_stride;
    v.s_page_stride = c->scale_page_stride;
    v.s_head_stride = c->scale_head_stride;
  }
  return v;
}

inline TableView table_of(const ss_page_pool* p, const int32_t* rows) {
  TableView t{};
  t.entries = p->page_table;
  t.rows = rows;
  t.stride = p->row_stride;
  t.num_rows = p->num_rows;
  t.max_pages = p->max_pages;
  return t;
}

}  // namespace ss

namespace ssc {
ss_status check_append(const ss_append_args* args);  // ss_cache.cu: the append and read calls' arguments
ss_status append_blocks(const ss_append_args* args, cudaStream_t s);  // ss_rope.cu: ss_cache_append into 8 bits
}  // namespace ssc

namespace ss {

inline ss_status finish(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return SS_OK;
  set_last_cuda_error(static_cast<int32_t>(e));
  return SS_ERR_CUDA;
}

#ifdef __CUDACC__

// The table row of request r, or NULL when it lies outside the table.
__device__ __forceinline__ const int32_t* table_row(const TableView& t, int32_t r) {
  const int32_t row = t.rows ? t.rows[r] : r;
  return (row < 0 || row >= t.num_rows) ? nullptr : t.entries + row * t.stride;
}

// The page that holds slot number `slot`, or -1.
__device__ __forceinline__ int32_t page_of(const TableView& t, const CacheView& c, const int32_t* row, int64_t slot) {
  const int64_t e = slot >> c.page_shift;
  if (e >= t.max_pages) return -1;
  const int32_t p = row[e];
  return (p < 0 || p >= c.num_pages) ? -1 : p;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values as a bf16 pair (round to nearest even; a in the low half).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Two fp32 operations in one instruction.  A mul_2 and an add_2 behind it become one
// fused step, in spite of their .rn: where each has to round, use __fmul_rn and
// __fadd_rn, which stay apart.
__device__ __forceinline__ uint64_t two(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ uint64_t add_2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& a, float& b) {
  a = __uint_as_float(static_cast<uint32_t>(v));
  b = __uint_as_float(static_cast<uint32_t>(v >> 32));
}

#endif  // __CUDACC__

}  // namespace ss
