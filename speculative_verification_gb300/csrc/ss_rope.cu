// ss_rope.cu -- rotary positions (ss_rope), the same with the cache's append in
// one launch (ss_rope_append), and the append into 8 bits, whose blocks of slots
// are written as a whole.
//
// The mathematics.  A pair (x, y) of a head's channels at position p becomes
// (m (x cos a - y sin a), m (y cos a + x sin a)), a = 2 pi p t.  t is a 64-bit
// fraction of a turn, so p t modulo one turn is one integer product, exact at
// any position.  Its upper 8 bits, rounded, are one of 256 angles A whose sine
// and cosine are tabled in two parts; with the rest d, |d| <= pi / 256, and the
// first terms of its series,
//   cos(A + d) = cos A + (cos A (cos d - 1) - sin A sin d), likewise the sine,
// where what is added is small, so that both come out to 2^-34, as two floats.
// Rotations are fp32 sums of the first.  Those of keys that go into a cache of 8
// or 4 bits take the second too and carry their remainders (2^-32 of magnitude
// (|x| + |y|)), so that they are rounded to fp32, and from there to bf16, as the exact
// sums are: there a unit of bf16 may become a step of the cache (one key in some
// 20,000 is rounded the other way in plain fp32).  It costs 16 registers a thread.
// In 8 bits the rows of a block (16 slots of one head) share a power of two by
// their largest value (ss_rows.cuh).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "ss.h"
#include "ss_cache.h"
#include "ss_nvtx.h"
#include "ss_rows.cuh"

namespace ssc {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / kRowLanes;  // rows in flight per CTA, and tokens of a chunk
constexpr int kNone = -1;                      // no cache: keys go to an array as the queries do
constexpr int kAppend8 = SS_CACHE_FP8;
constexpr int kPairs = 64;

struct StepArgs {
  CacheView c;
  TableView t;
  int32_t max_tokens, total_tokens;
  const int32_t* offsets;
  const int32_t* kv_len;
  const int32_t* parents;
  const int32_t* positions;
  const uint64_t* turns;
  int32_t half, layout;  // pairs; ss_rope_layout
  float magnitude;
  int32_t dim, q_heads, kv_heads, chunk_shift;
  const uint8_t* q;
  uint8_t* q_out;
  const uint8_t* k;
  uint8_t* k_out;
  const uint8_t* v;
  int64_t q_token, q_head, q_out_token, q_out_head;  // bytes
  int64_t k_token, k_head, k_out_token, k_out_head;  // (v's are k's)
  int32_t* status;
};

// Cosines and sines of 2 pi k / 256, as the sum of two floats each.
struct Circle {
  float4 at[256];
  static constexpr double series(double x, double first, int n) {  // sum of (-1)^i x^(2i+n) / (2i+n)!
    double term = first, sum = first;
    for (int i = 1; i < 14; ++i) {
      term *= -x * x / ((2 * i + n) * (2 * i + n - 1));
      sum += term;
    }
    return sum;
  }
  constexpr Circle() : at() {
    for (int k = 0; k < 256; ++k) {
      const int q = (k + 32) / 64, left = k - 64 * q;  // quadrant, and -32 .. 31 of it
      const double x = left * (6.283185307179586 / 256.0);
      const double c = series(x, 1.0, 0), s = series(x, x, 1);
      const double cs = q % 4 == 0 ? c : q % 4 == 1 ? -s : q % 4 == 2 ? -c : s;
      const double sn = q % 4 == 0 ? s : q % 4 == 1 ? c : q % 4 == 2 ? -s : -c;
      at[k].x = static_cast<float>(cs);
      at[k].y = static_cast<float>(cs - static_cast<double>(at[k].x));
      at[k].z = static_cast<float>(sn);
      at[k].w = static_cast<float>(sn - static_cast<double>(at[k].z));
    }
  }
};
__device__ const Circle kCircle = Circle();

// The cosine and sine of a fraction of a turn times a magnitude: each a float
// and what is left of it.
__device__ __forceinline__ void circle(uint64_t turn, float magnitude, float2& c, float2& s) {
  const uint32_t k = static_cast<uint32_t>((turn + (1ull << 55)) >> 56);  // modulo 256
  const int32_t left = static_cast<int32_t>(static_cast<int64_t>(turn - (static_cast<uint64_t>(k) << 56)) >> 24);
  constexpr double kUnit = 6.283185307179586 / 1099511627776.0;  // 2 pi / 2^40
  constexpr float kHigh = static_cast<float>(kUnit), kLow = static_cast<float>(kUnit - static_cast<double>(kHigh));
  const float n = static_cast<float>(left & ~0xff), m = static_cast<float>(left & 0xff), d = __fmul_rn(n, kHigh);
  const float rest = __fmaf_rn(n, kHigh, -d) + __fmaf_rn(n, kLow, m * kHigh);  // the angle less d
  const float d2 = d * d, sd = __fmaf_rn(d * d2, -1.0f / 6.0f, rest), cd = d2 * __fmaf_rn(d2, 1.0f / 24.0f, -0.5f);
  const float4 a = kCircle.at[k & 255u];
  // hi + lo + (first + left of it) d + first sd + hi cd
  const auto sum = [&](float hi, float lo, float first, float first_lo) {
    // (each rounding is said: none of these may be joined with another)
    const float f = __fmul_rn(first, d), h = __fadd_rn(hi, f), t = __fsub_rn(h, hi);
    const float small = __fmaf_rn(first, sd, __fmaf_rn(first_lo, d, __fmaf_rn(hi, cd, lo)));
    const float l =
        __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(h, t)), __fsub_rn(f, t)), __fadd_rn(__fmaf_rn(first, d, -f), small));
    const float p = __fmul_rn(magnitude, h), e = __fmaf_rn(magnitude, l, __fmaf_rn(magnitude, h, -p)), r = __fadd_rn(p, e);
    return make_float2(r, __fsub_rn(e, __fsub_rn(r, p)));
  };
  c = sum(a.x, a.y, -a.z, -a.w);
  s = sum(a.z, a.w, a.x, a.y);
}

// What one lane needs to turn its 8 channels: out = x c + partner s, partner
// the other channel of the pair, s with its sign; two channels at a time.
struct Turn {
  uint64_t c[4], s[4];
  uint32_t on;  // channels that turn
};

__device__ __forceinline__ Turn turn_of(const StepArgs& a, const float* cos_of, const float* sin_of, int lane) {
  Turn t;
  t.on = 0;
  const int c0 = lane * 8, rot = 2 * a.half;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c[2], s[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int ch = c0 + 2 * i + e;
      const bool second = a.layout == SS_ROPE_HALVES ? ch >= a.half : e == 1;
      int pair = a.layout == SS_ROPE_HALVES ? (second ? ch - a.half : ch) : ch >> 1;
      if (ch >= rot) pair = 0;
      c[e] = cos_of[pair];
      s[e] = second ? sin_of[pair] : -sin_of[pair];
      t.on |= static_cast<uint32_t>(ch < rot) << (2 * i + e);
    }
    t.c[i] = two(c[0], c[1]);
    t.s[i] = two(s[0], s[1]);
  }
  return t;
}

// The places of a channel's word in a token's row of what cosines and sines
// leave: a lane's 8 in two reads without conflicts.
__device__ __forceinline__ int low_at(int ch) { return (ch & 4) * 16 + (ch >> 3) * 4 + (ch & 3); }

// One row's 8 channels, turned.  All 16 lanes of the row call it.
// kOdd: pairs that do not come eight by eight (halves of rot_dim not in multiples of
// 8 channels, interleaved ones that end inside a lane's channels).  `row` is the row
// in global memory, read again where lanes' channels do not pair up.
// kClose: sums to 2^-32 of magnitude (|x| + |partner|) before they are rounded, to fp32 and
// to bf16, with `low`, what the floats c and s leave (cosine's below, sine's above in a
// word): these are known to 2^-34.3 of the magnitude, and rounded to bf16 by 2^-33 of it.
template <bool kOdd, bool kClose>
__device__ __forceinline__ uint4 turned(const StepArgs& a, const Turn& t, const uint4& x, const uint8_t* row, int lane,
                                        uint32_t lanes, const uint4* low) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint64_t p[4];
  if (a.layout == SS_ROPE_INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = two(bf16_hi(w[i]), bf16_lo(w[i]));
  } else if (!kOdd) {
    const int other = lane * 8 < a.half ? lane + a.half / 8 : lane - a.half / 8;  // past rot_dim: not used
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = __shfl_sync(lanes, w[i], other, kRowLanes);
      p[i] = two(bf16_lo(y), bf16_hi(y));
    }
  } else {
    const uint16_t* at = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[2] = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ch = lane * 8 + 2 * i + e;
        if (ch < 2 * a.half)
          v[e] = __uint_as_float(static_cast<uint32_t>(at[ch < a.half ? ch + a.half : ch - a.half]) << 16);
      }
      p[i] = two(v[0], v[1]);
    }
    __syncwarp(lanes);  // read before any lane writes the row's place (which may be the row)
  }
  uint32_t o[4];
  bool exact = false;
  if constexpr (kClose) {
    const uint4 l0 = low[lane], l1 = low[lane + kRowLanes];
    const uint32_t l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
    uint64_t all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // sum = a + b of two fp32 numbers, the rounded products: then what the sum took of
      // either (sum - b; the rest) is exact, and with it what is left of v c and p s (of
      // a sum in one fused step, whose bits may end below b's, it is not).  One float at
      // a time: of products and sums of two at once the compiler makes fused steps,
      // whatever their roundings are said to be (fp8 prompt 49.4 us in a graph with such
      // steps, 51.6; 53.4 with two at once and products kept apart by adding a -0 that
      // the compiler does not know, which takes more registers).
      float c[2], s[2], q[2], sum[2], less_a[2], less_b[2];
      split(t.c[i], c[0], c[1]);
      split(t.s[i], s[0], s[1]);
      split(p[i], q[0], q[1]);
      const float x2[2] = {bf16_lo(w[i]), bf16_hi(w[i])};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float b = __fmul_rn(q[e], s[e]);
        sum[e] = __fadd_rn(__fmul_rn(x2[e], c[e]), b);
        less_a[e] = __fsub_rn(b, sum[e]);
        less_b[e] = -__fadd_rn(sum[e], less_a[e]);
      }
      const uint64_t v = two(x2[0], x2[1]);
      // (the sine's low part with the cosine's bits below: rounded with them)
      const uint64_t of_x = fma_2(v, t.c[i], two(less_a[0], less_a[1]));
      const uint64_t of_p = fma_2(p[i], t.s[i], two(less_b[0], less_b[1]));
      const uint64_t left = add_2(fma_2(v, two(bf16_lo(l[2 * i]), bf16_lo(l[2 * i + 1])), of_x),
                                  fma_2(p[i], two(__uint_as_float(l[2 * i]), __uint_as_float(l[2 * i + 1])), of_p));
      all = add_2(all, left);
      float lo, hi;
      split(add_2(two(sum[0], sum[1]), left), lo, hi);
      o[i] = bf16_pair(lo, hi);
    }
    float lo, hi;
    split(all, lo, hi);
    exact = fabsf(lo + hi) < INFINITY;  // else something is not finite, and what is left of it no number
  }
  if (!exact) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      split(fma_2(two(bf16_lo(w[i]), bf16_hi(w[i])), t.c[i], mul_2(p[i], t.s[i])), lo, hi);
      o[i] = bf16_pair(lo, hi);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kOdd) {
      const uint32_t mask = ((t.on >> (2 * i)) & 1u ? 0xffffu : 0u) | ((t.on >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
      o[i] = (o[i] & mask) | (w[i] & ~mask);
    } else if (t.on == 0) {
      o[i] = w[i];
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// CTA (x, r, z): chunk x of request r's tokens (those of 16 slots, of 8 where a
// page has 8), and of their rows each gridDim.z-th.  The sines and cosines of
// the chunk's tokens are computed once, in shared memory; then 16 lanes take a
// token's rows of all heads, whose turns stay in registers.  Rows of 8 bits: 16
// lanes per slot of the block, those that hold rows from before among them.
//
// One cold launch under ncu (whose writes may still be in L2 at its end): 4 x 4096
// tokens, 32 heads on 8, 64 of 128 channels turned: 53 us, loads' latency and 56 % of
// the issue slots; 2 x 4096 tokens into bf16: 39 us, 61 % of the slots (100 to 126
// instructions for two rows).  Without turns, 4 x 2-6k tokens into 8 bits: 21 us, 64 %
// of the slots.  32 trees of 9-48 nodes into 8 bits: 16.8 us, barriers and latency.
// In a graph, the append alone: 2 x 4096 tokens into bf16 38 us, 8 bits 52, 4 bits 60;
// the 32 trees 13.4.  Registers set the CTAs of an SM: four where 64 of them do, three
// with the keys' close sums (80, which already spill), five without turns.
template <int kFormat, bool kRope, bool kOdd>
__global__ void __launch_bounds__(kThreads, kOdd ? 2 : !kRope ? 5 : kFormat > SS_CACHE_BF16 ? 3 : 4) step_kernel(const StepArgs a) {
  constexpr bool kBlocks = kFormat == SS_CACHE_FP8, kClose = kRope && (kBlocks || kFormat == SS_CACHE_INT4);
  constexpr int kEach = 4;
  __shared__ __align__(16) float s_cos[kRope ? kGroups : 1][kPairs], s_sin[kRope ? kGroups : 1][kPairs];
  __shared__ int32_t s_depth[kRope ? SS_TREE_MAX_NODES : 1];
  __shared__ __align__(16) uint32_t s_top[3][2 * kEach];
  __shared__ __align__(16) uint32_t s_low[kClose ? kGroups : 1][2 * kPairs];
  __shared__ uint64_t s_turns[kRope ? kPairs : 1];
  const int tid = threadIdx.x, r = blockIdx.y;
  if (kRope && tid < a.half) s_turns[tid] = a.turns[tid];
  const int32_t begin = a.offsets ? a.offsets[r] : r;
  const int32_t stop = a.offsets ? a.offsets[r + 1] : r + 1;
  const int32_t base = a.kv_len ? a.kv_len[r] : 0;
  const int32_t* row = kFormat == kNone ? nullptr : table_row(a.t, r);
  const int32_t n = stop - begin;
  const bool tree = kRope && a.parents;
  const bool ok = (kFormat == kNone || row) && base >= 0 && begin >= 0 && begin <= stop && stop <= a.total_tokens &&
                  n <= a.max_tokens && !(tree && n > SS_TREE_MAX_NODES);
  if (!ok) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) a.status[r] = SS_ROW_BAD_PARAM;
    return;
  }
  if (blockIdx.x == 0 && blockIdx.z == 0) {  // the status: parents, and does every slot have a page?
    int missing = 0, bad = 0;
    if (kFormat != kNone && n > 0) {
      const int64_t last = (static_cast<int64_t>(base) + n - 1) >> a.c.page_shift;
      for (int64_t e = (base >> a.c.page_shift) + tid; e <= last; e += kThreads)
        missing |= e >= a.t.max_pages || row[e] < 0 || row[e] >= a.c.num_pages;
    }
    if (tree && tid > 0 && tid < n) bad = a.parents[begin + tid] < 0 || a.parents[begin + tid] >= tid;
    if (kFormat != kNone) missing = __syncthreads_or(missing);
    if (tree) bad = __syncthreads_or(bad);
    if (tid == 0) a.status[r] = bad ? SS_ROW_BAD_PARAM : missing ? SS_ROW_BAD_INDEX : SS_ROW_OK;
  }
  // the chunk's tokens t0 .. t1 - 1; its first slot is token `from`
  const int32_t size = 1 << a.chunk_shift;
  const int64_t from = kFormat == kNone ? static_cast<int64_t>(blockIdx.x) << a.chunk_shift
                                        : (((base >> a.chunk_shift) + static_cast<int64_t>(blockIdx.x)) << a.chunk_shift) - base;
  const int32_t t0 = static_cast<int32_t>(from < 0 ? 0 : from < n ? from : n);
  const int32_t t1 = static_cast<int32_t>(from + size < n ? from + size : n);
  const int32_t tokens = t1 - t0;
  if (tokens <= 0) return;
  const int lane = tid % kRowLanes, group = tid / kRowLanes;
  const uint32_t lanes = 0xffffu << (tid & 16);
  const bool live = lane * 8 < a.dim;
  if (kBlocks && tid < 3 * 2 * kEach) (&s_top[0][0])[tid] = 0;
  // rows by themselves (below): 16 lanes have a token's rows first, first + step, ..
  const int per = kGroups / tokens;  // groups of 16 lanes per token
  const int token = group % tokens, first = group / tokens < per ? group / tokens + per * blockIdx.z : 0x3fffffff;
  const int32_t heads = !kRope ? 0 : a.q_heads + (kBlocks ? 0 : kFormat == kNone ? a.kv_heads : 2 * a.kv_heads);
  const int64_t at_row = static_cast<int64_t>(begin) + t0 + token;
  const uint8_t* of_q = a.q + at_row * a.q_token + lane * 16;
  const uint8_t* of_k = a.k + at_row * a.k_token + lane * 16 - a.q_heads * a.k_head;
  const uint8_t* of_v = a.v + at_row * a.k_token + lane * 16 - (a.q_heads + a.kv_heads) * a.k_head;
  const int32_t step = per * gridDim.z;
  const auto source = [&](int32_t h) {
    return (h < a.q_heads ? of_q : h < a.q_heads + a.kv_heads || kFormat == kNone ? of_k : of_v) +
           h * (h < a.q_heads ? a.q_head : a.k_head);
  };
  uint4 x[kEach];
  const auto load = [&](int32_t h0) {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (h0 + e * step < heads && live) x[e] = *reinterpret_cast<const uint4*>(source(h0 + e * step));
  };
#pragma unroll
  for (int e = 0; e < kEach; ++e) x[e] = make_uint4(0u, 0u, 0u, 0u);
  // 8 bits: the block's page
  const int64_t first_slot = base + from;
  const int32_t block_page = kBlocks ? page_of(a.t, a.c, row, first_slot) : -1;  // a block lies in one page
  if constexpr (kRope) {
    load(first);  // on their way while the angles are computed
    if constexpr (kClose && kOdd)  // a lane's channels that do not turn take part in its sums' check
      for (int i = tid; i < kGroups * 2 * kPairs; i += kThreads) (&s_low[0][0])[i] = 0;
    if (tree) {  // depths by jumps of 1, 2, 4 .. parents: a warp, nodes i and i + 32 in lane i
      if (tid < 32) {
        int32_t up[2], depth[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int32_t node = tid + 32 * h, p = node > 0 && node < n ? a.parents[begin + node] : 0;
          up[h] = p < 0 || p >= node ? 0 : p;
          depth[h] = node > 0;
        }
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          int32_t far[2], more[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int32_t u0 = __shfl_sync(0xffffffffu, up[0], up[h] & 31), u1 = __shfl_sync(0xffffffffu, up[1], up[h] & 31);
            const int32_t d0 = __shfl_sync(0xffffffffu, depth[0], up[h] & 31), d1 = __shfl_sync(0xffffffffu, depth[1], up[h] & 31);
            far[h] = up[h] < 32 ? u0 : u1;
            more[h] = up[h] < 32 ? d0 : d1;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            up[h] = far[h];
            depth[h] += more[h];
          }
        }
        s_depth[tid] = depth[0];
        s_depth[tid + 32] = depth[1];
      }
    }
    __syncthreads();
    for (int i = tid; i < tokens * a.half; i += kThreads) {
      const int token = i / a.half, pair = i - token * a.half;
      const int64_t at = a.positions ? a.positions[begin + t0 + token]
                                     : static_cast<int64_t>(base) + (tree ? s_depth[t0 + token] : t0 + token);
      const uint64_t turn = static_cast<uint64_t>(at) * s_turns[pair];
      float2 c, s;
      circle(turn, a.magnitude, c, s);
      s_cos[token][pair] = c.x;
      s_sin[token][pair] = s.x;
      if constexpr (kClose) {
        const int ch = a.layout == SS_ROPE_HALVES ? pair : 2 * pair, partner = a.layout == SS_ROPE_HALVES ? pair + a.half : ch + 1;
        // the cosine's low part as bf16 below; above it what brings the word, as a float, nearest to the sine's
        const uint32_t lower = bf16_pair(c.y, 0.0f), sine = __float_as_uint(s.y);
        const int32_t upper = static_cast<int32_t>(sine & 0x7fffffffu) + 0x8000 - static_cast<int32_t>(lower);
        const uint32_t low = (sine & 0x80000000u) | (static_cast<uint32_t>(max(upper, 0)) & 0x7fff0000u) | lower;
        s_low[token][low_at(ch)] = low ^ 0x80000000u;
        s_low[token][low_at(partner)] = low;
      }
    }
  }
  if (kRope || kBlocks) __syncthreads();

  // ---- rows by themselves: queries, and keys and values but in 8 bits
  if constexpr (kRope) {
    if (first < heads) {
      const Turn t = turn_of(a, s_cos[token], s_sin[token], lane);
      int32_t page = -1, in_page = 0;
      if (kFormat != kNone && !kBlocks) {
        const int64_t slot = static_cast<int64_t>(base) + t0 + token;
        page = page_of(a.t, a.c, row, slot);
        in_page = static_cast<int32_t>(slot) & ((1 << a.c.page_shift) - 1);
      }
      for (int32_t h0 = first;;) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int32_t h = h0 + e * step, k = h - a.q_heads, v = k - a.kv_heads;
          if (h >= heads) break;
          uint4 y = x[e];
          if (kClose && !kBlocks && k >= 0 && v < 0)
            y = turned<kOdd, kClose>(a, t, y, source(h) - lane * 16, lane, lanes,
                                     reinterpret_cast<const uint4*>(s_low[kClose ? token : 0]));
          else if (v < 0)
            y = turned<kOdd, false>(a, t, y, source(h) - lane * 16, lane, lanes, nullptr);
          if (k < 0 || kFormat == kNone) {
            uint8_t* to = k < 0 ? a.q_out + at_row * a.q_out_token + h * a.q_out_head
                                : a.k_out + at_row * a.k_out_token + k * a.k_out_head;
            if (live) *reinterpret_cast<uint4*>(to + lane * 16) = y;
            continue;
          }
          if constexpr (kFormat != kNone && !kBlocks) {
            const int32_t head = v < 0 ? k : v;
            const int64_t cell = max(page, 0) * a.c.page_stride + head * a.c.head_stride + in_page * a.c.slot_stride;
            uint8_t* to = (v < 0 ? a.c.k : a.c.v) + cell;
            if (kFormat == SS_CACHE_INT4) {
              uint32_t pair;
              const uint32_t w = quantise8(y, live, lanes, pair);
              if (page < 0) continue;
              if (live) *reinterpret_cast<uint32_t*>(to + lane * 4) = w;
              if (lane == 0)
                *reinterpret_cast<uint32_t*>((v < 0 ? a.c.ks : a.c.vs) + max(page, 0) * a.c.s_page_stride +
                                             head * a.c.s_head_stride + in_page * 4) = pair;
            } else if (live && page >= 0) {
              *reinterpret_cast<uint4*>(to + lane * 16) = y;
            }
          }
        }
        h0 += step * kEach;
        if (h0 >= heads) break;
        load(h0);
      }
    }
  }

  // ---- a block of 8 bits: 16 lanes per slot, kEach heads of K or V at a time.
  // Bound by instructions: what a batch of heads shares is computed once, the
  // maxima of its heads leave a warp together.
  if constexpr (kBlocks) {
    const int32_t page = block_page;
    if (page < 0) return;
    const int slot = group & (size - 1), side = group >> a.chunk_shift, sides = kGroups >> a.chunk_shift;
    const int64_t i = from + slot;  // the slot's token
    const bool fresh = i >= t0 && i < t1, kept = i < 0, had = from < 0;  // had: some slots hold rows from before
    const int32_t in_page = static_cast<int32_t>(first_slot) & ((1 << a.c.page_shift) - 1);
    const int64_t in_flat = (static_cast<int64_t>(begin) + (fresh ? i : 0)) * a.k_token + lane * 16;
    const int64_t in_cell = page * a.c.page_stride + (in_page + slot) * a.c.slot_stride + lane * 8;
    const int64_t in_scale = page * a.c.s_page_stride + (in_page >> a.chunk_shift) * 4;
    Turn t;
    if constexpr (kRope) t = turn_of(a, s_cos[fresh ? i - t0 : 0], s_sin[fresh ? i - t0 : 0], lane);
    const int32_t batch = sides * kEach, batches = (a.kv_heads + batch - 1) / batch;  // of K, and of V
    int turn = 0;
    for (int32_t n0 = blockIdx.z; n0 < 2 * batches; n0 += gridDim.z, turn = turn == 2 ? 0 : turn + 1) {
      const bool is_v = n0 >= batches;
      const int32_t head0 = (is_v ? n0 - batches : n0) * batch + side * kEach, more = a.kv_heads - head0;  // heads left
      const uint8_t* src = (is_v ? a.v : a.k) + in_flat + head0 * a.k_head;
      uint8_t* cell = (is_v ? a.c.v : a.c.k) + in_cell + head0 * a.c.head_stride;
      float* scale = reinterpret_cast<float*>((is_v ? a.c.vs : a.c.ks) + in_scale + head0 * a.c.s_head_stride);
      const auto scale_of = [&](int e) {
        return reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(scale) + e * a.c.s_head_stride);
      };
      float old[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        x[e] = make_uint4(0u, 0u, 0u, 0u);
        if (fresh && live && e < more) x[e] = *reinterpret_cast<const uint4*>(src + e * a.k_head);
      }
      if (had) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          old[e] = 0.0f;
          if (kept && live && e < more) {
            const uint2 w = *reinterpret_cast<const uint2*>(cell + e * a.c.head_stride);
            x[e].x = w.x;
            x[e].y = w.y;
            old[e] = *scale_of(e);
          }
        }
      }
      if constexpr (kRope)
        if (fresh && !is_v) {
#pragma unroll
          for (int e = 0; e < kEach; ++e)
            if (e < more)
              x[e] = turned<kOdd, kClose>(a, t, x[e], src - lane * 16 + e * a.k_head, lane, lanes,
                                          reinterpret_cast<const uint4*>(s_low[i - t0]));
        }
      uint32_t top[kEach], most = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        top[e] = magnitude(x[e]) << 16;
        if (!kept) most = max(most, top[e]);
      }
      const bool odd = most >= 0x7f800000u;  // a value is not finite
      if (had || odd) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          float f[8];
          if (kept) decode8(make_uint2(x[e].x, x[e].y), old[e], f);
          else floats_of(x[e], f);
          top[e] = __float_as_uint(finite_top(f));
        }
      }
      __syncwarp();
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, top[e]);
        if ((tid & 31) == e) mine = m;
      }
      if ((tid & 31) < kEach && mine != 0) atomicMax(&s_top[turn][side * kEach + (tid & 31)], mine);
      const bool slow = __syncthreads_or(odd) || had;
      const uint4 tops = *reinterpret_cast<const uint4*>(&s_top[turn][side * kEach]);
      const Scale8 to[kEach] = {scale8(__uint_as_float(tops.x)), scale8(__uint_as_float(tops.y)),
                                scale8(__uint_as_float(tops.z)), scale8(__uint_as_float(tops.w))};
      const bool row_here = live && (fresh || kept);
      if (!slow) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const uint2 w = encode8(x[e], to[e].inv);
          if (row_here && e < more) *reinterpret_cast<uint2*>(cell + e * a.c.head_stride) = w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          float f[8];
          if (kept) decode8(make_uint2(x[e].x, x[e].y), old[e], f);
          else floats_of(x[e], f);
          const uint2 w = encode8(f, to[e].inv);
          if (row_here && e < more) *reinterpret_cast<uint2*>(cell + e * a.c.head_stride) = w;
        }
      }
      if (lane == 0 && i == t1 - 1) {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          if (e < more) *scale_of(e) = to[e].s;
      }
      // the batch before's maxima were read before this batch's barrier; they are needed again in two batches
      if (tid < 2 * kEach) s_top[turn == 0 ? 2 : turn - 1][tid] = 0;
    }
  }
}

// ------------------------------------------------------------------- host --

static bool aligned_strides(std::initializer_list<int64_t> strides) {
  for (int64_t s : strides)
    if ((s & 7) != 0) return false;
  return true;
}

static bool check_table_of_turns(const ss_rope_table* t, int32_t dim) {
  return t && t->turns && (reinterpret_cast<uintptr_t>(t->turns) & 7u) == 0 && t->rot_dim >= 2 && (t->rot_dim & 1) == 0 &&
         t->rot_dim <= dim && (t->layout == SS_ROPE_HALVES || t->layout == SS_ROPE_INTERLEAVED) && isfinite(t->magnitude);
}

static void take_rope(StepArgs* a, const ss_rope_table* t) {
  a->turns = t->turns;
  a->half = t->rot_dim / 2;
  a->layout = t->layout;
  a->magnitude = t->magnitude;
}

// As many CTAs per chunk as give every SM `each` of them, up to one for every four rows of
// a token.  Three or four an SM: with keys and values that are encoded, whose CTAs
// are longer, four (in a graph, 2 x 4096 tokens into 8 bits 51.7 us, 55.5 with three; 4
// bits 59.5 and 68.0; 32 trees into 8 bits 13.4 and 13.8); else three, as each computes
// the angles again (bf16 39.5 with four and 37.8, half as many tokens 22.7 and 20.5).
static unsigned splits(int64_t chunks, int64_t rows, int64_t each) {
  const int64_t spare = (each * 152 + chunks - 1) / chunks, most = rows < 4 ? 1 : rows / 4;
  const int64_t z = spare < most ? spare : most;
  return static_cast<unsigned>(z < 1 ? 1 : z > 64 ? 64 : z);
}

template <int kFormat, bool kRope>
static ss_status launch_step(const StepArgs& a, int32_t num_requests, cudaStream_t s) {
  const int64_t size = 1ll << a.chunk_shift;
  // n tokens touch at most ceil((n + size - 1) / size) blocks of slots
  const int64_t n = a.max_tokens < a.total_tokens ? a.max_tokens : a.total_tokens;  // a generous max_tokens costs nothing
  const int64_t x = kFormat == kNone ? (n + size - 1) / size : (n + 2 * size - 2) / size;
  const int64_t rows = a.q_heads + (kFormat == kNone ? 1ll : 2ll) * a.kv_heads;
  const int64_t wide = x < 1 ? 1 : x;
  const dim3 grid(static_cast<unsigned>(wide), num_requests, splits(wide * num_requests, rows, kFormat > SS_CACHE_BF16 ? 4 : 3));
  if constexpr (kRope) {
    if (a.half % (a.layout == SS_ROPE_HALVES ? 8 : 4) != 0) {
      step_kernel<kFormat, true, true><<<grid, kThreads, 0, s>>>(a);
      return finish(cudaSuccess);
    }
  }
  step_kernel<kFormat, kRope, false><<<grid, kThreads, 0, s>>>(a);
  return finish(cudaSuccess);
}

static void take_append(StepArgs* a, const ss_append_args& A) {
  a->c = view_of(A.cache, A.layer);
  a->t = table_of(A.pool, A.table_rows);
  a->max_tokens = A.token_offsets ? A.max_tokens : 1;
  a->total_tokens = A.total_tokens;
  a->offsets = A.token_offsets;
  a->kv_len = A.kv_len;
  a->dim = a->c.dim;
  a->kv_heads = a->c.heads;
  a->chunk_shift = a->c.format == SS_CACHE_FP8 ? a->c.block_shift : 4;
  a->k = static_cast<const uint8_t*>(A.k);
  a->v = static_cast<const uint8_t*>(A.v);
  a->k_token = A.token_stride * 2;
  a->k_head = A.head_stride * 2;
  a->status = A.out_status;
}

ss_status append_blocks(const ss_append_args* args, cudaStream_t s) {
  const ss_status checked = check_append(args);
  if (checked != SS_OK || args->num_requests == 0) return checked;
  StepArgs a{};
  take_append(&a, *args);
  return launch_step<kAppend8, false>(a, args->num_requests, s);
}

}  // namespace ssc

extern "C" {

ss_status ss_rope_turns(int32_t rot_dim, double base, int32_t scaling, double factor, double length, double low,
                        double high, uint64_t* turns) {
  SS_NVTX_RANGE("ss_rope_turns");
  if (!turns || rot_dim < 2 || rot_dim > 128 || (rot_dim & 1) != 0 || !isfinite(base) || !(base > 0.0))
    return SS_ERR_INVALID_ARG;
  if (scaling != SS_ROPE_PLAIN && scaling != SS_ROPE_LINEAR && scaling != SS_ROPE_BY_PARTS) return SS_ERR_INVALID_ARG;
  if (scaling != SS_ROPE_PLAIN && (!isfinite(factor) || !(factor > 0.0))) return SS_ERR_INVALID_ARG;
  if (scaling == SS_ROPE_BY_PARTS && (!isfinite(length) || !(length > 0.0) || !isfinite(high) || !(low >= 0.0) || !(high > low)))
    return SS_ERR_INVALID_ARG;
  constexpr double kTau = 6.283185307179586;
  uint64_t out[64];
  for (int32_t i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == SS_ROPE_LINEAR) f /= factor;
    if (scaling == SS_ROPE_BY_PARTS) {
      double g = (length * f / kTau - low) / (high - low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = f * g + f / factor * (1.0 - g);
    }
    const double turn = f / kTau;  // of which a position is at most half
    if (!(turn <= 0.5)) return SS_ERR_INVALID_ARG;
    out[i] = static_cast<uint64_t>(ldexp(turn, 64) + 0.5);
  }
  for (int32_t i = 0; i < rot_dim / 2; ++i) turns[i] = out[i];
  return SS_OK;
}

ss_status ss_rope(const ss_rope_args* args, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_rope");
  using namespace ssc;
  if (!args) return SS_ERR_INVALID_ARG;
  const ss_rope_args& A = *args;
  if (A.head_dim < 8 || A.head_dim > 128 || A.head_dim % 8 != 0 || !check_table_of_turns(A.rope, A.head_dim) ||
      A.num_requests < 0 || A.num_requests > 65535 || A.max_tokens < 0 || A.total_tokens < 0 || A.num_heads < 0 ||
      A.num_heads > 65535 || A.num_kv_heads < 0 || A.num_kv_heads > 65535 || (A.parents && A.positions))
    return SS_ERR_INVALID_ARG;
  if (!A.token_offsets && A.total_tokens < A.num_requests) return SS_ERR_INVALID_ARG;
  if (A.num_requests == 0) return SS_OK;
  const bool any = A.total_tokens > 0;
  if ((!A.kv_len && !A.positions) || !A.out_status || (any && A.num_heads > 0 && A.q && !A.q_out) ||
      (any && A.num_kv_heads > 0 && A.k && !A.k_out) || !aligned16(A.q) || !aligned16(A.q_out) || !aligned16(A.k) ||
      !aligned16(A.k_out) ||
      !aligned_strides({A.q_token_stride, A.q_head_stride, A.q_out_token_stride, A.q_out_head_stride, A.k_token_stride,
                        A.k_head_stride, A.k_out_token_stride, A.k_out_head_stride}))
    return SS_ERR_INVALID_ARG;
  StepArgs a{};
  take_rope(&a, A.rope);
  a.max_tokens = A.token_offsets ? A.max_tokens : 1;
  a.total_tokens = A.total_tokens;
  a.offsets = A.token_offsets;
  a.kv_len = A.positions ? nullptr : A.kv_len;
  a.parents = A.parents;
  a.positions = A.positions;
  a.dim = A.head_dim;
  a.q_heads = A.q ? A.num_heads : 0;
  a.kv_heads = A.k ? A.num_kv_heads : 0;
  a.chunk_shift = 4;
  a.q = static_cast<const uint8_t*>(A.q);
  a.q_out = static_cast<uint8_t*>(A.q_out);
  a.k = static_cast<const uint8_t*>(A.k);
  a.k_out = static_cast<uint8_t*>(A.k_out);
  a.q_token = A.q_token_stride * 2;
  a.q_head = A.q_head_stride * 2;
  a.q_out_token = A.q_out_token_stride * 2;
  a.q_out_head = A.q_out_head_stride * 2;
  a.k_token = A.k_token_stride * 2;
  a.k_head = A.k_head_stride * 2;
  a.k_out_token = A.k_out_token_stride * 2;
  a.k_out_head = A.k_out_head_stride * 2;
  a.status = A.out_status;
  return launch_step<kNone, true>(a, A.num_requests, reinterpret_cast<cudaStream_t>(stream));
}

ss_status ss_rope_append(const ss_rope_append_args* args, ss_stream_t stream) {
  SS_NVTX_RANGE("ss_rope_append");
  using namespace ssc;
  if (!args) return SS_ERR_INVALID_ARG;
  const ss_status checked = check_append(args->append);
  if (checked != SS_OK) return checked;
  const ss_rope_append_args& A = *args;
  const ss_append_args& B = *A.append;
  if (!check_table_of_turns(A.rope, B.cache->head_dim) || A.num_heads < 0 || A.num_heads > 65535 || (A.parents && A.positions))
    return SS_ERR_INVALID_ARG;
  if (B.num_requests == 0) return SS_OK;
  if ((B.total_tokens > 0 && A.num_heads > 0 && (!A.q || !A.q_out)) || !aligned16(A.q) || !aligned16(A.q_out) ||
      !aligned_strides({A.q_token_stride, A.q_head_stride, A.q_out_token_stride, A.q_out_head_stride}))
    return SS_ERR_INVALID_ARG;
  StepArgs a{};
  take_append(&a, B);
  take_rope(&a, A.rope);
  a.parents = A.parents;
  a.positions = A.positions;
  a.q_heads = A.num_heads;
  a.q = static_cast<const uint8_t*>(A.q);
  a.q_out = static_cast<uint8_t*>(A.q_out);
  a.q_token = A.q_token_stride * 2;
  a.q_head = A.q_head_stride * 2;
  a.q_out_token = A.q_out_token_stride * 2;
  a.q_out_head = A.q_out_head_stride * 2;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (a.c.format) {
    case SS_CACHE_BF16: return launch_step<SS_CACHE_BF16, true>(a, B.num_requests, s);
    case SS_CACHE_INT4: return launch_step<SS_CACHE_INT4, true>(a, B.num_requests, s);
    default: return launch_step<SS_CACHE_FP8, true>(a, B.num_requests, s);
  }
}

}  // extern "C"
