// ss_attn_fp8.cu -- the attention kernel (ss_attn.cuh) for 8-bit caches.
#include "ss_attn.cuh"

namespace ssa {

template <int kHalves>
static ss_status pick(const AttnArgs& a, cudaStream_t s) {
  switch (a.block_rows) {
    case 8: return launch<8, true, kHalves, true>(a, s);
    case 16: return launch<16, true, kHalves, true>(a, s);
    case 32: return launch<32, true, kHalves, true>(a, s);
    default: return launch<64, true, kHalves, true>(a, s);
  }
}

ss_status launch_fp8(const AttnArgs& a, cudaStream_t s) { return a.c.dim <= 64 ? pick<1>(a, s) : pick<2>(a, s); }

}  // namespace ssa
