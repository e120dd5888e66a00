// ss_attn_bf16.cu -- the attention kernel (ss_attn.cuh) for bf16 caches.
#include "ss_attn.cuh"

namespace ssa {

template <int kHalves>
static ss_status pick(const AttnArgs& a, cudaStream_t s) {
  switch (a.block_rows) {
    case 8: return launch<8, false, kHalves>(a, s);
    case 16: return launch<16, false, kHalves>(a, s);
    case 32: return launch<32, false, kHalves>(a, s);
    case 64: return launch<64, false, kHalves>(a, s);
    default: return launch<128, false, kHalves>(a, s);
  }
}

ss_status launch_bf16(const AttnArgs& a, cudaStream_t s) { return a.c.dim <= 64 ? pick<1>(a, s) : pick<2>(a, s); }

}  // namespace ssa
