// Tensor-core cross-decoder attention over an e2m1 cache ("KV cache memory
// systems", "Quantized cache changes attention inputs"): instantiations of
// the kernels in attn_tc.cuh with half-byte pages and a scale byte for every
// 32 head dims of a token.
#include "attn_tc.cuh"

namespace yoco {

cudaError_t launch_attn_tc_e2m1(const CUtensorMap& mk, const CUtensorMap& mv,
                                const AttnParams& p, int D, int BS, int sms, cudaStream_t s) {
    if (D == 128) return launch_d<128, kE2m1>(mk, mv, p, BS, sms, s);
    return launch_d<256, kE2m1>(mk, mv, p, BS, sms, s);
}

}  // namespace yoco
