// Tensor-core cross-decoder attention over an e2m1 cache ("KV cache memory
// systems", "Quantized cache changes attention inputs"): instantiations of
// the kernels in attn_tc.cuh with half-byte pages and a scale byte for every
// 32 head dims of a token.
//
// What bounds them. The cache is 17/64 of a bf16 one's bytes, and so few that
// the work on a key, not its bytes, sets the time: widening codes to f16 (62
// lanes a clock and SM for a pair of codes), scaling scores and weights, and
// the products. us a layer, in a graph of layers, beside the time of its bytes
// at 6.80 TB/s:
//   64 requests of 1024..8192 keys, 8 query and 2 kv heads of 256:
//                           16-token blocks 47.0 (23.7), 32-token blocks 40.0
//   the same at head_dim 128                32.3 (11.9)
//   the same (256) with 4 rows a request   110.9 (24.0)
//   4 of 131072 keys, 16 heads on one of 128, 32-token blocks  37.4 (10.5)
// About 8 us of each are start and finish (plan, first page, joining pieces:
// 3 requests of a few keys take 8.9). Copies alone took 34 us of the first and
// 19.5 of the last, work on pages already there 45 and 36: the walk is bound by
// its instructions' latency at the warps that the accumulators' registers
// leave (issue slots 39% and 30% taken, tensor cores 17%, DRAM 39% and 21%).
// Tried without gain: more and fewer warps, two-page steps at head_dim 256,
// queries in shared memory for 16 columns (39.4 -> 40.2), products of two
// blocks interleaved.
#include "attn_tc.cuh"

namespace yoco {

cudaError_t launch_attn_tc_e2m1(const CUtensorMap& mk, const CUtensorMap& mv,
                                const AttnParams& p, int D, int BS, int sms, cudaStream_t s) {
    if (D == 128) return launch_d<128, kE2m1>(mk, mv, p, BS, sms, s);
    return launch_d<256, kE2m1>(mk, mv, p, BS, sms, s);
}

}  // namespace yoco
