// The 4-bit cache's rows: yoco_kv_append_e2m1 writes a step's new K^/V^ as
// e2m1 codes with one power-of-two scale for 32 head dims of a token, and
// yoco_kv_gather_e2m1 reads rows back as the bf16 values they stand for.
//
// "KV cache memory systems", "Quantized cache changes attention inputs": a
// quantized cache cuts the bytes per cached scalar and adds scale metadata.
//
// Format (the OCP microscaling block of 32 e2m1 elements): code = sign, two
// exponent bits, one mantissa bit (0, 0.5, 1, 1.5, 2, 3, 4, 6); a block's
// scale is 2^(b - 127), b one byte, here the smallest with every magnitude of
// the block at most 6 of it. A power of two divides exactly, so the code is
// the only rounding, and code * scale is a bf16 value exactly.
//
// Design: both move bytes, bound by HBM: 2 + 17/32 bytes an element. One warp
// per token strides over the token's rows of all kv heads, 8 elements (16
// bytes of bf16) a lane, so that 4 lanes hold a block and its largest
// magnitude takes two shuffles. K and V go together, two vectors of each in
// flight a lane. Replayed from a graph, 23900 tokens of 2 kv heads of 256
// (new rows 49 MB, codes and scales 13 MB): append 14.1 us, 4.4 TB/s, gather
// 8.8 us, 7.0 TB/s with the pages in L2 (cold they take 17 and 12.5); issue
// slots are 46% and 44% taken there, DRAM 36% and 14%, so append sits between
// the two. 64 tokens: 2.5 and 2.1 us, the launch.
#include "common.cuh"

namespace yoco {
namespace {

constexpr int kRowWarps = 8;

// Eight bf16 values with infinities and NaN as the largest finite value of
// their sign; returns the largest magnitude, as a bf16 bit pattern.
__device__ __forceinline__ uint32_t finite8(uint4& a) {
    uint32_t* w = &a.x;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t mag = __vminu2(w[i] & 0x7fff7fffu, 0x7f7f7f7fu);
        m = __vmaxu2(m, mag);
        w[i] = mag | (w[i] & 0x80008000u);
    }
    return max(m & 0xffffu, m >> 16);
}

// Scale byte of a block whose largest magnitude has these bf16 bits: the
// smallest b with magnitude <= 6 * 2^(b - 127). 6 = 1.5 * 2^2, so the
// exponent moves by one where the mantissa is above 1.5.
__device__ __forceinline__ int32_t scale_byte(uint32_t mag) {
    const int32_t e = static_cast<int32_t>(mag >> 7) - 2 + ((mag & 0x7fu) > 0x40u ? 1 : 0);
    return min(max(e, 1), 251);
}

__device__ __forceinline__ uint32_t e2m1x2_rn_sat(float lo, float hi) {
    uint32_t r;
    asm("{ .reg .b8 c; cvt.rn.satfinite.e2m1x2.f32 c, %1, %2; cvt.u32.u8 %0, c; }"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Eight finite bf16 values -> eight codes of value * inv (inv the power of two 1 / scale).
__device__ __forceinline__ uint32_t quantise8_e2m1(uint4 a, float inv) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e2m1x2_rn_sat(bf16lo_to_f32(w[i]) * inv, bf16hi_to_f32(w[i]) * inv);
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// Codes and scale byte of this lane's eight elements; the four lanes of a
// block (lane & ~3) agree on the byte. All lanes of the warp take part.
__device__ __forceinline__ void encode8(uint4 a, uint32_t& codes, int32_t& b) {
    uint32_t m = finite8(a);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    b = scale_byte(m);
    codes = quantise8_e2m1(a, __uint_as_float(static_cast<uint32_t>(254 - b) << 23));
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv_append_e2m1_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                          uint32_t* __restrict__ k_cache, uint32_t* __restrict__ v_cache,
                          uint8_t* __restrict__ scales, const int32_t* __restrict__ slots,
                          int32_t num_tokens, int64_t num_slots, int32_t bshift,
                          int32_t num_kv_heads, int32_t* err) {
    constexpr int RV = D / 8;                  // 8-element vectors of a row
    constexpr int RSH = D == 128 ? 4 : 5;
    constexpr int U = 2;
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const int64_t wstride = static_cast<int64_t>(gridDim.x) * kRowWarps;
    const int32_t nvec = num_kv_heads * RV, bs = 1 << bshift;
    for (int64_t tok = warp0; tok < num_tokens; tok += wstride) {
        const int64_t slot = __ldg(slots + tok);
        if (slot < 0) continue;  // padding
        if (slot >= num_slots) {
            if (lane == 0) set_err(err, YOCO_DEVERR_PAGE_RANGE);
            continue;
        }
        const int64_t page0 = (slot >> bshift) * num_kv_heads;
        const int32_t in_page = static_cast<int32_t>(slot) & (bs - 1);
        const uint4* ks = k_new + tok * nvec;
        const uint4* vs = v_new + tok * nvec;
        for (int32_t v0 = lane; v0 - lane < nvec; v0 += 32 * U) {
            uint4 kr[U], vr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t v = v0 + u * 32;
                kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
                if (v < nvec) {
                    kr[u] = __ldcs(ks + v);  // read once: stream past L1/L2
                    vr[u] = __ldcs(vs + v);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t v = v0 + u * 32;
                uint32_t kc, vc;
                int32_t kb, vb;
                encode8(kr[u], kc, kb);
                encode8(vr[u], vc, vb);
                if (v < nvec) {
                    const int64_t ph = page0 + (v >> RSH);  // (page, kv head)
                    const int32_t j = v & (RV - 1);
                    const int64_t d = (ph * bs + in_page) * RV + j;
                    k_cache[d] = kc;
                    v_cache[d] = vc;
                    if ((lane & 3) == 0) {
                        uint8_t* s = scales + (ph * 2 * bs + in_page) * (D / 32) + (j >> 2);
                        s[0] = static_cast<uint8_t>(kb);
                        s[bs * (D / 32)] = static_cast<uint8_t>(vb);
                    }
                }
            }
        }
    }
}

// Eight codes of a block with scale byte b as bf16 values (exact).
__device__ __forceinline__ uint4 decode8_bf16(uint32_t codes, uint32_t b) {
    uint32_t h[4];
    e2m1x8_to_f16x2(codes, h[0], h[1], h[2], h[3]);
    const float s = __uint_as_float(b << 23);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(f16lo_to_f32(h[i]) * s, f16hi_to_f32(h[i]) * s);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32)
    kv_gather_e2m1_kernel(const uint32_t* __restrict__ k_cache,
                          const uint32_t* __restrict__ v_cache, const uint8_t* __restrict__ scales,
                          const int32_t* __restrict__ slots, uint4* __restrict__ k_out,
                          uint4* __restrict__ v_out, int32_t num_tokens, int64_t num_slots,
                          int32_t bshift, int32_t num_kv_heads, int32_t* err) {
    constexpr int RV = D / 8;
    constexpr int RSH = D == 128 ? 4 : 5;
    constexpr int U = 2;
    const int lane = threadIdx.x & 31;
    const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    const int64_t wstride = static_cast<int64_t>(gridDim.x) * kRowWarps;
    const int32_t nvec = num_kv_heads * RV, bs = 1 << bshift;
    for (int64_t tok = warp0; tok < num_tokens; tok += wstride) {
        const int64_t slot = __ldg(slots + tok);
        const bool there = slot >= 0 && slot < num_slots;
        if (slot >= num_slots && lane == 0) set_err(err, YOCO_DEVERR_PAGE_RANGE);
        const int64_t page0 = there ? (slot >> bshift) * num_kv_heads : 0;
        const int32_t in_page = static_cast<int32_t>(slot) & (bs - 1);
        for (int32_t v0 = lane; v0 < nvec; v0 += 32 * U) {
            uint32_t kc[U], vc[U], kb[U], vb[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t v = v0 + u * 32;
                kc[u] = vc[u] = kb[u] = vb[u] = 0u;
                if (v < nvec && there) {
                    const int64_t ph = page0 + (v >> RSH);
                    const int32_t j = v & (RV - 1);
                    const int64_t d = (ph * bs + in_page) * RV + j;
                    const uint8_t* s = scales + (ph * 2 * bs + in_page) * (D / 32) + (j >> 2);
                    kc[u] = __ldcs(k_cache + d);
                    vc[u] = __ldcs(v_cache + d);
                    kb[u] = s[0];
                    vb[u] = s[bs * (D / 32)];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t v = v0 + u * 32;
                if (v < nvec) {
                    k_out[tok * nvec + v] = decode8_bf16(kc[u], kb[u]);
                    v_out[tok * nvec + v] = decode8_bf16(vc[u], vb[u]);
                }
            }
        }
    }
}

// Checks shared by the two calls. Returns YOCO_OK and `launch` when there is work.
yoco_status_t check_rows(const void* a, const void* b, const void* k, const void* v,
                         const void* scales, const int32_t* slots, int32_t num_tokens,
                         int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                         int32_t head_dim, bool& launch) {
    launch = false;
    if ((head_dim != 128 && head_dim != 256) || !block_size_ok(block_size))
        return YOCO_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_blocks <= 0 || num_kv_heads <= 0) return YOCO_ERR_INVALID_ARG;
    // slots are int32, a token's vectors are counted in one
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7fffffffll ||
        num_kv_heads > 0x7fffffff / 64)
        return YOCO_ERR_UNSUPPORTED;
    if (num_tokens == 0) return YOCO_OK;
    if (!a || !b || !k || !v || !scales || !slots) return YOCO_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(b) || !aligned16(k) || !aligned16(v) || !aligned16(scales))
        return YOCO_ERR_INVALID_ARG;
    launch = true;
    return YOCO_OK;
}

unsigned row_blocks(int32_t num_tokens) {
    const int64_t blocks = (static_cast<int64_t>(num_tokens) + kRowWarps - 1) / kRowWarps;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 16;
    return static_cast<unsigned>(blocks < cap ? blocks : cap);
}

}  // namespace
}  // namespace yoco

extern "C" yoco_status_t yoco_kv_append_e2m1(const void* k_new, const void* v_new, void* k_cache,
                                             void* v_cache, void* block_scales,
                                             const int32_t* slot_mapping, int32_t num_tokens,
                                             int32_t num_blocks, int32_t block_size,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             int32_t* err_word, void* stream) {
    using namespace yoco;
    bool launch;
    const yoco_status_t st = check_rows(k_new, v_new, k_cache, v_cache, block_scales, slot_mapping,
                                        num_tokens, num_blocks, block_size, num_kv_heads, head_dim,
                                        launch);
    if (!launch) return st;
    auto* kernel = head_dim == 128 ? kv_append_e2m1_kernel<128> : kv_append_e2m1_kernel<256>;
    kernel<<<row_blocks(num_tokens), kRowWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new),
        static_cast<uint32_t*>(k_cache), static_cast<uint32_t*>(v_cache),
        static_cast<uint8_t*>(block_scales), slot_mapping, num_tokens,
        static_cast<int64_t>(num_blocks) * block_size, block_size == 16 ? 4 : 5, num_kv_heads,
        err_word);
    return cuda_status(cudaGetLastError());
}

extern "C" yoco_status_t yoco_kv_gather_e2m1(const void* k_cache, const void* v_cache,
                                             const void* block_scales, const int32_t* slot_mapping,
                                             void* k_out, void* v_out, int32_t num_tokens,
                                             int32_t num_blocks, int32_t block_size,
                                             int32_t num_kv_heads, int32_t head_dim,
                                             int32_t* err_word, void* stream) {
    using namespace yoco;
    bool launch;
    const yoco_status_t st = check_rows(k_out, v_out, k_cache, v_cache, block_scales, slot_mapping,
                                        num_tokens, num_blocks, block_size, num_kv_heads, head_dim,
                                        launch);
    if (!launch) return st;
    auto* kernel = head_dim == 128 ? kv_gather_e2m1_kernel<128> : kv_gather_e2m1_kernel<256>;
    kernel<<<row_blocks(num_tokens), kRowWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint32_t*>(k_cache), static_cast<const uint32_t*>(v_cache),
        static_cast<const uint8_t*>(block_scales), slot_mapping, static_cast<uint4*>(k_out),
        static_cast<uint4*>(v_out), num_tokens, static_cast<int64_t>(num_blocks) * block_size,
        block_size == 16 ? 4 : 5, num_kv_heads, err_word);
    return cuda_status(cudaGetLastError());
}
