// yoco_retention: linear attention with a decay per head, the self-decoder's
// gated retention ("YOCO 论文与推理数据流详解" §4.1-§4.2: parallel, recurrent
// and chunkwise forms of one recurrence).
//
// For a head, with a_t = exp(g_t):  S_t = a_t S_(t-1) + k_t v_t^T (D x D),
// o_t = scale q_t^T S_t. With L_t the running sum of g within a chunk of C
// tokens and S the state before it, the chunk is
//   o_t = scale ( exp(L_t) q_t^T S + sum_(j<=t) exp(L_t - L_j) (q_t . k_j) v_j )
//   S' = exp(L_C) S + sum_j k_j (exp(L_C - L_j) v_j)^T
// Every exponent is a difference of running sums with the later one first, so
// no factor passes 1 for decays of at most 1. The sums run in 64 bits and are
// kept as two floats: a difference of two neighbours stays exact however far
// the sum has fallen.
//
// Kernels.
//   retention_step: requests of one token. Moves the state once (read and
//     write, fp32): bound by HBM.
//   retention_plan: cuts the longer requests into segments of whole chunks.
//   retention_chunks<.., false>: the state that each segment but a request's
//     last adds (from zero), all segments at once.
//   retention_scan: runs along a request's segments and turns those into the
//     state before each segment.
//   retention_chunks<.., true>: outputs of every segment, chunk by chunk, and
//     the state after a request's last one.
// A request of one segment needs neither the second pass nor the scan.
#include "common.cuh"

namespace yoco {
namespace {

constexpr int kChunk = 64;         // tokens of a chunk
constexpr int kSlice = 64;         // value dims of a CTA
constexpr int kChunkThreads = 256;
constexpr float kMinDecay = -80.f; // exp(-80) = 2e-35: less counts as this (and -inf stays a number)
constexpr float kLn2Inv = 1.4426950408889634f;

struct RetParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    const float* decay;        // log decay [H] or [num_tokens][H]
    const float* state;
    float* state_out;
    const int32_t* where;
    __nv_bfloat16* out;
    const int32_t* qsl;
    const int32_t* seq_lens;
    int32_t* err;
    int32_t num_reqs, num_tokens, max_q_len, num_states;
    int32_t H, G;              // heads, heads per k/v head
    int32_t by_token;          // decay has a row for each token
    float scale;
    int32_t seg_tokens;        // tokens of a segment, a multiple of kChunk
    int32_t max_segs, max_slots;
    // workspace
    struct RetSeg* segs;
    int32_t* num_segs;
    float* seg_decay;          // [slots][H]
    float* slots;              // [slots][H][D][D]
};

struct __align__(16) RetSeg {
    int32_t req, token, tokens, slot;  // slot: of the state before it, -1: the request's own state
    int32_t index, count, base, pad;   // which of its request's segments; the request's first slot
};

__device__ __forceinline__ float decay_of(const RetParams& p, int64_t token, int32_t h) {
    const float g = __ldg(p.decay + (p.by_token ? token * p.H : 0) + h);
    return g < kMinDecay ? kMinDecay : g;  // a NaN stays one
}

// Tokens [q0, q1) of request r if it is well formed and has some, else false.
// `report`: flag what is wrong with it.
__device__ __forceinline__ bool ret_request(const RetParams& p, int32_t r, bool report, int32_t& q0,
                                            int32_t& q1, int32_t& where, bool& fresh) {
    q0 = __ldg(p.qsl + r);
    q1 = __ldg(p.qsl + r + 1);
    const int32_t seq = __ldg(p.seq_lens + r);
    where = __ldg(p.where + r);
    if (q1 == q0) return false;
    int32_t bad = 0;
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_q_len) bad |= YOCO_DEVERR_OFFSETS;
    else if (seq < q1 - q0) bad |= YOCO_DEVERR_POS_RANGE;
    if (where < 0 || where >= p.num_states) bad |= YOCO_DEVERR_STATE;
    if (bad && report) set_err(p.err, bad);
    fresh = seq == q1 - q0;
    return bad == 0;
}

// ------------------------------------------------------------ single tokens

// One CTA per (request, head, 64 value dims): 16 threads along the value dims
// (16 bytes each), 16 row groups, so that every row piece is one 256-byte run
// and all of a thread's rows are in flight at once.
template <int D>
__global__ void __launch_bounds__(256) retention_step(const RetParams p) {
    constexpr int ROWS = D / 16;
    __shared__ float sq[D], sk[D];
    __shared__ float4 part[16][16];
    constexpr int NS = D / kSlice;
    const int32_t slice = blockIdx.x % NS, h = blockIdx.x / NS % p.H;
    const int32_t r = blockIdx.x / (NS * p.H);
    int32_t q0, q1, where;
    bool fresh;
    const bool ok = ret_request(p, r, h == 0 && slice == 0 && threadIdx.x == 0, q0, q1, where, fresh);
    if (!ok || q1 - q0 != 1) return;
    const int c = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t tok = q0;
    const int32_t hk = h / p.G, H_kv = p.H / p.G;
    const float a = exp2f(decay_of(p, tok, h) * kLn2Inv);
    const int64_t base = (static_cast<int64_t>(where) * p.H + h) * D * D + slice * kSlice + 4 * c;
    float4 s[ROWS];
    if (!fresh) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            s[i] = *reinterpret_cast<const float4*>(p.state + base + static_cast<int64_t>(i * 16 + rg) * D);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (threadIdx.x < D) {
        sq[threadIdx.x] = __bfloat162float(p.q[(tok * p.H + h) * D + threadIdx.x]);
        sk[threadIdx.x] = __bfloat162float(p.k[(tok * H_kv + hk) * D + threadIdx.x]);
    }
    const uint2 vw = __ldg(reinterpret_cast<const uint2*>(p.v + (tok * H_kv + hk) * D + slice * kSlice + 4 * c));
    const float4 v = make_float4(bf16lo_to_f32(vw.x), bf16hi_to_f32(vw.x), bf16lo_to_f32(vw.y),
                                 bf16hi_to_f32(vw.y));
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float kk = sk[i * 16 + rg], qq = sq[i * 16 + rg];
        float4 x = s[i];
        x.x = fmaf(a, x.x, kk * v.x);
        x.y = fmaf(a, x.y, kk * v.y);
        x.z = fmaf(a, x.z, kk * v.z);
        x.w = fmaf(a, x.w, kk * v.w);
        *reinterpret_cast<float4*>(p.state_out + base + static_cast<int64_t>(i * 16 + rg) * D) = x;
        o.x = fmaf(qq, x.x, o.x);
        o.y = fmaf(qq, x.y, o.y);
        o.z = fmaf(qq, x.z, o.z);
        o.w = fmaf(qq, x.w, o.w);
    }
    part[rg][c] = o;
    __syncthreads();
    if (threadIdx.x < kSlice) {  // one value dim a thread, the row groups in order
        const float* f = reinterpret_cast<const float*>(&part[0][0]) + threadIdx.x;
        float t = 0.f;
#pragma unroll
        for (int g = 0; g < 16; ++g) t += f[g * kSlice];
        p.out[(tok * p.H + h) * D + slice * kSlice + threadIdx.x] = __float2bfloat16_rn(t * p.scale);
    }
}

// ------------------------------------------------------------------ segments

// One CTA: segments of every request of two tokens or more, in request order.
__global__ void __launch_bounds__(1024) retention_plan(const RetParams p) {
    __shared__ int32_t tot[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t seg0 = 0, slot0 = 0;
    for (int32_t base = 0; base < p.num_reqs; base += 1024) {
        const int32_t r = base + tid;
        int32_t q0 = 0, q1 = 0, where, n = 0;
        bool fresh;
        if (r < p.num_reqs && ret_request(p, r, false, q0, q1, where, fresh) && q1 - q0 > 1)
            n = (q1 - q0 + p.seg_tokens - 1) / p.seg_tokens;
        const int32_t m = n > 1 ? n : 0;
        int32_t a = n, b = m;  // inclusive sums over the warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
            if (lane >= off) {
                a += x;
                b += y;
            }
        }
        if (lane == 31) {
            tot[0][warp] = a;
            tot[1][warp] = b;
        }
        __syncthreads();
        int64_t first = seg0 + a - n, slot = slot0 + b - m;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) {
                first += tot[0][w];
                slot += tot[1][w];
            }
            seg0 += tot[0][w];
            slot0 += tot[1][w];
        }
        // Offsets that run backwards can claim more than the workspace holds: a request
        // that does not fit is listed with no segment (count 0).
        const bool fits = first + n <= p.max_segs && slot + m <= p.max_slots;
        if (n > 0 && !fits) set_err(p.err, YOCO_DEVERR_OFFSETS);
        for (int32_t i = 0; i < n && first + i < p.max_segs; ++i) {
            RetSeg s;
            s.req = r;
            s.token = q0 + i * p.seg_tokens;
            s.tokens = min(p.seg_tokens, q1 - s.token);
            s.slot = m ? static_cast<int32_t>(slot) + i : -1;
            s.index = i;
            s.count = fits ? n : 0;
            s.base = static_cast<int32_t>(slot);
            s.pad = 0;
            p.segs[first + i] = s;
        }
        __syncthreads();
    }
    if (tid == 0) *p.num_segs = static_cast<int32_t>(seg0 < p.max_segs ? seg0 : p.max_segs);
}

// State before each segment of a request: slot 0 is its own state (or zero),
// slot i + 1 = decay of segment i * slot i + what segment i adds.
template <int D>
__global__ void __launch_bounds__(256) retention_scan(const RetParams p) {
    constexpr int PARTS = D * D / 1024;  // CTAs of a (request, head)
    const int32_t n = *p.num_segs;
    for (int64_t item = blockIdx.x; item < static_cast<int64_t>(n) * p.H * PARTS; item += gridDim.x) {
        const RetSeg s = p.segs[item / (p.H * PARTS)];
        if (s.count <= 1 || s.index != 0) continue;
        const int32_t h = static_cast<int32_t>(item / PARTS % p.H), part = static_cast<int32_t>(item % PARTS);
        const int64_t at = static_cast<int64_t>(part) * 1024 + threadIdx.x * 4;
        const int32_t q = __ldg(p.qsl + s.req + 1) - __ldg(p.qsl + s.req);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (__ldg(p.seq_lens + s.req) > q)
            x = *reinterpret_cast<const float4*>(
                p.state + (static_cast<int64_t>(__ldg(p.where + s.req)) * p.H + h) * D * D + at);
        float* slot = p.slots + (static_cast<int64_t>(s.base) * p.H + h) * D * D + at;
        const int64_t stride = static_cast<int64_t>(p.H) * D * D;
        *reinterpret_cast<float4*>(slot) = x;
        for (int32_t i = 0; i + 1 < s.count; ++i) {
            slot += stride;
            const float a = p.seg_decay[static_cast<int64_t>(s.base + i) * p.H + h];
            const float4 y = *reinterpret_cast<const float4*>(slot);
            x.x = fmaf(a, x.x, y.x);
            x.y = fmaf(a, x.y, y.y);
            x.z = fmaf(a, x.z, y.z);
            x.w = fmaf(a, x.w, y.w);
            *reinterpret_cast<float4*>(slot) = x;
        }
    }
}

// -------------------------------------------------------------------- chunks

// Byte offset of 16-byte piece j of row r in a tile of ROW-byte rows, swizzled
// so that the 8 rows of an ldmatrix fall in distinct banks.
template <int ROW>
__device__ __forceinline__ uint32_t tile_at(int r, int j) {
    return static_cast<uint32_t>(r * ROW + ((j ^ (r & 7)) << 4));
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
                 : "memory");
}

template <int D, bool OUT>
struct RetShape {
    static constexpr int ROWB = 2 * D;                       // bytes of a q or k row
    static constexpr int QB = OUT ? kChunk * ROWB : 0;
    static constexpr int KB = kChunk * ROWB;
    static constexpr int VB = kChunk * kSlice * 2;
    static constexpr int STAGE = QB + KB + VB;
    static constexpr int SB = OUT ? D * kSlice * 2 : 0;      // the state in bf16
    static constexpr int PB = OUT ? kChunk * kChunk * 2 : 0; // weights in bf16
    static constexpr int LB = 8 * (kChunk * 16 + 16);        // sums and factors of 8 chunks
    static constexpr int SMEM = 2 * STAGE + SB + PB + 3 * VB + LB + 1024;
    static constexpr int CTAS = 2 * SMEM <= 224 * 1024 ? 2 : 1;  // of an SM
    static constexpr int MT = D >= 128 ? D / 128 : 1;        // 16-row tiles of the state a warp holds
    static constexpr int NTS = D >= 128 ? 8 : 4;             // its 8-column tiles
};

// One CTA walks the chunks of one (segment, head, 64 value dims); the state
// slice [D][64] stays in the accumulator registers of its 8 warps. Products
// are m16n8k16 bf16 with fp32 accumulators. Roundings to bf16: the weights P,
// the state as an operand of q S (the state itself stays fp32), both below
// the rounding of the output; exp(L_C - L_j) v_j as a sum of three bf16 terms
// (24 bits) where the state leaves the kernel, of two (16 bits) where it only
// feeds later outputs of its segment.
template <int D, bool OUT>
__global__ void __launch_bounds__(kChunkThreads, RetShape<D, OUT>::CTAS)
    retention_chunks(const RetParams p) {
    using S = RetShape<D, OUT>;
    constexpr int NS = D / kSlice, MT = S::MT, NTS = S::NTS;
    extern __shared__ uint8_t ret_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ret_smem) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(smem);
    const uint32_t s_state = base + 2 * S::STAGE, s_p = s_state + S::SB, s_vw = s_p + S::PB;
    // of each of 8 chunks: 64 x {sum hi, sum lo, exp(L_t), exp(L_C - L_t)} in log2 units, then exp(L_C)
    float4* const fac = reinterpret_cast<float4*>(smem + 2 * S::STAGE + S::SB + S::PB + 3 * S::VB);
    float* const whole = reinterpret_cast<float*>(fac + 8 * kChunk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gl = lane >> 2, tq = lane & 3, mi = lane >> 3, rr = lane & 7;
    // this warp's part of the state: rows row0.. (16 * MT), columns col0.. (8 * NTS)
    const int row0 = D >= 128 ? warp * 16 * MT : (warp & 3) * 16;
    const int col0 = D >= 128 ? 0 : (warp >> 2) * 32;
    const int rb = warp & 3, cb = warp >> 2;  // 16 x 32 block of a 64 x 64 product
    const int32_t H_kv = p.H / p.G;
    const int32_t items = *p.num_segs * p.H * NS;

    for (int32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const RetSeg sg = p.segs[item / (p.H * NS)];
        const bool last = sg.index == sg.count - 1;
        if (sg.count == 0 || (!OUT && last)) continue;
        const int32_t h = item / NS % p.H, dv0 = item % NS * kSlice, hk = h / p.G;
        const int32_t chunks = (sg.tokens + kChunk - 1) / kChunk;

        auto load = [&](int32_t c) {  // chunk c into its stage
            const uint32_t st = base + (c & 1) * S::STAGE;
            const int32_t left = sg.tokens - c * kChunk;
            const int64_t t0 = sg.token + static_cast<int64_t>(c) * kChunk;
            constexpr int J = D / 8;
#pragma unroll
            for (int x = tid; x < kChunk * J; x += kChunkThreads) {
                const int t = x / J, j = x % J;
                const bool there = t < left;
                const int64_t row = there ? t0 + t : t0;
                if constexpr (OUT)
                    cp_async_16_or_zero(st + tile_at<S::ROWB>(t, j), p.q + (row * p.H + h) * D + j * 8, there);
                cp_async_16_or_zero(st + S::QB + tile_at<S::ROWB>(t, j), p.k + (row * H_kv + hk) * D + j * 8, there);
            }
#pragma unroll
            for (int x = tid; x < kChunk * 8; x += kChunkThreads) {
                const int t = x >> 3, j = x & 7;
                const bool there = t < left;
                const int64_t row = there ? t0 + t : t0;
                cp_async_16_or_zero(st + S::QB + S::KB + tile_at<128>(t, j),
                                    p.v + (row * H_kv + hk) * D + dv0 + j * 8, there);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        __syncthreads();  // the previous item is done with the stages
        load(0);

        // the state before the segment
        float s[MT][NTS][4];
        {
            const float* src = nullptr;
            if (OUT) {
                const int32_t q = __ldg(p.qsl + sg.req + 1) - __ldg(p.qsl + sg.req);
                if (sg.slot >= 0)
                    src = p.slots + (static_cast<int64_t>(sg.slot) * p.H + h) * D * D + dv0;
                else if (__ldg(p.seq_lens + sg.req) > q)
                    src = p.state + (static_cast<int64_t>(__ldg(p.where + sg.req)) * p.H + h) * D * D + dv0;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NTS; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float2 x = make_float2(0.f, 0.f);
                        if (src)
                            x = *reinterpret_cast<const float2*>(
                                src + static_cast<int64_t>(row0 + m * 16 + gl + 8 * e) * D + col0 + n * 8 + 2 * tq);
                        s[m][n][2 * e] = x.x;
                        s[m][n][2 * e + 1] = x.y;
                    }
        }
        double decay_all = 0.0;  // warp 0: sum of the segment's log decays (log2 units)

        for (int32_t c = 0; c < chunks; ++c) {
            if ((c & 7) == 0) {  // running sums and factors of 8 chunks, one a warp
                if (c) __syncthreads();
                const int32_t cc = c + warp;
                const int64_t t0 = sg.token + static_cast<int64_t>(cc) * kChunk;
                const int32_t left = cc < chunks ? min(kChunk, sg.tokens - cc * kChunk) : 0;
                // lane l has tokens 2l and 2l + 1
                const double g0 = 2 * lane < left ? static_cast<double>(decay_of(p, t0 + 2 * lane, h)) : 0.0;
                const double g1 = 2 * lane + 1 < left ? static_cast<double>(decay_of(p, t0 + 2 * lane + 1, h)) : 0.0;
                double sum = g0 + g1;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double x = __shfl_up_sync(0xffffffffu, sum, off);
                    if (lane >= off) sum += x;
                }
                constexpr double kLog2E = 1.4426950408889634074;
                const double total = __shfl_sync(0xffffffffu, sum, 31) * kLog2E;
                const double l1 = sum * kLog2E, l0 = (sum - g1) * kLog2E;
                auto factors = [&](double l) {
                    const float hi = static_cast<float>(l);
                    return make_float4(hi, static_cast<float>(l - hi), exp2f(hi),
                                       exp2f(static_cast<float>(total - l)));
                };
                fac[warp * kChunk + 2 * lane] = factors(l0);
                fac[warp * kChunk + 2 * lane + 1] = factors(l1);
                if (lane == 0) whole[warp] = exp2f(static_cast<float>(total));
                if (!OUT && dv0 == 0) decay_all += total;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // chunk c is in shared memory; everyone is done with chunk c - 1
            if (c + 1 < chunks) load(c + 1);
            const uint32_t sq = base + (c & 1) * S::STAGE, sk = sq + S::QB, sv = sk + S::KB;
            const float4* f = fac + (c & 7) * kChunk;
            const bool update = !OUT || last || c + 1 < chunks;
            const int terms = (!OUT || last) ? 3 : 2;

            if constexpr (OUT) {
                // weights P = (q k^T) exp(L_t - L_j), lower triangle: rows 16 rb.., columns 32 cb..
                const int nt = min(4, 2 * (rb + 1) - 4 * cb);  // 8-column tiles that reach it
                if (nt > 0) {
                    float a[4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[n][e] = 0.f;
#pragma unroll 4
                    for (int kk = 0; kk < D / 16; ++kk) {
                        uint32_t a0, a1, a2, a3, b[8];
                        ldsm_x4(sq + tile_at<S::ROWB>(rb * 16 + (mi & 1) * 8 + rr, kk * 2 + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            ldsm_x4(sk + tile_at<S::ROWB>(cb * 32 + n * 16 + (mi >> 1) * 8 + rr, kk * 2 + (mi & 1)),
                                    b[4 * n], b[4 * n + 1], b[4 * n + 2], b[4 * n + 3]);
#pragma unroll
                        for (int n = 0; n < 4; ++n) mma_bf16_16816(a[n], a0, a1, a2, a3, b[2 * n], b[2 * n + 1]);
                    }
                    const int t0 = rb * 16 + gl;
                    const float4 ft[2] = {f[t0], f[t0 + 8]};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        if (n >= nt) continue;
                        const int j = cb * 32 + n * 8 + 2 * tq;
                        const float4 fj[2] = {f[j], f[j + 1]};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = t0 + 8 * e;
                            float w[2];
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                w[u] = j + u <= t ? a[n][2 * e + u] * exp2_approx((ft[e].x - fj[u].x) + (ft[e].y - fj[u].y))
                                                  : 0.f;
                            const uint32_t at = s_p + tile_at<128>(t, cb * 4 + n) + 4 * tq;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack_bf16x2(w[0], w[1])) : "memory");
                        }
                    }
                }
                // the state before the chunk, as an operand
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NTS; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t at = s_state + tile_at<128>(row0 + m * 16 + gl + 8 * e, (col0 >> 3) + n) + 4 * tq;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at),
                                         "r"(pack_bf16x2(s[m][n][2 * e], s[m][n][2 * e + 1]))
                                         : "memory");
                        }
            }
            if (update) {  // exp(L_C - L_j) v_j in bf16 terms
#pragma unroll
                for (int x = tid; x < kChunk * 8; x += kChunkThreads) {
                    const int t = x >> 3, j = x & 7;
                    const uint32_t at = tile_at<128>(t, j);
                    const uint4 w = *reinterpret_cast<const uint4*>(smem + (sv - base) + at);
                    const float fw = f[t].w;
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                    uint32_t o[3][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo = bf16lo_to_f32(in[i]) * fw, hi = bf16hi_to_f32(in[i]) * fw;
#pragma unroll
                        for (int u = 0; u < 3; ++u) {
                            o[u][i] = pack_bf16x2(lo, hi);
                            lo -= bf16lo_to_f32(o[u][i]);
                            hi -= bf16hi_to_f32(o[u][i]);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 3; ++u)
                        *reinterpret_cast<uint4*>(smem + (s_vw - base) + u * S::VB + at) =
                            make_uint4(o[u][0], o[u][1], o[u][2], o[u][3]);
                }
            }
            __syncthreads();
            if constexpr (OUT) {
                float o[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll 4
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a0, a1, a2, a3, b[8];
                    ldsm_x4(sq + tile_at<S::ROWB>(rb * 16 + (mi & 1) * 8 + rr, kk * 2 + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        ldsm_x4_trans(s_state + tile_at<128>(kk * 16 + (mi & 1) * 8 + rr, cb * 4 + n * 2 + (mi >> 1)),
                                      b[4 * n], b[4 * n + 1], b[4 * n + 2], b[4 * n + 3]);
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma_bf16_16816(o[n], a0, a1, a2, a3, b[2 * n], b[2 * n + 1]);
                }
                const float e0 = f[rb * 16 + gl].z, e1 = f[rb * 16 + gl + 8].z;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    o[n][0] *= e0;
                    o[n][1] *= e0;
                    o[n][2] *= e1;
                    o[n][3] *= e1;
                }
                for (int kk = 0; kk <= rb; ++kk) {  // later columns of P are zero for these rows
                    uint32_t a0, a1, a2, a3, b[8];
                    ldsm_x4(s_p + tile_at<128>(rb * 16 + (mi & 1) * 8 + rr, kk * 2 + (mi >> 1)), a0, a1, a2, a3);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        ldsm_x4_trans(sv + tile_at<128>(kk * 16 + (mi & 1) * 8 + rr, cb * 4 + n * 2 + (mi >> 1)),
                                      b[4 * n], b[4 * n + 1], b[4 * n + 2], b[4 * n + 3]);
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma_bf16_16816(o[n], a0, a1, a2, a3, b[2 * n], b[2 * n + 1]);
                }
                const int32_t left = sg.tokens - c * kChunk;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = rb * 16 + gl + 8 * e;
                    if (t >= left) continue;
                    __nv_bfloat16* dst = p.out + ((sg.token + static_cast<int64_t>(c) * kChunk + t) * p.H + h) * D + dv0 +
                                         cb * 32 + 2 * tq;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        *reinterpret_cast<uint32_t*>(dst + n * 8) =
                            pack_bf16x2(o[n][2 * e] * p.scale, o[n][2 * e + 1] * p.scale);
                }
            }
            if (update) {
                const float aC = whole[c & 7];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NTS; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[m][n][e] *= aC;
#pragma unroll 1
                for (int kk = 0; kk < kChunk / 16; ++kk) {
                    uint32_t a[MT][4];
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        ldsm_x4_trans(sk + tile_at<S::ROWB>(kk * 16 + (mi >> 1) * 8 + rr, (row0 >> 3) + m * 2 + (mi & 1)),
                                      a[m][0], a[m][1], a[m][2], a[m][3]);
                    for (int u = 0; u < terms; ++u) {
#pragma unroll
                        for (int n = 0; n < NTS / 2; ++n) {
                            uint32_t b[4];
                            ldsm_x4_trans(s_vw + u * S::VB +
                                              tile_at<128>(kk * 16 + (mi & 1) * 8 + rr, (col0 >> 3) + n * 2 + (mi >> 1)),
                                          b[0], b[1], b[2], b[3]);
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                mma_bf16_16816(s[m][2 * n], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
                                mma_bf16_16816(s[m][2 * n + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
                            }
                        }
                    }
                }
            }
        }
        // the state after the segment
        float* dst = nullptr;
        if (!OUT)
            dst = p.slots + (static_cast<int64_t>(sg.slot + 1) * p.H + h) * D * D + dv0;
        else if (last)
            dst = p.state_out + (static_cast<int64_t>(__ldg(p.where + sg.req)) * p.H + h) * D * D + dv0;
        if (dst) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NTS; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float2*>(dst + static_cast<int64_t>(row0 + m * 16 + gl + 8 * e) * D + col0 +
                                                   n * 8 + 2 * tq) = make_float2(s[m][n][2 * e], s[m][n][2 * e + 1]);
        }
        if (!OUT && dv0 == 0) {  // every warp has the sums of its own chunks
            __syncthreads();
            double* all = reinterpret_cast<double*>(fac);
            if (lane == 0) all[warp] = decay_all;
            __syncthreads();
            if (tid == 0) {
                double t = 0.0;
                for (int w = 0; w < 8; ++w) t += all[w];
                p.seg_decay[static_cast<int64_t>(sg.slot) * p.H + h] = exp2f(static_cast<float>(t));
            }
        }
    }
}

// ------------------------------------------------------------------ host side

constexpr int kMinSegment = 256;  // tokens

// Segments to aim for: about two CTAs for every SM over heads and slices.
int64_t ret_target(int H, int D) {
    const int64_t units = static_cast<int64_t>(H) * (D / kSlice);
    const int64_t n = (2ll * device_sm_count() + units - 1) / units;
    return n < 1 ? 1 : n;
}

struct RetPlan {
    int64_t seg_tokens, max_segs, max_slots;
    size_t list_bytes, decay_bytes, bytes;
};

// The same for every call within the bounds (and no larger for smaller ones).
RetPlan ret_plan(int64_t R, int64_t T, int64_t max_q, int H, int D) {
    RetPlan x = {};
    if (max_q <= 1 || R <= 0 || T <= 1) return x;
    const int64_t target = ret_target(H, D);
    int64_t seg = ((T + target - 1) / target + kChunk - 1) / kChunk * kChunk;
    if (seg < kMinSegment) seg = kMinSegment;
    x.seg_tokens = seg;
    // whole segments, and at most one shorter one for each request of two tokens or more
    const int64_t shorter = R < T / 2 ? R : T / 2;
    const int64_t cut = max_q > seg ? T / seg : 0;
    x.max_segs = T / seg + shorter;
    x.max_slots = 2 * cut;
    return x;
}

// Workspace of the largest plan up to these bounds.
RetPlan ret_sizes(int64_t R, int64_t T, int64_t max_q, int H, int D) {
    RetPlan x = ret_plan(R, T, max_q, H, D);
    if (x.seg_tokens == 0) return x;
    const int64_t target = ret_target(H, D), whole = T / kMinSegment < target ? T / kMinSegment : target;
    const int64_t segs = whole + (R < T / 2 ? R : T / 2), slots = max_q > kMinSegment ? 2 * whole : 0;
    x.list_bytes = (16 + static_cast<size_t>(segs) * sizeof(RetSeg) + 255) & ~static_cast<size_t>(255);
    x.decay_bytes = (static_cast<size_t>(slots) * H * 4 + 255) & ~static_cast<size_t>(255);
    x.bytes = x.list_bytes + x.decay_bytes + static_cast<size_t>(slots) * H * D * D * 4;
    return x;
}

template <typename K>
cudaError_t ret_smem_attr(K kernel, int bytes, unsigned long long& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? (1ull << dev) : 0;
    if (bit && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit) __atomic_fetch_or(&done, bit, __ATOMIC_RELEASE);
    return e;
}

template <int D>
cudaError_t launch_retention(const RetParams& p, cudaStream_t s) {
    constexpr int NS = D / kSlice;
    retention_step<D><<<static_cast<unsigned>(static_cast<int64_t>(p.num_reqs) * p.H * NS), 256, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.seg_tokens == 0) return e;
    static unsigned long long done_out = 0, done_add = 0;
    e = ret_smem_attr(retention_chunks<D, true>, RetShape<D, true>::SMEM, done_out);
    if (e == cudaSuccess) e = ret_smem_attr(retention_chunks<D, false>, RetShape<D, false>::SMEM, done_add);
    if (e != cudaSuccess) return e;
    retention_plan<<<1, 1024, 0, s>>>(p);
    const int64_t sms = device_sm_count(), items = static_cast<int64_t>(p.max_segs) * p.H * NS;
    auto grid = [&](int64_t per) { return static_cast<unsigned>(items < sms * per ? items : sms * per); };
    if (p.max_slots > 0) {
        retention_chunks<D, false><<<grid(RetShape<D, false>::CTAS), kChunkThreads, RetShape<D, false>::SMEM, s>>>(p);
        const int64_t parts = static_cast<int64_t>(p.max_segs) * p.H * (D * D / 1024);
        retention_scan<D><<<static_cast<unsigned>(parts < 16 * sms ? parts : 16 * sms), 256, 0, s>>>(p);
    }
    retention_chunks<D, true><<<grid(RetShape<D, true>::CTAS), kChunkThreads, RetShape<D, true>::SMEM, s>>>(p);
    return cudaGetLastError();
}

bool ret_shape_ok(int32_t H, int32_t D) {
    return head_dim_ok(D) && H > 0 && H <= 0x7fffffff / (256 * 64);
}

}  // namespace
}  // namespace yoco

extern "C" size_t yoco_retention_workspace_size(int32_t num_reqs, int32_t num_tokens,
                                                int32_t max_q_len, int32_t num_q_heads,
                                                int32_t head_dim) {
    if (num_reqs < 0 || num_tokens < 0 || !yoco::ret_shape_ok(num_q_heads, head_dim)) return 0;
    return yoco::ret_sizes(num_reqs, num_tokens, max_q_len, num_q_heads, head_dim).bytes;
}

extern "C" yoco_status_t yoco_retention(
    const void* q, const void* k, const void* v, const float* log_decay, int32_t decay_per_token,
    const float* state, float* state_out, const int32_t* state_indices, void* out,
    const int32_t* query_start_loc, const int32_t* seq_lens, int32_t num_reqs, int32_t num_tokens,
    int32_t max_q_len, int32_t num_states, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, float scale, void* workspace, size_t workspace_bytes, int32_t* err_word,
    void* stream) {
    using namespace yoco;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0) return YOCO_ERR_INVALID_ARG;
    if (!ret_shape_ok(num_q_heads, head_dim)) return YOCO_ERR_UNSUPPORTED;
    if (num_reqs < 0 || num_tokens < 0 || max_q_len < 1 || num_states <= 0 || !(scale == scale))
        return YOCO_ERR_INVALID_ARG;
    if (num_reqs == 0 || num_tokens == 0) return YOCO_OK;
    if (!q || !k || !v || !log_decay || !state || !state_out || !state_indices || !out || !query_start_loc || !seq_lens)
        return YOCO_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(state) || !aligned16(state_out) || !aligned16(out))
        return YOCO_ERR_INVALID_ARG;
    // one CTA per (request, head, slice)
    if (static_cast<int64_t>(num_reqs) * num_q_heads * (head_dim / kSlice) > 0x7fffffffll) return YOCO_ERR_UNSUPPORTED;
    const int32_t longest = max_q_len < num_tokens ? max_q_len : num_tokens;
    const RetPlan pl = ret_plan(num_reqs, num_tokens, longest, num_q_heads, head_dim);
    const RetPlan sz = ret_sizes(num_reqs, num_tokens, longest, num_q_heads, head_dim);
    if (sz.bytes > 0) {
        if (!workspace || workspace_bytes < sz.bytes) return YOCO_ERR_WORKSPACE;
        if (!aligned16(workspace)) return YOCO_ERR_INVALID_ARG;
        // items are counted in 32 bits
        if (pl.max_segs * num_q_heads * (head_dim / kSlice) > 0x7fffffffll - (1 << 20)) return YOCO_ERR_UNSUPPORTED;
    }
    RetParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.decay = log_decay;
    p.state = state;
    p.state_out = state_out;
    p.where = state_indices;
    p.out = static_cast<__nv_bfloat16*>(out);
    p.qsl = query_start_loc;
    p.seq_lens = seq_lens;
    p.err = err_word;
    p.num_reqs = num_reqs;
    p.num_tokens = num_tokens;
    p.max_q_len = max_q_len;
    p.num_states = num_states;
    p.H = num_q_heads;
    p.G = num_q_heads / num_kv_heads;
    p.by_token = decay_per_token ? 1 : 0;
    p.scale = scale;
    p.seg_tokens = static_cast<int32_t>(pl.seg_tokens);
    p.max_segs = static_cast<int32_t>(pl.max_segs);
    p.max_slots = static_cast<int32_t>(pl.max_slots);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.num_segs = reinterpret_cast<int32_t*>(ws);
    p.segs = reinterpret_cast<RetSeg*>(ws + 16);
    p.seg_decay = reinterpret_cast<float*>(ws + sz.list_bytes);
    p.slots = reinterpret_cast<float*>(ws + sz.list_bytes + sz.decay_bytes);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (head_dim) {
        case 64: e = launch_retention<64>(p, s); break;
        case 128: e = launch_retention<128>(p, s); break;
        default: e = launch_retention<256>(p, s); break;
    }
    return cuda_status(e);
}
