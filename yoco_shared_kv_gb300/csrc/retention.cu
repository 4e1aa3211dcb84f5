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
// no factor passes 1 for decays of at most 1. The sums run as two floats (48
// bits): a difference of two neighbours stays exact however far the sum has
// fallen.
//
// Kernels.
//   retention_step: requests of one token. Moves the state once (read and
//     write, fp32): bound by HBM.
//   retention_plan: cuts the longer requests into segments of whole chunks.
//   retention_add<false>: the state that each segment adds (from zero), all
//     segments at once.
//   retention_scan: runs along a request's segments and turns those into the
//     state before each segment and after the last.
//   retention_out: outputs of every segment, chunk by chunk.
//   retention_add<true>: the state after requests of one segment that the
//     workspace had no room for in the first pass.
//
// Measured, replayed from a graph. Single tokens of 64 requests, 8 heads of
// 256: 43.9 us, 6.1 TB/s on the states' 269 MB (90% of what a copy reaches);
// of 5, 8 heads of 128: 3.2 us, the launch. 16 single tokens and 4 prompts of
// 1024..4096, 8 heads of 256: 186 us, where the bytes take 36 and the products
// 11; one prompt of 16384, 8 heads of 128: 83 us (12 and 5). Of the prompts'
// time the outputs take half, the segments' states a third, the scan a tenth,
// the plan 4%. A walk without segments reads every token once and needs no
// scan, but has 64 CTAs for the first and 8 for the second: at the time of a
// chunk (below) 220 and 590 us.
#include "common.cuh"

namespace yoco {
namespace {

constexpr int kChunk = 64;         // tokens of a chunk
constexpr int kSlice = 64;         // value dims of a single token's CTA
constexpr int kAddThreads = 256;   // and a warp that issues the products, and one for the factors
constexpr int kOutThreads = 512;   // likewise
constexpr uint64_t kRetWaitNs = 1000000000ull;  // before a wait gives up
constexpr int kMaxChunks = 512;                 // of a segment
constexpr int kMaxSegment = kMaxChunks * kChunk;
constexpr int kChooseReqs = 4096;               // with more requests segments take the shortest length
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
    int32_t seg_tokens;        // tokens of a segment at least, a multiple of kChunk
    int32_t max_segs, max_slots;
    // workspace
    struct RetSeg* segs;
    int32_t* num_segs;         // segments; whether a request has no slot
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

// A sum as two floats, the second what the first rounds off (48 bits together).
struct Sum {
    float h, l;
};
__device__ __forceinline__ Sum operator+(Sum a, Sum b) {
    const float s = a.h + b.h, v = s - a.h;
    const float e = ((a.h - (s - v)) + (b.h - v)) + (a.l + b.l);
    const float h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ float operator-(Sum a, Sum b) { return (a.h - b.h) + (a.l - b.l); }
__device__ __forceinline__ Sum in_log2(float g) {  // g log2(e)
    const float h = g * 1.44269502f;                // log2(e) = 1.44269502 + 1.92596e-8
    return {h, fmaf(g, 1.44269502f, -h) + g * 1.925963033e-8f};
}
__device__ __forceinline__ Sum shfl_up(Sum a, int n) {
    return {__shfl_up_sync(0xffffffffu, a.h, n), __shfl_up_sync(0xffffffffu, a.l, n)};
}
__device__ __forceinline__ Sum warp_total(Sum a) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        a = a + Sum{__shfl_xor_sync(0xffffffffu, a.h, off), __shfl_xor_sync(0xffffffffu, a.l, off)};
    return a;
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
// and all of a thread's rows are in flight at once (2048 CTAs for 64 requests
// of 8 heads of 256: DRAM 67% taken over the launch, its start and end in it).
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
    // Where it was launched beside the segments' pass, this kernel ends after that one (what
    // follows it in the stream waits for this one alone).
    if (!ok || q1 - q0 != 1) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ segments

// Time of both chunk passes, in chunks with outputs, if requests are cut into `segs` segments
// of up to `chunks` chunks (`cut` of them of requests of several, `all` chunks together) over
// `units` heads and slices: rounds of whole segments on all SMs, or the work evenly spread and
// one segment more, whichever is less. A segment costs about 4 chunks beside its own; a chunk
// without outputs two thirds of one with.
__device__ __forceinline__ float pass_time(int32_t segs, int32_t cut, int32_t all, int32_t chunks, int32_t units,
                                           int32_t sms) {
    const float per = static_cast<float>(units) / static_cast<float>(sms), own = static_cast<float>(chunks + 4);
    auto one = [&](float n, float work) { return fminf(ceilf(n * per) * own, (work + 4.f * n) * per + own); };
    const float n = static_cast<float>(segs), m = static_cast<float>(cut);
    return one(n, static_cast<float>(all)) + (cut ? 0.67f * one(m, m * static_cast<float>(chunks)) : 0.f);
}

// One CTA: segments of every request of two tokens or more, in request order. Their length
// is the best of 32, from the shortest that the workspace has room for upwards.
__global__ void __launch_bounds__(1024) retention_plan(RetParams p, int32_t units, int32_t sms) {
    __shared__ int32_t tot[3][32], need[32];
    __shared__ float cost[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int64_t single0 = p.max_slots;  // slots that requests of one segment may take
    if (p.max_slots > 0 && p.num_reqs <= kChooseReqs) {
        const float grown = static_cast<float>(p.seg_tokens) * exp2f(static_cast<float>(warp) / 6.f);
        const int32_t seg = min((static_cast<int32_t>(fminf(grown, 1e6f)) + kChunk - 1) / kChunk * kChunk, kMaxSegment);
        int32_t segs = 0, slots = 0, cut = 0, all = 0, longest = 0;
        for (int32_t r = lane; r < p.num_reqs; r += 32) {
            int32_t q0, q1, where;
            bool fresh;
            if (!ret_request(p, r, false, q0, q1, where, fresh) || q1 - q0 < 2) continue;
            const int32_t n = (q1 - q0 + seg - 1) / seg;
            segs += n;
            if (n > 1) slots += n + 1;
            if (n > 1) cut += n;
            all += (q1 - q0 + kChunk - 1) / kChunk;
            longest = max(longest, min(q1 - q0, seg));
        }
        segs = __reduce_add_sync(0xffffffffu, segs);
        slots = __reduce_add_sync(0xffffffffu, slots);
        cut = __reduce_add_sync(0xffffffffu, cut);
        all = __reduce_add_sync(0xffffffffu, all);
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 0) need[warp] = slots;
        if (lane == 0)
            cost[warp] = segs > p.max_segs || slots > p.max_slots
                             ? INFINITY
                             : pass_time(segs, cut, all, (longest + kChunk - 1) / kChunk, units, sms);
        __syncthreads();
        const uint32_t mine = __float_as_uint(cost[lane]);  // not negative: its bits are in order
        const uint32_t least = __reduce_min_sync(0xffffffffu, mine);
        const int best = __ffs(__ballot_sync(0xffffffffu, mine == least)) - 1;
        const float chosen = static_cast<float>(p.seg_tokens) * exp2f(static_cast<float>(best) / 6.f);
        p.seg_tokens = min((static_cast<int32_t>(fminf(chosen, 1e6f)) + kChunk - 1) / kChunk * kChunk, kMaxSegment);
        single0 = need[best];
    }
    int64_t seg0 = 0, slot0 = 0;
    int32_t finals = 0;
    for (int32_t base = 0; base < p.num_reqs; base += 1024) {
        const int32_t r = base + tid;
        int32_t q0 = 0, q1 = 0, where, n = 0;
        bool fresh;
        if (r < p.num_reqs && ret_request(p, r, false, q0, q1, where, fresh) && q1 - q0 > 1)
            n = (q1 - q0 + p.seg_tokens - 1) / p.seg_tokens;
        // slots: before each segment and after the last; for one segment of some length too,
        // as far as there is room, so that its state is worked out beside the others'
        const int32_t m = n > 1 ? n + 1 : 0, k = n == 1 && q1 - q0 > 2 * kChunk ? 2 : 0;
        int32_t a = n, b = m, d = k;  // inclusive sums over the warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, a, off), y = __shfl_up_sync(0xffffffffu, b, off);
            const int32_t z = __shfl_up_sync(0xffffffffu, d, off);
            if (lane >= off) {
                a += x;
                b += y;
                d += z;
            }
        }
        if (lane == 31) {
            tot[0][warp] = a;
            tot[1][warp] = b;
            tot[2][warp] = d;
        }
        __syncthreads();
        int64_t first = seg0 + a - n, slot = slot0 + b - m, single = single0 + d - k;
        auto over_warps = [&](int i, int64_t& before, int64_t& all) {  // the warps' sums
            int64_t v = tot[i][lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += x;
            }
            const int64_t x = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
            if (warp > 0) before += x;
            all += __shfl_sync(0xffffffffu, v, 31);
        };
        over_warps(0, first, seg0);
        over_warps(1, slot, slot0);
        over_warps(2, single, single0);
        // Offsets that run backwards can claim more than the workspace holds: a request
        // that does not fit is listed with no segment (count 0).
        const bool fits = first + n <= p.max_segs && slot + m <= p.max_slots;
        if (n > 0 && !fits) set_err(p.err, YOCO_DEVERR_OFFSETS);
        const bool slotted = m > 0 || (k > 0 && single + k <= p.max_slots);
        const int32_t at = static_cast<int32_t>(m ? slot : single);
        if (n > 0 && fits && !slotted) ++finals;
        for (int32_t i = 0; i < n && first + i < p.max_segs; ++i) {
            RetSeg s;
            s.req = r;
            s.token = q0 + i * p.seg_tokens;
            s.tokens = min(p.seg_tokens, q1 - s.token);
            s.slot = slotted ? at + i : -1;
            s.index = i;
            s.count = fits ? n : 0;
            s.base = at;
            s.pad = 0;
            p.segs[first + i] = s;
        }
        __syncthreads();
    }
    finals = __syncthreads_count(finals > 0);
    if (tid == 0) {
        p.num_segs[0] = static_cast<int32_t>(seg0 < p.max_segs ? seg0 : p.max_segs);
        p.num_segs[1] = finals;
    }
}

// State before each segment of a request with slots: slot 0 gets its own state (or zero), slot i + 1
// the decay of segment i * slot i + what segment i adds, which it holds; the last of them is
// the state after the request. Four elements of a state a thread, eight segments' loads ahead
// of the sums: a tenth of the call's time, the slots out of L2 for the most part (DRAM 14%
// taken).
template <int D>
__global__ void __launch_bounds__(256) retention_scan(const RetParams p) {
    constexpr int PARTS = D * D / 1024;  // CTAs of a (request, head)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t n = *p.num_segs;
    for (int64_t item = blockIdx.x; item < static_cast<int64_t>(n) * p.H * PARTS; item += gridDim.x) {
        const RetSeg s = p.segs[item / (p.H * PARTS)];
        if (s.count == 0 || s.index != 0 || s.slot < 0) continue;
        const int32_t h = static_cast<int32_t>(item / PARTS % p.H), part = static_cast<int32_t>(item % PARTS);
        const int64_t at = static_cast<int64_t>(part) * 1024 + threadIdx.x * 4;
        const int64_t own = (static_cast<int64_t>(__ldg(p.where + s.req)) * p.H + h) * D * D + at;
        const int32_t q = __ldg(p.qsl + s.req + 1) - __ldg(p.qsl + s.req);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (__ldg(p.seq_lens + s.req) > q) x = *reinterpret_cast<const float4*>(p.state + own);
        float* slot = p.slots + (static_cast<int64_t>(s.base) * p.H + h) * D * D + at;
        const int64_t stride = static_cast<int64_t>(p.H) * D * D;
        constexpr int AHEAD = 8;  // loads do not wait for the sums
        for (int32_t i = 0; i < s.count; i += AHEAD) {
            float4 y[AHEAD];
            float a[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (i + u < s.count) {
                    y[u] = *reinterpret_cast<const float4*>(slot + (u + 1) * stride);
                    a[u] = p.seg_decay[static_cast<int64_t>(s.base + i + u) * p.H + h];
                }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (i + u < s.count) {
                    *reinterpret_cast<float4*>(slot + u * stride) = x;
                    x.x = fmaf(a[u], x.x, y[u].x);
                    x.y = fmaf(a[u], x.y, y[u].y);
                    x.z = fmaf(a[u], x.z, y[u].z);
                    x.w = fmaf(a[u], x.w, y[u].w);
                }
            slot += AHEAD * stride;
        }
        *reinterpret_cast<float4*>(p.state_out + own) = x;
    }
}

// -------------------------------------------------------------------- chunks
//
// One CTA walks the chunks of one (segment, head, slice of up to 128 value
// dims) with the state transposed, S^T (value dims x key dims), as fp32
// accumulators in tensor memory. A chunk of 64 tokens is four products of
// 16-bit operands (128 value dims are the M side, so that the widest one has
// the full 128 x 256 shape):
//   P (tokens x tokens)  = q k^T
//   O1^T (value x token) = S^T q^T            S^T as a bf16 copy in tensor memory
//   S^T                 += (decayed v)^T k    after S^T was scaled by exp(L_C)
//   O2^T                 = v^T P^T            P decayed, bf16, in shared memory
// q, k and v lie in shared memory as blocks of 64 elements a row with the
// 128-byte swizzle, which serve as K-major and as MN-major operands alike: no
// operand is transposed by a thread. Roundings to bf16: P and the state's copy,
// both below the rounding of the output; the decayed v as a sum of bf16 terms: two
// (16 bits) for the state that feeds later outputs of its segment, three (24
// bits) for states that leave the call, which retention_add works out apart:
// the tensor cores cut every sum towards zero, 2^-24 of it on average, so that
// a state added to for a whole prompt would lose some 10^-6 of itself. There
// a chunk's products start from zero and are added to the state in fp32, to
// nearest.

constexpr int kVal = 128;                  // value dims of a CTA (head_dim 64: 64 of its rows idle)
constexpr int kBlockBytes = kChunk * 128;  // 64 tokens x 64 elements
constexpr int kTensorCols = 512;

// Value dims a CTA really has, slices of a head, bytes of a chunk's q or k and v.
template <int D>
struct RetDims {
    static constexpr int VD = D < kVal ? D : kVal, NS = D / VD;
    static constexpr int KB = D / 64 * kBlockBytes, VB = VD / 64 * kBlockBytes;
    // an operand of 128 rows over a block of 64 reads on into what follows; at head_dim 64
    // that can be the end of the terms
    static constexpr int PAD = D == 64 ? kBlockBytes : 0;
};

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte piece j of row t in swizzled blocks of 8 pieces a row.
__device__ __forceinline__ uint32_t block_at(int t, int j) {
    return static_cast<uint32_t>((j >> 3) * kBlockBytes + t * 128 + (((j & 7) ^ (t & 7)) << 4));
}

// Rows of a chunk (PIECES 16-byte pieces each, `left` of them there, zeros behind) into
// swizzled blocks, by THREADS threads: each takes one piece of every few rows.
template <int PIECES, int THREADS>
__device__ __forceinline__ void load_rows(uint32_t dst, const __nv_bfloat16* src, int64_t stride, int32_t left,
                                          int thread) {
    constexpr int RS = THREADS / PIECES;  // rows a pass takes
    static_assert(RS >= 4 && (RS == 4 || RS % 8 == 0), "the swizzle of a thread's rows");
    const int t0 = thread / PIECES, j = thread % PIECES;
    const __nv_bfloat16* at = src + t0 * stride + j * 8;
#pragma unroll
    for (int t = 0; t < kChunk; t += RS) {
        const bool there = t0 + t < left;
        cp_async_16_or_zero(dst + block_at(t0 + t, j), there ? at : src, there);
        at += RS * stride;
    }
}

// exp(L_end - L_j) v_j as bf16 terms, each cut from what the ones before it leave, into
// `terms` (TERMS of VB bytes each); w: the factors of the chunk's tokens.
template <int VD, int VB, int TERMS, int THREADS>
__device__ __forceinline__ void decayed_terms(const uint8_t* v, uint8_t* terms, const float* w, int thread) {
#pragma unroll
    for (int x = thread; x < kChunk * (VD / 8); x += THREADS) {
        const int t = x / (VD / 8), j = x % (VD / 8);
        const uint32_t o = block_at(t, j);
        const uint4 in4 = *reinterpret_cast<const uint4*>(v + o);
        const float fw = w[t];
        const uint32_t in[4] = {in4.x, in4.y, in4.z, in4.w};
        uint32_t r0[4], r1[4], r2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo = bf16lo_to_f32(in[i]) * fw, hi = bf16hi_to_f32(in[i]) * fw;
            r0[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
            lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
            hi -= __uint_as_float(__float_as_uint(hi) & 0xffff0000u);
            r1[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
            if (TERMS == 3) {
                lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
                hi -= __uint_as_float(__float_as_uint(hi) & 0xffff0000u);
                r2[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
            }
        }
        *reinterpret_cast<uint4*>(terms + o) = make_uint4(r0[0], r0[1], r0[2], r0[3]);
        *reinterpret_cast<uint4*>(terms + VB + o) = make_uint4(r1[0], r1[1], r1[2], r1[3]);
        if (TERMS == 3) *reinterpret_cast<uint4*>(terms + 2 * VB + o) = make_uint4(r2[0], r2[1], r2[2], r2[3]);
    }
}

// A value that is not finite makes its dim's products with the weights NaN for all of a chunk's
// tokens, the earlier ones (weight 0) too. Rare: a warp whose lanes (value dim dv each) meet NaN
// (`again`) puts sum_(j <= t) P[t][j] v[j][dv] in their place, 32 tokens from t0 on at `at`. A call
// of its own, so that it takes no registers from the loop.
__device__ __noinline__ void sum_again(uint32_t at, bool again, const uint8_t* weights, const uint8_t* v, int t0,
                                       int dv) {
#pragma unroll 1
    for (int b = 0; b < 32; b += 16) {
        uint32_t x[16];
        tmem_ld(at + b, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (!again) continue;
            const int t = t0 + b + i;
            float a = 0.f;
#pragma unroll 1
            for (int j = 0; j <= t; ++j)
                a = fmaf(__bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(weights + block_at(t, j >> 3) + (j & 7) * 2)),
                         __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(v + block_at(j, dv >> 3) + (dv & 7) * 2)), a);
            x[i] = __float_as_uint(a);
        }
        __syncwarp();
        tmem_st(at + b, x);
        tmem_st_wait();
    }
}

// S^T (+)= (decayed v)^T k in TERMS bf16 terms, the smallest first: the tensor cores cut each
// sum to the accumulator's 24 bits (towards zero), which costs nothing while it is small. The
// issuing warp.
template <int D, int TERMS>
__device__ __forceinline__ void issue_update(uint32_t state, uint32_t terms, uint32_t k, bool add) {
    constexpr uint32_t ID = bf16_product(128, D, true, true);
#pragma unroll
    for (int u = TERMS - 1; u >= 0; --u)
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk)
            tmem_mma(state, smem_operand(terms + u * RetDims<D>::VB + kk * 2048, kBlockBytes, 1024),
                     smem_operand(k + kk * 2048, kBlockBytes, 1024), ID, add || u < TERMS - 1 || kk > 0);
}

// Log decays of chunk c of a segment: lane l has tokens 2l and 2l + 1 (0 behind the last).
__device__ __forceinline__ float2 chunk_decays(const RetParams& p, const RetSeg& sg, int32_t h, int32_t c, int lane) {
    const int64_t t0 = sg.token + static_cast<int64_t>(c) * kChunk;
    const int32_t left = sg.tokens - c * kChunk;
    return make_float2(2 * lane < left ? decay_of(p, t0 + 2 * lane, h) : 0.f,
                       2 * lane + 1 < left ? decay_of(p, t0 + 2 * lane + 1, h) : 0.f);
}
// Running sums over the chunk, up to and with tokens 2l and 2l + 1. (No sum takes a later token's
// decay in and out again: one that is not a number stays with the tokens from its own on.)
__device__ __forceinline__ void running_sums(float2 g, int lane, Sum& l0, Sum& l1) {
    const Sum g0 = in_log2(g.x);
    l1 = g0 + in_log2(g.y);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sum x = shfl_up(l1, off);
        if (lane >= off) l1 = l1 + x;
    }
    const Sum before = shfl_up(l1, 1);
    l0 = lane > 0 ? g0 + before : g0;
}

// States. Without FINAL, what each segment adds, from zero, into its slot; with FINAL, the
// state after each request without slots (of one segment). v is decayed to the segment's end,
// so that chunks only add up. Copies run ahead (k of the next chunk, v of the one after), and
// the terms of a chunk are worked out while the products of the one before run, which are done
// by then: a chunk (4500 clocks at head_dim 256, products 1600 of them) is terms, fold and
// copies one after the other. Products in two halves of the key dims, one folded while the
// other runs, read v's terms twice and took 114 us for 68; 16 warps instead of 8 gained 1 us
// at head_dim 256 and lost 2 at 128.
template <int D>
struct RetAddShape : RetDims<D> {
    using B = RetDims<D>;
    static constexpr int AT_V = 2 * B::KB, AT_W = AT_V + 3 * B::VB, AT_F = AT_W + 2 * 3 * B::VB + B::PAD;
    static constexpr int AT_T = AT_F + 2 * kChunk * 4;  // factors of two chunks, then decay sums of all
    static constexpr int SMEM = AT_T + kMaxChunks * 8 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool FINAL>
__global__ void __launch_bounds__(kAddThreads + 64, 1) retention_add(const RetParams p) {
    using S = RetAddShape<D>;
    constexpr int NS = S::NS, VD = S::VD, T = kAddThreads;
    extern __shared__ uint8_t ret_smem[];
    __shared__ __align__(8) uint64_t bar;  // a chunk's products
    __shared__ uint32_t tmem_base;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ret_smem) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(smem);
    float* const fac = reinterpret_cast<float*>(smem + S::AT_F);
    Sum* const totals = reinterpret_cast<Sum*>(smem + S::AT_T);
    if (FINAL) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (p.num_segs[1] == 0) return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool issuer = warp == T / 32;  // the warp that issues the products
    const bool decays = warp > T / 32;   // the warp that works out the factors
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    if (issuer) tmem_alloc(&tmem_base, kTensorCols);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");               // the segments are listed
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // single tokens may run beside this
    uint32_t ph = 0;
    bool bad = false;  // a wait has given up
    auto wait = [&]() {
        if (!bad && !mbar_wait_bounded(&bar, ph, kRetWaitNs)) bad = true;
        ph ^= 1;
        __syncwarp();  // the lanes have polled each for itself
        tmem_fence_after();
    };
    // A thread's columns of its lane: a half of D, CW at a time. Products in columns 0.., the
    // state in columns D...
    constexpr int PARTS = T / 128, CW = D / PARTS < 32 ? D / PARTS : 32;
    const int col0 = (warp >> 2) * (D / PARTS);
    auto fold = [&](bool first, float* dst) {  // the state += the products; its value to dst
        if (warp >= T / 32) return;
#pragma unroll
        for (int b = 0; b < D / PARTS / CW; ++b) {
            const int c0 = col0 + b * CW;
            uint32_t x[CW], y[CW];
            tmem_ld(tm + lanes + c0, x);
            if (!first) tmem_ld(tm + lanes + D + c0, y);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < CW; ++i)
                if (!first) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
            if (dst) {
                if (row < VD)
#pragma unroll
                    for (int i = 0; i < CW; ++i) dst[static_cast<int64_t>(c0 + i) * D + row] = __uint_as_float(x[i]);
            } else {
                tmem_st(tm + lanes + D + c0, x);
            }
        }
        tmem_st_wait();
    };
    const int32_t H_kv = p.H / p.G;
    const int32_t items = *p.num_segs * p.H * NS;
    for (int32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const RetSeg sg = p.segs[item / (p.H * NS)];
        if (sg.count == 0 || FINAL != (sg.slot < 0)) continue;
        const int32_t h = item / NS % p.H, dv0 = item % NS * VD, hk = h / p.G;
        const int32_t chunks = (sg.tokens + kChunk - 1) / kChunk;
        auto load_k = [&](int32_t c) {
            if (warp >= T / 32 || c >= chunks) return;
            const int64_t t0 = sg.token + static_cast<int64_t>(c) * kChunk;
            load_rows<D / 8, T>(base + (c & 1) * S::KB, p.k + (t0 * H_kv + hk) * D, static_cast<int64_t>(H_kv) * D,
                                sg.tokens - c * kChunk, tid);
        };
        auto load_v = [&](int32_t c) {
            if (warp >= T / 32 || c >= chunks) return;
            const int64_t t0 = sg.token + static_cast<int64_t>(c) * kChunk;
            load_rows<VD / 8, T>(base + S::AT_V + c % 3 * S::VB, p.v + (t0 * H_kv + hk) * D + dv0,
                                 static_cast<int64_t>(H_kv) * D, sg.tokens - c * kChunk, tid);
        };
        // factors of chunk c from its decays: one warp
        auto factors = [&](int32_t c, float2 g) {
            Sum l0, l1;
            running_sums(g, lane, l0, l1);
            Sum end = {0.f, 0.f};  // of this chunk and all after it
            for (int32_t x = c + lane; x < chunks; x += 32) end = end + totals[x];
            end = warp_total(end);
            *reinterpret_cast<float2*>(fac + (c & 1) * kChunk + 2 * lane) = make_float2(exp2f(end - l0), exp2f(end - l1));
        };
        __syncthreads();  // the previous item is done with shared and tensor memory
        load_v(0);
        load_k(0);
        load_v(1);
        cp_async_commit();
        if (warp < T / 32)
            for (int32_t c = warp; c < chunks; c += T / 32) {
                const float2 g = chunk_decays(p, sg, h, c, lane);
                const Sum t = warp_total(in_log2(g.x) + in_log2(g.y));
                if (lane == 0) totals[c] = t;
            }
        // factors are worked out a chunk ahead of the terms, from decays loaded a chunk before;
        // that takes as long as the terms and the fold together, so this warp meets the others
        // once a chunk only
        float2 g = make_float2(0.f, 0.f);
        __syncthreads();
        if (decays) {
            factors(0, chunk_decays(p, sg, h, 0, lane));
            g = chunk_decays(p, sg, h, 1, lane);
        }
        const int64_t state_at = static_cast<int64_t>(FINAL ? __ldg(p.where + sg.req) : sg.slot + 1) * p.H + h;
        float* const dst = (FINAL ? p.state_out : p.slots) + state_at * D * D + dv0;
        if (FINAL && warp < T / 32) {  // the state before the request, decayed to its end
            Sum t = {0.f, 0.f};
            for (int32_t x = lane; x < chunks; x += 32) t = t + totals[x];
            const float a = exp2f(warp_total(t).h);
            const int32_t q = __ldg(p.qsl + sg.req + 1) - __ldg(p.qsl + sg.req);
            const float* src = __ldg(p.seq_lens + sg.req) > q && row < VD ? p.state + state_at * D * D + dv0 : nullptr;
#pragma unroll
            for (int b = 0; b < D / PARTS / CW; ++b) {
                const int c0 = col0 + b * CW;
                uint32_t x[CW];
#pragma unroll
                for (int i = 0; i < CW; ++i)
                    x[i] = src ? __float_as_uint(a * src[static_cast<int64_t>(c0 + i) * D + row]) : 0u;
                tmem_st(tm + lanes + D + c0, x);
            }
            tmem_st_wait();
        }
        for (int32_t c = 0; c < chunks; ++c) {
            if (c == 0) cp_async_wait<0>();
            else cp_async_wait<1>();
            fence_proxy_async_smem();
            bad = __syncthreads_or(bad);  // v and the factors of chunk c are there
            if (bad) break;
            const uint32_t terms = S::AT_W + (c & 1) * 3 * S::VB;
            if (decays) {
                if (c + 1 < chunks) {
                    factors(c + 1, g);
                    g = chunk_decays(p, sg, h, c + 2, lane);
                }
                continue;
            }
            if (!issuer)
                decayed_terms<VD, S::VB, 3, T>(smem + S::AT_V + c % 3 * S::VB, smem + terms, fac + (c & 1) * kChunk, tid);
            cp_async_wait<0>();  // k of chunk c
            fence_proxy_async_smem();
            if (c > 0) {  // the chunk before: done with its k and terms
                wait();
                fold(!FINAL && c == 1, nullptr);
            }
            tmem_fence_before();
            __syncwarp();
            asm volatile("bar.sync 1, %0;" ::"n"(T + 32) : "memory");  // all but the factors' warp
            tmem_fence_after();
            if (issuer) {
                issue_update<D, 3>(tm, base + terms, base + (c & 1) * S::KB, false);
                tmem_commit(&bar);
            }
            load_k(c + 1);
            load_v(c + 2);
            cp_async_commit();
        }
        if (!bad && !decays) wait();
        bad = __syncthreads_or(bad);
        if (bad) break;
        fold(!FINAL && chunks == 1, dst);
        if (!FINAL && dv0 == 0 && warp == 0) {  // the segment's decay
            Sum t = {0.f, 0.f};
            for (int32_t x = lane; x < chunks; x += 32) t = t + totals[x];
            t = warp_total(t);
            if (lane == 0) p.seg_decay[static_cast<int64_t>(sg.slot) * p.H + h] = exp2f(t.h);
        }
        tmem_fence_before();
    }
    cp_async_wait<0>();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (bad && tid == 0) set_err(p.err, YOCO_DEVERR_TIMEOUT);
    if (issuer) tmem_dealloc(tm, kTensorCols);
}

// Outputs, chunk by chunk. Three groups of warps meet three times a chunk:
//   8 state warps   scale the state and copy it to bf16, then (those whose lanes hold
//                   tokens) decay P, the others copy the next chunk's k
//   8 value warps   work out the terms of v, then copy the next chunk's q and v and write
//                   the outputs of the chunk before
//   1 issuing warp  P | O1 and the state's update | O2
//   1 warp          the next chunk's factors; it meets the others once a chunk (in a loading
//                   warp they were the longest of its third: 184 us against 181 for 16 sequences
//                   with 4 prompts, 10000 tokens)
// A chunk at head_dim 256 takes 6800 clocks: 1000 to the first meeting (outputs of the chunk
// before out of tensor memory), 2100 to the second (P, and v's terms), 3700 to the third (P
// decayed, copies, stores). Its products need 2700, the shared memory they and the copies pass
// through 3100; the tensor cores are 28% busy, DRAM 21%.
// so that copies, arithmetic, stores and products of one and the next chunk overlap.
template <int D>
struct RetOutShape : RetDims<D> {
    using B = RetDims<D>;
    static constexpr int STAGE = 2 * B::KB + B::VB;  // q, k, v
    static constexpr int AT_W = 2 * STAGE, AT_P = AT_W + 2 * B::VB, AT_F = AT_P + kBlockBytes + B::PAD;
    // of each of 4 chunks, for its 64 tokens t: the running sum L_t (high and low parts, log2
    // units), exp(L_t), exp(L_end - L_t), exp(L_t - L_mid), exp(L_mid - L_t)
    static constexpr int FACTORS = 6;
    // then of each exp(L_C), and whether L_mid serves (the chunk's sums span less than 2^100)
    static constexpr int SMEM = AT_F + 4 * (FACTORS * kChunk * 4 + 8) + 1024;
    // tensor memory columns: S^T, its bf16 copy, O1^T, O2^T (and P before it)
    static constexpr int TS = 0, TC = D, TO1 = D + D / 2, TO2 = TO1 + kChunk;
    static_assert(TO2 + kChunk <= kTensorCols, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kOutThreads + 64, 1) retention_out(const RetParams p) {
    using S = RetOutShape<D>;
    constexpr int NS = S::NS, VD = S::VD, F = S::FACTORS * kChunk;
    constexpr int CW = D / 2 < 32 ? D / 2 : 32;  // columns of a step through a state warp's half
    constexpr int HT = kChunk / 2;               // tokens of a half of a chunk
    extern __shared__ uint8_t ret_smem[];
    __shared__ __align__(8) uint64_t bar_p, bar_o, bar_s;
    __shared__ uint32_t tmem_base;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ret_smem) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_u32(smem);
    float* const fac = reinterpret_cast<float*>(smem + S::AT_F);
    float2* const whole = reinterpret_cast<float2*>(fac + 4 * F);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool of_state = warp < 8, of_value = warp >= 8 && warp < 16, issuer = warp == 16;
    const bool decays = warp == 17;
    const bool loader = of_state && (warp & 2);   // state warps without tokens: 2, 3, 6, 7
    const int half = (warp >> 2) & 1;             // which half of the columns this warp takes
    const int row = (warp & 3) * 32 + lane;       // its lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    if (tid == 0) {
        mbar_init(&bar_p, 1);
        mbar_init(&bar_o, 1);
        mbar_init(&bar_s, 1);
        fence_mbar_init();
    }
    if (issuer) tmem_alloc(&tmem_base, kTensorCols);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the segments and their states are there
    // Phases of the barriers. P: waited for by the token warps; O: by the value warps; the
    // state's update: by the state warps. Each is waited for before the chunk's products that
    // complete it next are issued.
    uint32_t ph_p = 0, ph_o = 0, ph_s = 0;
    bool bad = false;  // a wait has given up
    auto wait = [&](uint64_t* bar, uint32_t& ph) {
        if (!bad && !mbar_wait_bounded(bar, ph, kRetWaitNs)) bad = true;
        ph ^= 1;
        __syncwarp();  // the lanes have polled each for itself
    };
    auto meet = [] {  // all but the factors' warp
        __syncwarp();
        asm volatile("bar.sync 1, %0;" ::"n"(kOutThreads + 32) : "memory");
    };
    const int32_t H_kv = p.H / p.G;
    const int32_t items = *p.num_segs * p.H * NS;

    for (int32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const RetSeg sg = p.segs[item / (p.H * NS)];
        if (sg.count == 0) continue;
        const int32_t h = item / NS % p.H, dv0 = item % NS * VD, hk = h / p.G;
        const int32_t chunks = (sg.tokens + kChunk - 1) / kChunk;
        // chunk c into its stage: k by the 128 loader threads, q and v by the value warps
        auto load = [&](int32_t c) {
            const uint32_t st = base + (c & 1) * S::STAGE;
            const int32_t left = sg.tokens - c * kChunk;
            const int64_t t0 = sg.token + static_cast<int64_t>(c) * kChunk;
            if (of_state) {
                load_rows<D / 8, 128>(st + S::KB, p.k + (t0 * H_kv + hk) * D, static_cast<int64_t>(H_kv) * D, left,
                                      (half * 2 + (warp & 1)) * 32 + lane);
            } else {
                load_rows<D / 8, 256>(st, p.q + (t0 * p.H + h) * D, static_cast<int64_t>(p.H) * D, left, tid - 256);
                load_rows<VD / 8, 256>(st + 2 * S::KB, p.v + (t0 * H_kv + hk) * D + dv0, static_cast<int64_t>(H_kv) * D,
                                       left, tid - 256);
            }
            cp_async_commit();
        };
        const bool copies = loader || of_value;
        auto factors = [&](int32_t c, float2 g) {  // from the chunk's decays: one warp
            Sum l0, l1;
            running_sums(g, lane, l0, l1);
            auto of_lane = [](Sum a, int l) {
                return Sum{__shfl_sync(0xffffffffu, a.h, l), __shfl_sync(0xffffffffu, a.l, l)};
            };
            const Sum end = of_lane(l1, 31), first = of_lane(l0, 0), mid = of_lane(l0, 16);
            auto put = [&](int i, float x, float y) {
                *reinterpret_cast<float2*>(fac + (c & 3) * F + i * kChunk + 2 * lane) = make_float2(x, y);
            };
            put(0, l0.h, l1.h);
            put(1, l0.l, l1.l);
            put(2, exp2f(l0.h), exp2f(l1.h));
            put(3, exp2f(end - l0), exp2f(end - l1));
            put(4, exp2f(l0 - mid), exp2f(l1 - mid));
            put(5, exp2f(mid - l0), exp2f(mid - l1));
            if (lane == 0) whole[c & 3] = make_float2(exp2f(end.h), fabsf(first - end) < 100.f ? 1.f : 0.f);
        };
        __syncthreads();  // the previous item is done with shared and tensor memory
        if (copies) load(0);
        float2 g = make_float2(0.f, 0.f);  // decays of the chunk after next
        if (decays) {
            factors(0, chunk_decays(p, sg, h, 0, lane));
            g = chunk_decays(p, sg, h, 1, lane);
        }
        if (of_state) {  // the state before the segment
            const float* src = nullptr;
            const int32_t q = __ldg(p.qsl + sg.req + 1) - __ldg(p.qsl + sg.req);
            if (sg.slot >= 0)
                src = p.slots + (static_cast<int64_t>(sg.slot) * p.H + h) * D * D + dv0;
            else if (__ldg(p.seq_lens + sg.req) > q)
                src = p.state + (static_cast<int64_t>(__ldg(p.where + sg.req)) * p.H + h) * D * D + dv0;
            if (row >= VD) src = nullptr;
#pragma unroll
            for (int b = 0; b < D / 2 / CW; ++b) {
                const int c0 = half * (D / 2) + b * CW;
                uint32_t x[CW];
#pragma unroll
                for (int i = 0; i < CW; ++i)
                    x[i] = src ? __float_as_uint(src[static_cast<int64_t>(c0 + i) * D + row]) : 0u;
                tmem_st(tm + lanes + S::TS + c0, x);
            }
            tmem_st_wait();
        }
        bool pending = false;  // an update of the state is under way
        uint32_t y[HT / 2];    // value warps: outputs of the chunk before, two tokens a word
        auto take_outputs = [&](int32_t c) {  // of chunk c, from tensor memory
            wait(&bar_o, ph_o);
            tmem_fence_after();
            const float* et = fac + (c & 3) * F + 2 * kChunk + half * HT;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t o1[16], o2[16];
                tmem_ld(tm + lanes + S::TO1 + half * HT + b * 16, o1);
                tmem_ld(tm + lanes + S::TO2 + half * HT + b * 16, o2);
                tmem_ld_wait();
                if (b == 0) {
                    const bool again = row < VD && isnan(__uint_as_float(o2[0]));
                    if (__any_sync(0xffffffffu, again)) {
                        sum_again(tm + lanes + S::TO2 + half * HT, again, smem + S::AT_P,
                                  smem + (c & 1) * S::STAGE + 2 * S::KB, half * HT, row);
                        tmem_ld(tm + lanes + S::TO1 + half * HT, o1);
                        tmem_ld(tm + lanes + S::TO2 + half * HT, o2);
                        tmem_ld_wait();
                    }
                }
#pragma unroll
                for (int t = 0; t < 16; t += 2) {
                    const float2 e = *reinterpret_cast<const float2*>(et + b * 16 + t);
                    y[b * 8 + t / 2] =
                        pack_bf16x2(p.scale * fmaf(e.x, __uint_as_float(o1[t]), __uint_as_float(o2[t])),
                                    p.scale * fmaf(e.y, __uint_as_float(o1[t + 1]), __uint_as_float(o2[t + 1])));
                }
            }
        };
        auto write_outputs = [&](int32_t c) {
            // two lanes exchange, so that each writes two value dims of every other token: a
            // warp's 32 lanes are 64 bytes of two tokens' rows
            const int odd = lane & 1;
            const int32_t left = sg.tokens - c * kChunk - half * HT - odd;
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                p.out + ((sg.token + static_cast<int64_t>(c) * kChunk + half * HT + odd) * p.H + h) * D + dv0 + (row & ~1));
            const int64_t step = static_cast<int64_t>(p.H) * D;  // two tokens on, in words
#pragma unroll
            for (int t = 0; t < HT; t += 2) {
                const uint32_t z = __shfl_xor_sync(0xffffffffu, y[t / 2], 1);
                if (row < VD && t < left) *dst = odd ? __byte_perm(z, y[t / 2], 0x7632) : __byte_perm(y[t / 2], z, 0x5410);
                dst += step;
            }
        };

        for (int32_t c = 0; c < chunks; ++c) {
            const uint32_t at = (c & 1) * S::STAGE;  // of the chunk's q, k, v
            const uint32_t sq = base + at, sk = sq + S::KB, sv = sk + S::KB;
            const float* f = fac + (c & 3) * F;
            const bool update = c + 1 < chunks;
            if (copies) {
                cp_async_wait<0>();
                fence_proxy_async_smem();
            }
            if (of_state && pending) wait(&bar_s, ph_s);  // the state before this chunk is complete
            pending = update;
            if (of_value && c > 0) take_outputs(c - 1);
            tmem_fence_before();
            bad = __syncthreads_or(bad);  // (1) chunk c, its factors and its place are there
            if (bad) break;
            if (decays) {  // meets the others here alone
                if (update) {
                    factors(c + 1, g);
                    g = chunk_decays(p, sg, h, c + 2, lane);
                }
                continue;
            }
            tmem_fence_after();
            if (issuer) {  // P = q k^T (128 rows: the upper 64 are not looked at)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk >> 2) * kBlockBytes + (kk & 3) * 32;
                    tmem_mma(tm + S::TO2, smem_operand(sq + o, 16, 1024), smem_operand(sk + o, 16, 1024),
                             bf16_product(128, kChunk, false, false), kk > 0);
                }
                tmem_commit(&bar_p);
            } else if (of_state) {  // the state as a bf16 operand, then scaled by the chunk's decay
                const float aC = whole[c & 3].x;
#pragma unroll
                for (int b = 0; b < D / 2 / CW; ++b) {
                    const int c0 = half * (D / 2) + b * CW;
                    uint32_t x[CW], z[CW / 2];
                    tmem_ld(tm + lanes + S::TS + c0, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < CW / 2; ++i) {
                        z[i] = pack_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                        x[2 * i] = __float_as_uint(__uint_as_float(x[2 * i]) * aC);
                        x[2 * i + 1] = __float_as_uint(__uint_as_float(x[2 * i + 1]) * aC);
                    }
                    tmem_st(tm + lanes + S::TC + c0 / 2, z);
                    if (update) tmem_st(tm + lanes + S::TS + c0, x);
                }
                tmem_st_wait();
            } else if (update) {
                decayed_terms<VD, S::VB, 2, 256>(smem + at + 2 * S::KB, smem + S::AT_W, f + 3 * kChunk, tid - 256);
                fence_proxy_async_smem();
            }
            tmem_fence_before();
            meet();  // (2) the state's copy and the terms are complete
            tmem_fence_after();
            if (issuer) {  // O1^T = S^T q^T, and the state after the chunk
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tmem_mma_ta(tm + S::TO1, tm + S::TC + kk * 8,
                                smem_operand(sq + (kk >> 2) * kBlockBytes + (kk & 3) * 32, 16, 1024),
                                bf16_product(128, kChunk, false, false), kk > 0);
                if (update) {
                    issue_update<D, 2>(tm + S::TS, base + S::AT_W, sk, true);
                    tmem_commit(&bar_s);
                }
            } else if (of_value) {
                if (c + 1 < chunks) load(c + 1);
                if (c > 0) write_outputs(c - 1);
            } else if (loader) {
                if (c + 1 < chunks) load(c + 1);  // its stage: the products of chunk c - 1 are done
            } else {  // weights of token `row` for 32 tokens
                wait(&bar_p, ph_p);
                tmem_fence_after();
                uint8_t* dst = smem + S::AT_P;
                if ((warp & 3) < half) {  // all later tokens
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4*>(dst + block_at(row, half * 4 + i)) = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    uint32_t x[HT];
                    tmem_ld(tm + lanes + S::TO2 + half * HT, x);
                    tmem_ld_wait();
                    const bool near = whole[c & 3].y != 0.f, diagonal = (warp & 3) == half;
                    const float th = f[row], tl = f[kChunk + row], tf = f[4 * kChunk + row];
#pragma unroll
                    for (int q4 = 0; q4 < HT / 4; ++q4) {
                        const int j0 = half * HT + q4 * 4;
                        float w[4];
                        if (near) {  // one factor of the row, one of the column
                            const float4 m = *reinterpret_cast<const float4*>(f + 5 * kChunk + j0);
                            w[0] = tf * m.x;
                            w[1] = tf * m.y;
                            w[2] = tf * m.z;
                            w[3] = tf * m.w;
                        } else {
                            const float4 jh = *reinterpret_cast<const float4*>(f + j0);
                            const float4 jl = *reinterpret_cast<const float4*>(f + kChunk + j0);
                            w[0] = exp2_approx((th - jh.x) + (tl - jl.x));
                            w[1] = exp2_approx((th - jh.y) + (tl - jl.y));
                            w[2] = exp2_approx((th - jh.z) + (tl - jl.z));
                            w[3] = exp2_approx((th - jh.w) + (tl - jl.w));
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            w[i] *= __uint_as_float(x[q4 * 4 + i]);
                            if (diagonal && j0 + i > row) w[i] = 0.f;
                        }
                        *reinterpret_cast<uint2*>(dst + block_at(row, half * 4 + (q4 >> 1)) + (q4 & 1) * 8) =
                            make_uint2(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]));
                    }
                }
                fence_proxy_async_smem();
            }
            tmem_fence_before();
            meet();  // (3) P is in shared memory, its columns are free
            tmem_fence_after();
            if (issuer) {  // O2^T = v^T P^T
#pragma unroll
                for (int kk = 0; kk < kChunk / 16; ++kk)
                    tmem_mma(tm + S::TO2, smem_operand(sv + kk * 2048, kBlockBytes, 1024),
                             smem_operand(base + S::AT_P + kk * 32, 16, 1024), bf16_product(128, kChunk, true, false),
                             kk > 0);
                tmem_commit(&bar_o);
            }
        }
        if (!bad) {
            if (of_value) {
                take_outputs(chunks - 1);
                write_outputs(chunks - 1);
            }
        }
        bad = __syncthreads_or(bad);
        if (bad) break;
        tmem_fence_after();
        tmem_fence_before();
    }
    cp_async_wait<0>();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (bad && tid == 0) set_err(p.err, YOCO_DEVERR_TIMEOUT);
    if (issuer) tmem_dealloc(tm, kTensorCols);
}

// ------------------------------------------------------------------ host side

constexpr int kMinSegment = 256;  // tokens

// Segments to aim for: about two CTAs for every SM over heads and slices.
int64_t ret_target(int H, int D) {
    const int64_t units = static_cast<int64_t>(H) * (D > kVal ? D / kVal : 1);
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
    if (seg > kMaxSegment) seg = kMaxSegment;
    x.seg_tokens = seg;
    // whole segments, and at most one shorter one for each request of two tokens or more
    const int64_t shorter = R < T / 2 ? R : T / 2;
    const int64_t cut = max_q > seg ? T / seg : 0;
    x.max_segs = T / seg + shorter;
    x.max_slots = 3 * cut;  // at most n + 1 for a request of n > 1 segments, n / 2 of them whole
    return x;
}

// Workspace of the largest plan up to these bounds.
RetPlan ret_sizes(int64_t R, int64_t T, int64_t max_q, int H, int D) {
    RetPlan x = ret_plan(R, T, max_q, H, D);
    if (x.seg_tokens == 0) return x;
    int64_t whole = ret_target(H, D);
    if (whole < T / kMaxSegment) whole = T / kMaxSegment;
    if (whole > T / kMinSegment) whole = T / kMinSegment;
    const int64_t segs = whole + (R < T / 2 ? R : T / 2), slots = max_q > kMinSegment ? 3 * whole : 0;
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
    const unsigned steps = static_cast<unsigned>(static_cast<int64_t>(p.num_reqs) * p.H * (D / kSlice));
    const bool cut = p.seg_tokens > 0 && p.max_slots > 0;
    cudaError_t e;
    if (!cut) {
        retention_step<D><<<steps, 256, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess || p.seg_tokens == 0) return e;
    }
    static unsigned long long done_out = 0, done_add = 0, done_final = 0;
    e = ret_smem_attr(retention_out<D>, RetOutShape<D>::SMEM, done_out);
    if (e == cudaSuccess) e = ret_smem_attr(retention_add<D, false>, RetAddShape<D>::SMEM, done_add);
    if (e == cudaSuccess) e = ret_smem_attr(retention_add<D, true>, RetAddShape<D>::SMEM, done_final);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), units = p.H * RetDims<D>::NS;
    const int64_t items = static_cast<int64_t>(p.max_segs) * units;
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);  // one CTA an SM
    retention_plan<<<1, 1024, 0, s>>>(p, units, sms);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The chunk passes start while the kernel before them ends (they wait for it before
    // they read), single tokens beside the segments' pass: bound by HBM next to products.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cut) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kAddThreads + 64);
        cfg.dynamicSmemBytes = RetAddShape<D>::SMEM;
        e = cudaLaunchKernelEx(&cfg, retention_add<D, false>, p);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(steps);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, retention_step<D>, p);
        if (e != cudaSuccess) return e;
        const int64_t parts = static_cast<int64_t>(p.max_segs) * p.H * (D * D / 1024);
        retention_scan<D><<<static_cast<unsigned>(parts < 16 * sms ? parts : 16 * sms), 256, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kOutThreads + 64);
    cfg.dynamicSmemBytes = RetOutShape<D>::SMEM;
    e = cudaLaunchKernelEx(&cfg, retention_out<D>, p);
    if (e != cudaSuccess) return e;
    // requests without slots: their states may lie in the place of those that the outputs
    // start from, so they are written last
    cfg.blockDim = dim3(kAddThreads + 64);
    cfg.dynamicSmemBytes = RetAddShape<D>::SMEM;
    return cudaLaunchKernelEx(&cfg, retention_add<D, true>, p);
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
    if (out == q || out == k || out == v) return YOCO_ERR_INVALID_ARG;  // read while it is written
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
