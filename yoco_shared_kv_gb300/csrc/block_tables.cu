// yoco_build_block_tables: extend the block tables by the pages a step's new
// tokens need and work out every token's slot, from request lengths alone.
//
// "KV cache memory systems", "Contiguous allocation wastes capacity": a
// request's logical blocks map through its block table to physical pages that
// are handed out as it grows; "You Only Cache Once, in vLLM" names the
// block_table_tensor and slot_mapping of a step's metadata.
//
// Request r with q scheduled tokens and seq tokens after the step holds
// ceil((seq - q) / bs) pages and needs ceil(seq / bs). The n-th page taken in
// the whole step (requests in order, then logical order) is the n-th from the
// top of the free stack, so a page's identity follows from a running sum over
// the requests alone.
//
// Design: bound by latency (the metadata is a few KB), so the call is one
// launch without any wait between CTAs. A CTA of 256 tokens sums the demand of
// the requests before its first token itself (one coalesced pass, which also
// finds that request), then scans on over the requests that its tokens belong
// to. The token that opens a page writes the table entry. One more CTA walks
// all requests for the count of pages left and the error bits. Every CTA
// repeating the sum costs less than a second launch or a look back along the
// CTAs: replayed from a graph a call takes 3.1 us for 64 requests of a token
// (an empty launch takes 2) and 5.4 us for 1500 of one and 12 prompts, 26000
// tokens together (bytes: 0.02 us).
#include "common.cuh"

namespace yoco {
namespace {

constexpr int kTableThreads = 256;

struct Request {
    int32_t q0, q1;      // its tokens
    int32_t first;       // position of its first token
    int32_t held;        // pages already in its table row
    int32_t take;        // pages to take from the free stack
    int32_t bad;         // YOCO_DEVERR_* of unusable lengths, 0 if fine
};

__device__ __forceinline__ Request load_request(const int32_t* __restrict__ qsl,
                                                const int32_t* __restrict__ seq_lens, int32_t r,
                                                int32_t num_tokens, int32_t bshift,
                                                int32_t max_blocks, bool take_pages) {
    Request x;
    x.q0 = __ldg(qsl + r);
    x.q1 = __ldg(qsl + r + 1);
    const int32_t seq = __ldg(seq_lens + r);
    x.bad = 0;
    x.first = x.held = x.take = 0;
    if (x.q0 < 0 || x.q1 < x.q0 || x.q1 > num_tokens) {
        x.bad = YOCO_DEVERR_OFFSETS;
        return x;
    }
    const int32_t q = x.q1 - x.q0;
    if (q == 0) return x;  // schedules nothing: its row and lengths are not looked at
    const int32_t need = seq <= 0 ? 0 : ((seq - 1) >> bshift) + 1;
    if (seq < q || need > max_blocks) {
        x.bad = YOCO_DEVERR_POS_RANGE;
        return x;
    }
    x.first = seq - q;
    x.held = !take_pages ? need : x.first == 0 ? 0 : ((x.first - 1) >> bshift) + 1;
    x.take = need - x.held;
    return x;
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Exclusive running sum over the CTA's threads; `total` gets the sum. Ends
// with the scratch free for the next call.
__device__ __forceinline__ int64_t block_excl_scan(int64_t v, int64_t* warp_tot, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kTableThreads / 32; ++w) {
        const int64_t t = warp_tot[w];
        if (w < warp) before += t;
        total += t;
    }
    __syncthreads();
    return before + incl - v;
}

__global__ void __launch_bounds__(kTableThreads)
    block_tables_kernel(int32_t* block_table, int32_t max_blocks,
                        const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ qsl,
                        int32_t num_reqs, int32_t num_tokens, int32_t num_blocks, int32_t bshift,
                        const int32_t* __restrict__ free_pages, int32_t free_capacity,
                        const int32_t* __restrict__ num_free, int32_t* num_free_after,
                        int32_t* __restrict__ slots, int32_t* err) {
    __shared__ int64_t warp_tot[kTableThreads / 32];
    __shared__ int32_t s_end[kTableThreads];   // q1 of the requests in hand
    __shared__ int64_t s_excl[kTableThreads];  // pages taken before each
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool take = free_pages != nullptr;
    const int32_t stated = take ? __ldg(num_free) : 0;
    const int32_t avail = min(max(stated, 0), free_capacity);

    if (blockIdx.x == 0) {  // the pages left, and the error bits of the requests
        int64_t carry = 0, taken = 0;
        int32_t bits = avail != stated ? YOCO_DEVERR_OFFSETS : 0;
        for (int32_t base = 0; base < num_reqs; base += kTableThreads) {
            const int32_t r = base + tid;
            Request x = {};
            if (r < num_reqs)
                x = load_request(qsl, seq_lens, r, num_tokens, bshift, max_blocks, take);
            int64_t total;
            const int64_t end = carry + block_excl_scan(x.take, warp_tot, total) + x.take;
            bits |= x.bad;
            if (end <= avail) taken = end;  // the sums rise: the last that fits is the largest
            else if (x.take > 0) bits |= YOCO_DEVERR_NO_PAGES;
            carry += total;
        }
        if (bits) set_err(err, bits);
        if (num_free_after != nullptr) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const int64_t t = __shfl_xor_sync(0xffffffffu, taken, off);
                taken = t > taken ? t : taken;
            }
            if (lane == 0) warp_tot[warp] = taken;
            __syncthreads();
            if (tid == 0) {
                for (int w = 1; w < kTableThreads / 32; ++w)
                    taken = warp_tot[w] > taken ? warp_tot[w] : taken;
                *num_free_after = avail - static_cast<int32_t>(taken);
            }
        }
        return;
    }

    const int32_t t0 = static_cast<int32_t>(blockIdx.x - 1) * kTableThreads;
    const int32_t t = t0 + tid;
    // the requests that end at or before this CTA's first token: how many, and their demand
    int64_t before = 0;
    int32_t count = 0;
#pragma unroll 4
    for (int32_t r = tid; r < num_reqs; r += kTableThreads) {
        const Request x = load_request(qsl, seq_lens, r, num_tokens, bshift, max_blocks, take);
        if (x.q1 <= t0) {
            ++count;
            before += x.take;
        }
    }
    int64_t r_first;
    {
        const int64_t c = warp_sum(count), b = warp_sum(before);
        if (lane == 0) {
            warp_tot[warp] = b;
            s_end[warp] = static_cast<int32_t>(c);
        }
        __syncthreads();
        r_first = before = 0;
        for (int w = 0; w < kTableThreads / 32; ++w) {
            before += warp_tot[w];
            r_first += s_end[w];
        }
        __syncthreads();
    }
    int32_t slot = -1;
    bool placed = t >= num_tokens || t >= __ldg(qsl + num_reqs);  // padding behind the last request
    const int32_t t_last = min(t0 + kTableThreads, num_tokens) - 1;
    for (int64_t base = r_first; base < num_reqs; base += kTableThreads) {
        const int64_t r = base + tid;
        Request x = {};
        if (r < num_reqs)
            x = load_request(qsl, seq_lens, static_cast<int32_t>(r), num_tokens, bshift, max_blocks,
                             take);
        int64_t total;
        const int64_t excl = before + block_excl_scan(x.take, warp_tot, total);
        s_end[tid] = r < num_reqs ? x.q1 : 0x7fffffff;
        s_excl[tid] = excl;
        __syncthreads();
        const int n = static_cast<int>(min(static_cast<int64_t>(kTableThreads), num_reqs - base));
        if (!placed && t < s_end[n - 1]) {
            int lo = 0, hi = n - 1;  // first request in hand that ends after t
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_end[mid] > t) hi = mid;
                else lo = mid + 1;
            }
            placed = true;
            const int64_t row = base + lo;
            const Request y = load_request(qsl, seq_lens, static_cast<int32_t>(row), num_tokens,
                                           bshift, max_blocks, take);
            const bool served = y.take == 0 || s_excl[lo] + y.take <= avail;
            if (y.bad == 0 && y.q0 <= t && served) {
                const int32_t pos = y.first + (t - y.q0);
                const int32_t lp = pos >> bshift, in_page = pos & ((1 << bshift) - 1);
                int32_t* entry = block_table + row * max_blocks + lp;
                int32_t page;
                if (lp < y.held) {
                    page = *entry;
                } else {
                    page = __ldg(free_pages + (avail - 1 - (s_excl[lo] + lp - y.held)));
                    if (page < 0 || page >= num_blocks) page = -1;
                    if (in_page == 0) *entry = page;  // this token opens the page
                }
                if (page < 0 || page >= num_blocks) set_err(err, YOCO_DEVERR_PAGE_RANGE);
                else slot = (page << bshift) + in_page;
            } else if (y.bad == 0 && y.q0 > t) {
                set_err(err, YOCO_DEVERR_OFFSETS);  // a token before every request
            }
        }
        if (s_end[n - 1] > t_last) break;  // the same for every thread
        before += total;
        __syncthreads();  // the next round overwrites the requests in hand
    }
    if (t < num_tokens) slots[t] = slot;
}

}  // namespace
}  // namespace yoco

extern "C" yoco_status_t yoco_build_block_tables(
    int32_t* block_table, int32_t max_blocks_per_req, const int32_t* seq_lens,
    const int32_t* query_start_loc, int32_t num_reqs, int32_t num_tokens, int32_t num_blocks,
    int32_t block_size, const int32_t* free_pages, int32_t free_capacity, const int32_t* num_free,
    int32_t* num_free_after, int32_t* slot_mapping, int32_t* err_word, void* stream) {
    using namespace yoco;
    if (!block_size_ok(block_size)) return YOCO_ERR_UNSUPPORTED;
    if (num_reqs < 0 || num_tokens < 0 || num_blocks <= 0 || max_blocks_per_req <= 0 ||
        free_capacity < 0)
        return YOCO_ERR_INVALID_ARG;
    // a slot is an int32, and so is a token's index in the last CTA
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7fffffffll ||
        num_tokens > 0x7fffffff - kTableThreads)
        return YOCO_ERR_UNSUPPORTED;
    if (free_pages != nullptr && (!num_free || !num_free_after)) return YOCO_ERR_INVALID_ARG;
    // every CTA reads the count while one of them writes the new one
    if (num_free != nullptr && num_free == num_free_after) return YOCO_ERR_INVALID_ARG;
    if (!query_start_loc || (num_reqs > 0 && (!block_table || !seq_lens)) ||
        (num_tokens > 0 && !slot_mapping))
        return YOCO_ERR_INVALID_ARG;
    if (free_pages == nullptr) num_free = num_free_after = nullptr;  // nothing is taken
    const int64_t ctas = 1 + (static_cast<int64_t>(num_tokens) + kTableThreads - 1) / kTableThreads;
    block_tables_kernel<<<static_cast<unsigned>(ctas), kTableThreads, 0,
                          static_cast<cudaStream_t>(stream)>>>(
        block_table, max_blocks_per_req, seq_lens, query_start_loc, num_reqs, num_tokens,
        num_blocks, block_size == 16 ? 4 : 5, free_pages, free_capacity, num_free, num_free_after,
        slot_mapping, err_word);
    return cuda_status(cudaGetLastError());
}
