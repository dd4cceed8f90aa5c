// Upkeep of a paged K/V cache on the device: block tables and slot maps from
// request lengths (attn_paged_plan), and new K/V rows into their slots
// (attn_paged_write).
#include <cuda_runtime.h>

#include "packed.h"

namespace exattn {
namespace {

// ------------------------------------------------------------ plan
// need_i = ceil((old_i + new_i) / page) - ceil(old_i / page) pages for request
// i, taken from the top of the free stack in request order; token t of request
// i goes to slot table[i, pos / page] * page + pos % page, pos = old_i + j.
//
// The work is a prefix sum over the requests followed by independent fills,
// and bound by latency (a decode step's tables are a few KB). Every block
// works the whole prefix sum out for itself (8 bytes per request, from L2),
// so one launch does it without any block waiting for another; it then fills
// its own share of the tokens and of the table rows. Requests are taken
// kPlanChunk at a time through shared memory, with the sums carried over.
// (48 requests: 9.5 us a call, of which the host takes 9; 700 requests with
// 105,000 new tokens: 10.5 us.)
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = 4;
constexpr int kPlanChunk = kPlanThreads * kPlanPer;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
    __shared__ int64_t s_tok[kPlanChunk + 1];   // first token of each request of the chunk
    __shared__ int64_t s_page[kPlanChunk + 1];  // first of its new pages
    __shared__ int s_old[kPlanChunk];
    __shared__ int64_t s_wt[kPlanThreads / 32], s_wp[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    const int64_t free_n = min(max(__ldg(a.free_count), 0), a.num_free);
    // this block's tokens and requests
    const int64_t t0 = a.max_tokens * blockIdx.x / gridDim.x, t1 = a.max_tokens * (blockIdx.x + 1) / gridDim.x;
    const int r0 = static_cast<int>(static_cast<int64_t>(a.b) * blockIdx.x / gridDim.x);
    const int r1 = static_cast<int>(static_cast<int64_t>(a.b) * (blockIdx.x + 1) / gridDim.x);
    auto pages = [&](int64_t n) { return static_cast<int>((min(n, cap) + a.page_size - 1) / a.page_size); };
    // the free stack's page k places below its top (-1: none left)
    auto taken = [&](int64_t k) { return k < free_n ? __ldg(a.free_pages + (free_n - 1 - k)) : -1; };

    int64_t tok0 = 0, page0 = 0;  // before this chunk
    for (int i0 = 0; i0 < a.b; i0 += kPlanChunk) {
        // each thread sums kPlanPer neighbours, then warps and the block
        int old[kPlanPer], fresh[kPlanPer], need[kPlanPer];
        int64_t st = 0, sp = 0;
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int i = i0 + tid * kPlanPer + k;
            old[k] = i < a.b ? max(__ldg(a.seqlens + i), 0) : 0;
            fresh[k] = i < a.b ? max(__ldg(a.new_lens + i), 0) : 0;
            need[k] = pages(static_cast<int64_t>(old[k]) + fresh[k]) - pages(old[k]);
            st += fresh[k];
            sp += need[k];
        }
        int64_t it = st, ip = sp;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t yt = __shfl_up_sync(0xffffffffu, it, o), yp = __shfl_up_sync(0xffffffffu, ip, o);
            if (lane >= o) {
                it += yt;
                ip += yp;
            }
        }
        if (lane == 31) {
            s_wt[warp] = it;
            s_wp[warp] = ip;
        }
        __syncthreads();
        int64_t at = tok0 + it - st, ap = page0 + ip - sp, all_t = 0, all_p = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            at += w < warp ? s_wt[w] : 0;
            ap += w < warp ? s_wp[w] : 0;
            all_t += s_wt[w];
            all_p += s_wp[w];
        }
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int j = tid * kPlanPer + k, i = i0 + j;
            s_tok[j] = at;
            s_page[j] = ap;
            s_old[j] = old[k];
            if (i >= r0 && i < r1) {
                a.cu_seqlens_q[i] = static_cast<int32_t>(min(at, static_cast<int64_t>(0x7fffffff)));
                a.seqlens_out[i] = static_cast<int32_t>(min(static_cast<int64_t>(old[k]) + fresh[k], cap));
            }
            at += fresh[k];
            ap += need[k];
        }
        if (tid == kPlanThreads - 1) {
            s_tok[kPlanChunk] = at;
            s_page[kPlanChunk] = ap;
        }
        __syncthreads();
        const int here = min(kPlanChunk, a.b - i0);
        // table rows of this block's requests: a warp per request
        for (int i = max(r0, i0) + warp; i < min(r1, i0 + here); i += kPlanThreads / 32) {
            const int j = i - i0, have = pages(s_old[j]);
            const int n = static_cast<int>(s_page[j + 1] - s_page[j]);
            for (int k = lane; k < n; k += 32)
                a.block_table[static_cast<int64_t>(i) * a.max_pages + have + k] = taken(s_page[j] + k);
        }
        // slots of this block's tokens: the token's request by bisection
        for (int64_t t = max(t0, s_tok[0]) + tid; t < min(t1, s_tok[here]); t += kPlanThreads) {
            int lo = 0, hi = here - 1;  // the last request that begins at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_tok[mid] <= t)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int64_t pos = s_old[lo] + (t - s_tok[lo]);
            int64_t slot = -1;
            if (pos < cap) {
                const int p = static_cast<int>(pos / a.page_size), have = pages(s_old[lo]);
                const int page =
                    p < have ? __ldg(a.block_table + static_cast<int64_t>(i0 + lo) * a.max_pages + p)
                             : taken(s_page[lo] + p - have);
                if (page >= 0) slot = static_cast<int64_t>(page) * a.page_size + pos % a.page_size;
            }
            a.slot_map[t] = slot;
        }
        tok0 += all_t;
        page0 += all_p;
        __syncthreads();  // before the next chunk writes the shared arrays
    }
    // entries behind the last token
    for (int64_t t = max(t0, tok0) + tid; t < t1; t += kPlanThreads) a.slot_map[t] = -1;
    if (blockIdx.x == 0 && tid == 0) {
        a.cu_seqlens_q[a.b] = static_cast<int32_t>(min(tok0, static_cast<int64_t>(0x7fffffff)));
        a.free_left[0] = static_cast<int32_t>(max(free_n - page0, static_cast<int64_t>(-0x7fffffff)));
    }
}

// ------------------------------------------------------------ write
// A copy: 2 rows of h_kv * d values per token, read and written once, bound by
// HBM. Rows are runs of 16-byte words; a thread moves one word of K and the
// same one of V, and takes kWriteIter tokens' words at once so that enough
// loads are in flight (16391 tokens of 8 heads, d128: 24.5 us, 5.5 TB/s, 81% of
// the copy bandwidth; 20.8 us where calls repeat on the same tensors).
constexpr int kWriteThreads = 256;
constexpr int kWriteIter = 4;

__global__ void __launch_bounds__(kWriteThreads) write_kernel(const WriteArgs a) {
    const int64_t n = a.tokens * a.words;  // 16-byte words of K (and of V)
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kWriteThreads * kWriteIter + threadIdx.x;
    // word `base` is word c of token t; the thread's next ones lie a block apart
    int64_t t;
    int c;
    if (n <= 0xffffffffLL) {
        t = static_cast<uint32_t>(base) / static_cast<uint32_t>(a.words);
        c = static_cast<int>(static_cast<uint32_t>(base) - static_cast<uint32_t>(t) * static_cast<uint32_t>(a.words));
    } else {
        t = base / a.words;
        c = static_cast<int>(base - t * a.words);
    }
    uint4 kw[kWriteIter], vw[kWriteIter];
    int64_t to[kWriteIter];
#pragma unroll
    for (int i = 0; i < kWriteIter; ++i) {
        to[i] = -1;
        if (t < a.tokens) {
            const int64_t slot = __ldg(a.slot_map + t);
            if (slot >= 0 && slot < a.slots) to[i] = slot * a.words + c;
            kw[i] = __ldcs(a.k + t * a.k_stride + c);
            vw[i] = __ldcs(a.v + t * a.v_stride + c);
        }
        t += a.step_tokens;
        c += a.step_words;
        if (c >= a.words) {
            c -= a.words;
            ++t;
        }
    }
#pragma unroll
    for (int i = 0; i < kWriteIter; ++i)
        if (to[i] >= 0) {
            a.k_pages[to[i]] = kw[i];
            a.v_pages[to[i]] = vw[i];
        }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs &a, int num_sms, cudaStream_t stream) {
    // a block for each 1024 tokens or 64 requests
    int64_t blocks = (a.max_tokens + 1023) / 1024;
    if (blocks < (a.b + 63) / 64) blocks = (a.b + 63) / 64;
    if (blocks > 2 * num_sms) blocks = 2 * num_sms;
    if (blocks < 1) blocks = 1;
    plan_kernel<<<static_cast<unsigned>(blocks), kPlanThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_write(const WriteArgs &args, cudaStream_t stream) {
    WriteArgs a = args;
    a.step_tokens = kWriteThreads / a.words;
    a.step_words = kWriteThreads % a.words;
    const int64_t per = kWriteThreads * kWriteIter;
    const int64_t blocks = (a.tokens * a.words + per - 1) / per;
    write_kernel<<<static_cast<unsigned>(blocks), kWriteThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace exattn
