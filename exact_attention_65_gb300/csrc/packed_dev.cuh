// Device side of the packed kernels' work line (packed_sched.h): the length
// of the line by the whole block, the CTA's part of it by one warp, and the
// messages through which that warp tells the block's other warps what comes
// next.
#pragma once

#include "internal.h"
#include "packed_sched.h"
#include "ptx.cuh"

namespace exattn {

// One sequence of a packed batch: its first query row and first key row (0 in
// a paged cache) and its lengths. Whatever the arrays on the device hold, the
// rows stay inside the tensors.
struct SeqInfo {
    int q0, sq, k0, sk;
};

__device__ __forceinline__ SeqInfo seq_info(const SeqArrays &s, int i) {
    SeqInfo x;
    x.q0 = min(max(__ldg(s.cu_q + i), 0), s.total_q);
    x.sq = min(max(__ldg(s.cu_q + i + 1), x.q0), s.total_q) - x.q0;
    if (s.cu_k != nullptr) {
        x.k0 = min(max(__ldg(s.cu_k + i), 0), s.max_k);
        x.sk = min(max(__ldg(s.cu_k + i + 1), x.k0), s.max_k) - x.k0;
    } else {
        x.k0 = 0;
        x.sk = min(max(__ldg(s.seqlens + i), 0), s.max_k);
    }
    return x;
}

// A unit, or a range of a cut unit's steps, as the block's warps are told it.
struct alignas(16) UnitMsg {
    int live;   // 0: no more units
    int head;   // K/V head
    int tok0;   // the unit's first query token (by_key: key) within its sequence
    int seq;
    int q0, sq, k0, sk;
    int step0, nstep;  // steps [step0, step0 + nstep)
    int slot;          // -1: the whole unit; else the CTA's slot for this range's partial result
    int first_part;    // of a cut unit: the first CTA that shares it, and how many do
    int nparts;
    int pad[3];
};
static_assert(sizeof(UnitMsg) == 64, "four 16-byte words");

constexpr int kMsgSlots = 4;

// The line's sums: every thread of the block adds some sequences, warp sums
// go to `sums` (one LineSum per warp) for line_total() after a barrier.
__device__ __forceinline__ void line_sum_warps(const SeqArrays &s, const LineShape &shape, LineSum *sums) {
    LineSum t{0, 0, 0};
    for (int i = threadIdx.x; i < s.b; i += blockDim.x) {
        const SeqInfo x = seq_info(s, i);
        line_add(&t, shape, x.sq, x.sk);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t.cost += __shfl_xor_sync(0xffffffffu, t.cost, o);
        t.units += __shfl_xor_sync(0xffffffffu, t.units, o);
        t.longest = max(t.longest, __shfl_xor_sync(0xffffffffu, t.longest, o));
    }
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
}

__device__ __forceinline__ LineSum line_total(const LineSum *sums, int warps) {
    LineSum t{0, 0, 0};
    for (int i = 0; i < warps; ++i) {
        t.cost += sums[i].cost;
        t.units += sums[i].units;
        t.longest = max(t.longest, sums[i].longest);
    }
    return t;
}

// Run by one warp: finds part `part` of the line dealt to `ctas` CTAs and
// posts its units.
// `full` / `empty`: kMsgSlots barriers each; `site`: where a timeout of the
// wait for a free message slot is recorded.
__device__ __forceinline__ void post_units(const SeqArrays &seqs, const LineShape &shape, const LineSum &total,
                                           UnitMsg *msgs, uint32_t full, uint32_t empty, const WaitGuard &g,
                                           uint32_t site, int part, int ctas) {
    const int lane = threadIdx.x & 31;
    const LineDeal deal = line_deal(shape, total, ctas);
    Place p{seqs.b, 0, 0, 0}, e = p;
    int64_t seq_x0 = 0;  // the line before sequence p.seq
    if (part < deal.parts) {
        const int64_t want[2] = {part_begin(deal, part), part_begin(deal, part + 1)};
        bool got[2] = {false, false};
        int64_t before = 0;
        for (int i0 = 0; i0 < seqs.b && !(got[0] && got[1]); i0 += 32) {
            SeqInfo x{0, 0, 0, 0};
            if (i0 + lane < seqs.b) x = seq_info(seqs, i0 + lane);
            const int64_t cost =
                shape.heads * deal_before(shape, deal, x.sq, x.sk, line_units(shape, x.sq, x.sk));
            int64_t upto = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const int64_t x0 = before + upto - cost;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const bool here = want[w] >= x0 && want[w] < x0 + cost;
                const uint32_t who = __ballot_sync(0xffffffffu, here);
                if (who == 0) continue;
                const int src = __ffs(who) - 1;
                Place q{0, 0, 0, 0};
                if (here) q = place_in_seq(shape, deal, i0 + lane, x.sq, x.sk, want[w] - x0);
                q.seq = __shfl_sync(0xffffffffu, q.seq, src);
                q.head = __shfl_sync(0xffffffffu, q.head, src);
                q.unit = __shfl_sync(0xffffffffu, q.unit, src);
                q.step = __shfl_sync(0xffffffffu, q.step, src);
                got[w] = true;
                if (w == 0) {
                    p = q;
                    seq_x0 = __shfl_sync(0xffffffffu, x0, src);
                } else {
                    e = q;
                }
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if (lane != 0) return;

    int n = 0;  // messages posted
    auto post = [&](const UnitMsg &m) {
        const int s = n % kMsgSlots;
        if (!mbar_wait(empty + 8u * s, ((n / kMsgSlots) & 1) ^ 1, g, site)) return false;
        const int4 *src = reinterpret_cast<const int4 *>(&m);
        int4 *dst = reinterpret_cast<int4 *>(msgs + s);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = src[i];
        mbar_arrive(full + 8u * s);
        ++n;
        return true;
    };
    SeqInfo x{0, 0, 0, 0};
    bool ok = true;
    walk_part(
        shape, deal, seqs.b, part, p, e, seq_x0,
        [&](int i) {
            x = seq_info(seqs, i);
            return SeqLen{x.sq, x.sk};
        },
        [&](const UnitRange &r) {
            UnitMsg m;
            m.live = 1;
            m.head = r.head;
            m.tok0 = r.unit * shape.unit_len;
            m.seq = r.seq;
            m.q0 = x.q0;
            m.sq = x.sq;
            m.k0 = x.k0;
            m.sk = x.sk;
            m.step0 = r.step0;
            m.nstep = r.nstep;
            m.slot = r.slot;
            m.first_part = r.first_part;
            m.nparts = r.nparts;
            return ok = post(m);
        });
    if (!ok) return;
    UnitMsg m{};
    post(m);
}

// Takes message n: waits for it, copies it and frees its slot (one arrival
// per consumer: a lone thread, or a warp whose lanes all call this).
template <bool WARP>
__device__ __forceinline__ bool take_unit(UnitMsg *m, int n, const UnitMsg *msgs, uint32_t full, uint32_t empty,
                                          const WaitGuard &g, uint32_t site) {
    const int s = n % kMsgSlots;
    bool ok = mbar_wait(full + 8u * s, (n / kMsgSlots) & 1, g, site);
    if (WARP) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const int4 *src = reinterpret_cast<const int4 *>(msgs + s);
    int4 *dst = reinterpret_cast<int4 *>(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = src[i];
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * s);
    return m->live != 0;
}

// Warps meet (as many as the barrier counts): a bounded wait, as a warp that
// gave up elsewhere never comes.
__device__ __forceinline__ bool meet(uint32_t bar, int &phase, const WaitGuard &g) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    const bool ok = mbar_wait(bar, phase & 1, g, 19);
    ++phase;
    return __all_sync(0xffffffffu, ok);
}

// Counts an arrival of call number `call` (24 bits) and tells whether it is
// the last of n. The counter holds (call << 8 | arrivals): what a call that
// gave up left there counts as none; the last arrival clears it.
__device__ __forceinline__ bool arrive_last(uint32_t *counter, uint32_t call, int n) {
    uint32_t old = *reinterpret_cast<volatile uint32_t *>(counter), seen;
    do {
        seen = old;
        old = atomicCAS(counter, seen, ((seen >> 8) == call ? seen : call << 8) + 1);
    } while (old != seen);
    const bool last = ((seen >> 8) == call ? seen & 0xffu : 0u) + 1 == static_cast<uint32_t>(n);
    if (last) atomicExch(counter, 0u);
    return last;
}

// The two halves of take_unit() for warps that are short of registers: wait
// for message n and read its fields from shared memory as they are needed,
// then free its slot.
__device__ __forceinline__ const volatile UnitMsg *wait_unit(int n, const UnitMsg *msgs, uint32_t full,
                                                             const WaitGuard &g, uint32_t site) {
    const int s = n % kMsgSlots;
    const bool ok = mbar_wait(full + 8u * s, (n / kMsgSlots) & 1, g, site);
    if (!__all_sync(0xffffffffu, ok)) return nullptr;
    const volatile UnitMsg *m = msgs + s;
    return m->live ? m : nullptr;
}

__device__ __forceinline__ void free_unit(int n, uint32_t empty) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * (n % kMsgSlots));
}

}  // namespace exattn
