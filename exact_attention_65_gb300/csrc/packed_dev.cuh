// Device side of the packed kernels' work line (packed_sched.h): the length
// of the line by the whole block, the CTA's part of it by one warp, and the
// messages through which that warp tells the block's other warps what comes
// next.
#pragma once

#include "packed.h"
#include "packed_sched.h"
#include "ptx.cuh"

namespace exattn {

// mbar_wait() with one copy of the poll in it: these kernels have some thirty
// waits and have to stay small (packed_sched.h). Same bounds, same report.
__device__ __forceinline__ bool await(uint32_t bar, uint32_t parity, const WaitGuard &g, uint32_t site) {
    uint32_t t0 = 0;
#pragma unroll 1
    for (uint32_t polls = 0; !mbar_try_wait(bar, parity);) {
        if ((++polls & 15u) != 0u) continue;
        // microseconds, wrapping after an hour
        const uint32_t now = static_cast<uint32_t>(global_timer_ns() >> 10) | 1u;
        if (t0 == 0) t0 = now;
        if (*g.abort != 0u) return false;
        if (now - t0 > static_cast<uint32_t>(kWaitTimeoutNs >> 10) || polls >= kWaitMaxPolls) {
            *g.abort = 1u;
            atomicCAS(g.status, 0u, (g.kernel << 8) | site);
            return false;
        }
    }
    return true;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// A value that all lanes hold, known as such to the compiler: what an MMA's
// descriptors are made of then stays in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// One sequence of a packed batch: its first query row and first key row (0 in
// a paged cache) and its lengths. Whatever the arrays on the device hold, the
// rows stay inside the tensors.
struct SeqInfo {
    int q0, sq, k0, sk;
};

__device__ __forceinline__ SeqInfo seq_info(const SeqArrays &s, int i, bool *ordered = nullptr) {
    SeqInfo x;
    bool in_order = clamp_rows(__ldg(s.cu_q + i), __ldg(s.cu_q + i + 1), s.total_q, &x.q0, &x.sq);
    if (s.cu_k != nullptr) {
        in_order &= clamp_rows(__ldg(s.cu_k + i), __ldg(s.cu_k + i + 1), s.max_k, &x.k0, &x.sk);
    } else {
        x.k0 = 0;
        x.sk = min(max(__ldg(s.seqlens + i), 0), s.max_k);
    }
    if (ordered != nullptr) *ordered = in_order;
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
    int first_part;    // of a cut unit: the first CTA that shares it, and how many
    int nparts;        //   do; there once the slot's `shared` barrier has been passed
    int pad[3];
};
static_assert(sizeof(UnitMsg) == 64, "four 16-byte words");

constexpr int kMsgSlots = 4;

// What each kernel knows of its line: half of the arithmetic's code.
template <int BY_KEY>
__device__ __forceinline__ void known_shape(LineShape *s) {
    s->by_key = BY_KEY;
    if (BY_KEY) {
        s->unit_len = 128;
        s->unit_mul = 1u << 31;
        s->unit_div = 38;
    } else {
        s->step_len = 128;
        s->step_mul = 1u << 31;
        s->step_div = 38;
    }
}

// The line's sums: every thread of the block adds some sequences, warp sums go
// to `sums` (one LineSum per warp) for line_total() after a barrier.
template <int BY_KEY>
__device__ __forceinline__ void line_sum_warps(const SeqArrays &s, LineShape shape, LineSum *sums) {
    known_shape<BY_KEY>(&shape);
    LineSum t{0, 0, 0};
#pragma unroll 1
    for (int i = threadIdx.x; i < s.b; i += blockDim.x) {
        bool ordered;
        const SeqInfo x = seq_info(s, i, &ordered);
        line_add(&t, shape, x.sq, x.sk, ordered);
    }
    t.cost = __reduce_add_sync(0xffffffffu, t.cost);
    t.units = __reduce_add_sync(0xffffffffu, t.units);
    t.longest = __reduce_max_sync(0xffffffffu, t.longest);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = t;
}

// The block's total, by one warp.
__device__ __forceinline__ LineSum line_total(const LineSum *sums, int warps) {
    const int lane = threadIdx.x & 31;
    LineSum t{0, 0, 0};
    if (lane < warps) t = sums[lane];
    t.cost = __reduce_add_sync(0xffffffffu, t.cost);
    t.units = __reduce_add_sync(0xffffffffu, t.units);
    t.longest = __reduce_max_sync(0xffffffffu, t.longest);
    return t;
}

// Run by one warp: finds part `part` of the line dealt to `ctas` CTAs and
// posts its units. total(): the line's sums where there are more than 32
// sequences. `full` / `empty` / `shared`: kMsgSlots barriers each; `site`:
// where a timeout of the wait for a free message slot is recorded.
template <int BY_KEY, class Total>
__device__ __forceinline__ void post_units(const SeqArrays &seqs, LineShape shape, Total total, UnitMsg *msgs,
                                           uint32_t full, uint32_t empty, uint32_t shared, const WaitGuard &g,
                                           uint32_t site, int part, int ctas) {
    const int lane = threadIdx.x & 31;
    known_shape<BY_KEY>(&shape);
    SeqInfo x{0, 0, 0, 0};
    bool ordered = true;
    if (lane < seqs.b) x = seq_info(seqs, lane, &ordered);
    int n = line_units(shape, x.sq, x.sk);         // units of a head
    int per = line_before(shape, x.sq, x.sk, n);   // and their cost
    LineSum sum;
    if (seqs.b <= 32) {
        sum.cost = __reduce_add_sync(0xffffffffu, shape.heads * per);
        sum.units = __reduce_add_sync(0xffffffffu, shape.heads * n);
        const int longest = !ordered ? kOutOfOrder
                            : n == 0 ? 0
                            : BY_KEY ? line_before(shape, x.sq, x.sk, 1)
                                     : per - line_before(shape, x.sq, x.sk, n - 1);
        sum.longest = __reduce_max_sync(0xffffffffu, longest);
    } else {
        sum = total();
    }
    const LineDeal deal = line_deal(&shape, sum, ctas);
    if (shape.weight == 0) per = n;

    // The part's begin (lanes 0-15 look for it) and end (lanes 16-31): 32
    // sequences at a time, by a prefix sum
    Place p{seqs.b, 0, 0, 0}, e = p;
    SeqLen p_len{0, 0};
    int p_units = 0, p_x0 = 0;
    SeqInfo cur{0, 0, 0, 0};
    if (part < deal.parts) {
        const int want0 = part_begin(deal, part), want1 = part_begin(deal, part + 1);
        int before = 0;
#pragma unroll 1
        for (int i0 = 0;;) {
            const int cost = shape.heads * per;
            int upto = cost;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const int x0 = before + upto - cost;
            const uint32_t b0 = __ballot_sync(0xffffffffu, want0 >= x0 && want0 < x0 + cost);
            const uint32_t b1 = __ballot_sync(0xffffffffu, want1 >= x0 && want1 < x0 + cost);
            if ((b0 | b1) != 0) {
                const int half = lane & 16, sub = lane & 15;
                const uint32_t mine = half ? b1 : b0;
                const int src = mine ? __ffs(mine) - 1 : 0;  // (a half that found nothing works for nothing)
                const int sq = __shfl_sync(0xffffffffu, x.sq, src), sk = __shfl_sync(0xffffffffu, x.sk, src);
                const int units = __shfl_sync(0xffffffffu, n, src);
                const int per_head = max(__shfl_sync(0xffffffffu, per, src), 1);
                const int seq_x0 = __shfl_sync(0xffffffffu, x0, src);
                int rem = max((half ? want1 : want0) - seq_x0, 0);
                Place q;
                q.seq = i0 + src;
                q.head = static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(per_head));
                rem -= q.head * per_head;
                // the last unit that begins at or before rem, one of [q.unit, q.unit + left)
                q.unit = 0;
                int left = units;
#pragma unroll 1
                do {
                    const int stride = (left + 15) >> 4;
                    const bool in = sub * stride < left && line_before(shape, sq, sk, q.unit + sub * stride) <= rem;
                    const uint32_t yes = (__ballot_sync(0xffffffffu, in) >> half) & 0xffffu;
                    const int k = yes ? 31 - __clz(yes) : 0;
                    q.unit += k * stride;
                    left = min(stride, left - k * stride);
                } while (__any_sync(0xffffffffu, left > 1));
                // even lanes its beginning, odd ones its end
                const int f = line_before(shape, sq, sk, q.unit + (lane & 1));
                const int u0 = __shfl_sync(0xffffffffu, f, half), u1 = __shfl_sync(0xffffffffu, f, half + 1);
                int first, count;
                line_steps(shape, sq, sk, q.unit, &first, &count);
                q.step = place_step(shape, rem - u0, u1 - u0, count);
                if (b0 != 0) {
                    p.seq = __shfl_sync(0xffffffffu, q.seq, 0);
                    p.head = __shfl_sync(0xffffffffu, q.head, 0);
                    p.unit = __shfl_sync(0xffffffffu, q.unit, 0);
                    p.step = __shfl_sync(0xffffffffu, q.step, 0);
                    p_len.sq = __shfl_sync(0xffffffffu, sq, 0);
                    p_len.sk = __shfl_sync(0xffffffffu, sk, 0);
                    p_units = __shfl_sync(0xffffffffu, units, 0);
                    p_x0 = __shfl_sync(0xffffffffu, seq_x0, 0);
                    cur.q0 = __shfl_sync(0xffffffffu, x.q0, p.seq - i0);
                    cur.k0 = __shfl_sync(0xffffffffu, x.k0, p.seq - i0);
                    cur.sq = p_len.sq;
                    cur.sk = p_len.sk;
                }
                if (b1 != 0) {
                    e.seq = __shfl_sync(0xffffffffu, q.seq, 16);
                    e.head = __shfl_sync(0xffffffffu, q.head, 16);
                    e.unit = __shfl_sync(0xffffffffu, q.unit, 16);
                    e.step = __shfl_sync(0xffffffffu, q.step, 16);
                }
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
            i0 += 32;
            if (i0 >= seqs.b || before > want1) break;
            x = SeqInfo{0, 0, 0, 0};
            if (i0 + lane < seqs.b) x = seq_info(seqs, i0 + lane);
            n = line_units(shape, x.sq, x.sk);
            per = line_before(shape, x.sq, x.sk, n);
        }
    }

    int posted = 0;
    auto post = [&](const UnitMsg &m) {
        const int s = posted % kMsgSlots;
        const bool ok = await(empty + 8u * s, ((posted / kMsgSlots) & 1) ^ 1, g, site);
        if (!__all_sync(0xffffffffu, ok)) return false;
        if (lane == 0) {
            const int4 *src = reinterpret_cast<const int4 *>(&m);
            int4 *dst = reinterpret_cast<int4 *>(msgs + s);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = src[i];
            mbar_arrive(full + 8u * s);
        }
        ++posted;
        return true;
    };
    bool ok = true;
    walk_part(
        shape, seqs.b, p, e, p_len, p_units, p_x0,
        [&](int i) {
            cur = seq_info(seqs, i);
            return SeqLen{cur.sq, cur.sk};
        },
        [&](const UnitRange &r) {
            UnitMsg m;
            m.live = 1;
            m.head = r.head;
            m.tok0 = r.unit * shape.unit_len;
            m.seq = r.seq;
            m.q0 = cur.q0;
            m.sq = cur.sq;
            m.k0 = cur.k0;
            m.sk = cur.sk;
            m.step0 = r.step0;
            m.nstep = r.nstep;
            m.slot = r.slot;
            m.first_part = part;
            m.nparts = 1;
            if (!(ok = post(m))) return false;
            if (r.slot >= 0) {
                // who shares a cut unit is needed at its end only: worked out
                // (32 parts at a time) once the unit is on its way
                int cuts = 0, first = 0;
#pragma unroll 1
                for (int c0 = 0; c0 < deal.parts; c0 += 32) {
                    const uint32_t in = __ballot_sync(
                        0xffffffffu, c0 + lane < deal.parts &&
                                         part_cuts(shape, deal, c0 + lane, r.x0, r.cost, r.steps));
                    if (in != 0 && cuts == 0) first = c0 + __ffs(in) - 2;
                    cuts += __popc(in);
                }
                if (lane == 0) {
                    volatile UnitMsg *w = msgs + (posted - 1) % kMsgSlots;
                    w->first_part = first;
                    w->nparts = cuts + 1;
                    mbar_arrive(shared + 8u * ((posted - 1) % kMsgSlots));
                }
            } else if (lane == 0) {
                mbar_arrive(shared + 8u * ((posted - 1) % kMsgSlots));
            }
            return true;
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
    bool ok = await(full + 8u * s, (n / kMsgSlots) & 1, g, site);
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
    const bool ok = await(bar, phase & 1, g, 19);
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
    const bool ok = await(full + 8u * s, (n / kMsgSlots) & 1, g, site);
    if (!__all_sync(0xffffffffu, ok)) return nullptr;
    const volatile UnitMsg *m = msgs + s;
    return m->live ? m : nullptr;
}

__device__ __forceinline__ void free_unit(int n, uint32_t empty) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * (n % kMsgSlots));
}

}  // namespace exattn
