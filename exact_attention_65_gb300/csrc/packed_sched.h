// How the packed kernels deal out their work: host and device share this
// arithmetic, so that the plan can be checked without a GPU.
//
// The work of a call is a line: sequences one behind the other, within a
// sequence its K/V heads, within a head its units (row tiles of the forward
// and dQ kernels, key tiles of the dK/dV kernel), within a unit its steps
// (the streamed tiles). A unit of n steps takes a fixed cost plus the keys
// (or query tokens) it streams; under the causal mask that is linear in the
// unit's index, so that the line's length and any place on it have closed
// forms, and no list of tiles is made or sorted. CTA c of G takes the part
// [W c / G, W (c + 1) / G) of a line of length W, cut at step boundaries: a
// long sequence is spread over many CTAs and short ones share a CTA, whatever
// the mix of lengths. The CTAs that share a unit join their partial results
// (no CTA waits for another: the last one to finish joins them).
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define EXATTN_HD __host__ __device__ __forceinline__
#else
#define EXATTN_HD inline
#endif

namespace exattn {

EXATTN_HD int64_t smax64(int64_t a, int64_t b) { return a > b ? a : b; }
EXATTN_HD int64_t smin64(int64_t a, int64_t b) { return a < b ? a : b; }
EXATTN_HD int smax(int a, int b) { return a > b ? a : b; }
EXATTN_HD int smin(int a, int b) { return a < b ? a : b; }

// What the line is made of; the same for every CTA of a launch.
struct LineShape {
    int heads;       // K/V heads
    int unit_len;    // tokens (or keys) of one unit
    int step_len;    // keys (or tokens) of one step
    int causal;
    int by_key;      // 0: units over query tokens, steps over keys; 1: the other way round
    int unit_cost;   // a unit's fixed cost, in keys (or tokens) streamed
    int min_steps;   // a unit is not cut this close to its ends
    int64_t min_part;  // the least a CTA takes of the line before units are cut
};

// Units of one head of a sequence of sq query rows and sk keys.
EXATTN_HD int line_units(const LineShape &s, int sq, int sk) {
    const int n = s.by_key ? sk : sq;
    return n <= 0 ? 0 : (n - 1) / s.unit_len + 1;
}

// The steps [first, first + count) of unit u. With the causal mask query
// token i sees key j only if j <= i + sk - sq.
EXATTN_HD void line_steps(const LineShape &s, int sq, int sk, int u, int *first, int *count) {
    *first = 0;
    if (!s.by_key) {
        const int all = sk <= 0 ? 0 : (sk - 1) / s.step_len + 1;
        *count = all;
        if (s.causal) {
            const int64_t last = smin64(static_cast<int64_t>(u + 1) * s.unit_len, sq) - 1;
            const int64_t kmax = last + sk - sq;
            *count = kmax < 0 ? 0 : static_cast<int>(smin64(all, kmax / s.step_len + 1));
        }
    } else {
        const int all = sq <= 0 ? 0 : (sq - 1) / s.step_len + 1;
        *count = all;
        if (s.causal) {
            const int64_t q0 = static_cast<int64_t>(u) * s.unit_len - (static_cast<int64_t>(sk) - sq);
            *first = q0 <= 0 ? 0 : static_cast<int>(smin64(q0 / s.step_len, all));
            *count = all - *first;
        }
    }
}

// Cost of the units before unit n of one head (n up to line_units()).
EXATTN_HD int64_t line_before(const LineShape &s, int sq, int sk, int n) {
    const int64_t off = static_cast<int64_t>(sk) - sq, len = s.unit_len;
    int64_t sum = static_cast<int64_t>(n) * s.unit_cost;
    if (!s.causal) return sum + static_cast<int64_t>(n) * (s.by_key ? sq : sk);
    if (!s.by_key) {
        // unit u streams max(0, off + (u + 1) len) keys
        const int64_t u0 = off >= 0 ? 0 : smin64(-off / len, n);
        sum += (n - u0) * off + len * ((static_cast<int64_t>(n) * (n + 1) - u0 * (u0 + 1)) / 2);
    } else {
        // unit u streams sq tokens while u len <= off, then sk - u len
        const int64_t u0 = off < 0 ? 0 : smin64(off / len + 1, n);
        sum += u0 * sq + (n - u0) * sk - len * ((static_cast<int64_t>(n) * (n - 1) - u0 * (u0 - 1)) / 2);
    }
    return sum;
}

// The longest unit of a head: the last one over query tokens, the first one
// over keys.
EXATTN_HD int64_t line_longest(const LineShape &s, int sq, int sk) {
    const int n = line_units(s, sq, sk);
    if (n == 0) return 0;
    const int u = s.by_key ? 0 : n - 1;
    return line_before(s, sq, sk, u + 1) - line_before(s, sq, sk, u);
}

// Sums over the sequences, and what follows from them.
struct LineSum {
    int64_t cost;     // with the heads
    int64_t units;    // with the heads
    int64_t longest;  // of one unit
};

EXATTN_HD void line_add(LineSum *t, const LineShape &s, int sq, int sk) {
    const int n = line_units(s, sq, sk);
    t->cost += static_cast<int64_t>(s.heads) * line_before(s, sq, sk, n);
    t->units += static_cast<int64_t>(s.heads) * n;
    t->longest = smax64(t->longest, line_longest(s, sq, sk));
}

// How the line is dealt: `parts` CTAs take a share each. Where every unit is
// short and there is a CTA for each, each takes one whole unit (`whole`:
// every unit then counts 1).
struct LineDeal {
    int64_t length;
    int parts;
    int whole;
};

EXATTN_HD LineDeal line_deal(const LineShape &s, const LineSum &t, int ctas) {
    LineDeal d;
    d.whole = t.units <= ctas && t.longest <= 2 * s.min_part;
    d.length = d.whole ? t.units : t.cost;
    d.parts = static_cast<int>(d.whole ? t.units : smin64(ctas, smax64(1, t.cost / s.min_part)));
    return d;
}

EXATTN_HD int64_t deal_before(const LineShape &s, const LineDeal &d, int sq, int sk, int n) {
    return d.whole ? n : line_before(s, sq, sk, n);
}

// Where part c begins on the line.
EXATTN_HD int64_t part_begin(const LineDeal &d, int c) {
    // length < 2^62 / parts: tokens times keys of one device's memory
    return d.parts > 0 ? d.length * c / d.parts : 0;
}

// A place x (counted from the unit's beginning) as a step of a unit of n
// steps. Cuts near the unit's ends move to the ends.
EXATTN_HD int place_step(const LineShape &s, const LineDeal &d, int64_t x, int n) {
    if (d.whole || n == 0) return 0;
    const int64_t y = x - s.unit_cost;
    int64_t t = y <= 0 ? 0 : (y + s.step_len / 2) / s.step_len;
    if (n < 2 * s.min_steps) return 2 * t < n ? 0 : n;
    if (t < s.min_steps) return 0;
    return n - t < s.min_steps ? n : static_cast<int>(t);
}

// A place on the line: step `step` of `unit` of `head` of sequence `seq`.
// step == count of the unit means its end.
struct Place {
    int seq, head, unit, step;
};

// The place `rem` into the sequence's part of the line (0 <= rem < its cost).
EXATTN_HD Place place_in_seq(const LineShape &s, const LineDeal &d, int seq, int sq, int sk, int64_t rem) {
    Place p;
    p.seq = seq;
    const int n = line_units(s, sq, sk);
    const int64_t per_head = deal_before(s, d, sq, sk, n);
    p.head = static_cast<int>(rem / per_head);
    rem -= p.head * per_head;
    int lo = 0, hi = n - 1;  // the last unit that begins at or before rem
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (deal_before(s, d, sq, sk, mid) <= rem)
            lo = mid;
        else
            hi = mid - 1;
    }
    p.unit = lo;
    int first, count;
    line_steps(s, sq, sk, lo, &first, &count);
    p.step = place_step(s, d, rem - deal_before(s, d, sq, sk, lo), count);
    return p;
}

// The parts that share a unit whose place on the line is [x0, x1) and which
// has n steps: the first one, and how many. The unit is known to be cut.
EXATTN_HD void unit_sharers(const LineShape &s, const LineDeal &d, int64_t x0, int64_t x1, int n, int *first,
                            int *count) {
    // part c cuts the unit if it begins inside it, away from its ends
    int a = static_cast<int>(x0 * d.parts / d.length);
    while (part_begin(d, a) < x0) ++a;
    while (a < d.parts && place_step(s, d, part_begin(d, a) - x0, n) == 0) ++a;
    int z = static_cast<int>(smin64((x1 * d.parts + d.length - 1) / d.length, d.parts - 1));
    while (z > a && (part_begin(d, z) >= x1 || place_step(s, d, part_begin(d, z) - x0, n) >= n)) --z;
    *first = a - 1;
    *count = z - a + 2;
}

// A sequence of the line: its query rows and keys.
struct SeqLen {
    int sq, sk;
};

// A unit, or a range of a cut unit's steps.
struct UnitRange {
    int seq, head, unit;
    int step0, nstep;  // steps [step0, step0 + nstep), counted from the sequence's first key (token)
    int slot;          // -1: the whole unit; 0: a range that does not begin the unit; 1: one that does
    int first_part;    // the parts that share the unit
    int nparts;
};

// Part `part`'s units in order, from place p (before it lie seq_x0 of the
// line up to p's sequence) to place e (seq == b: the line's end). len(i): a
// sequence's lengths; emit(range): false ends the walk.
template <class Len, class Emit>
EXATTN_HD void walk_part(const LineShape &s, const LineDeal &d, int b, int part, Place p, const Place &e,
                         int64_t seq_x0, Len len, Emit emit) {
    if (p.seq >= b) return;
    SeqLen x = len(p.seq);
    int units = line_units(s, x.sq, x.sk);
    for (;;) {
        const bool last = p.seq == e.seq && p.head == e.head && p.unit == e.unit;
        if (last && p.step >= e.step) return;
        int first, count;
        line_steps(s, x.sq, x.sk, p.unit, &first, &count);
        const int stop = last ? e.step : count;
        if (p.step < count || count == 0) {
            UnitRange r;
            r.seq = p.seq;
            r.head = p.head;
            r.unit = p.unit;
            r.step0 = first + p.step;
            r.nstep = stop - p.step;
            r.slot = -1;
            r.first_part = part;
            r.nparts = 1;
            if (p.step > 0 || stop < count) {
                r.slot = p.step > 0 ? 0 : 1;
                const int64_t u0 = line_before(s, x.sq, x.sk, p.unit);
                const int64_t x0 = seq_x0 + p.head * line_before(s, x.sq, x.sk, units) + u0;
                const int64_t x1 = x0 + line_before(s, x.sq, x.sk, p.unit + 1) - u0;
                unit_sharers(s, d, x0, x1, count, &r.first_part, &r.nparts);
            }
            if (!emit(r)) return;
        }
        if (last) return;
        p.step = 0;
        if (++p.unit < units) continue;
        p.unit = 0;
        if (++p.head < s.heads) continue;
        p.head = 0;
        do {
            seq_x0 += s.heads * deal_before(s, d, x.sq, x.sk, units);
            if (++p.seq >= b) return;
            x = len(p.seq);
            units = line_units(s, x.sq, x.sk);
        } while (units == 0);
    }
}

}  // namespace exattn
