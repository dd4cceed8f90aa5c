// How the packed kernels deal out their work: host and device share this
// arithmetic, so that the plan can be checked without a GPU.
//
// The work of a call is a line: sequences one behind the other, within a
// sequence its K/V heads, within a head its units (row tiles of the forward
// and dQ kernels, key tiles of the dK/dV kernel), within a unit its steps
// (the streamed tiles). A unit costs a fixed amount plus what it streams;
// under the causal mask that is linear in the unit's index, so that the
// line's length and any place on it have closed forms, and no list of tiles
// is made or sorted. CTA c of G takes the part [W c / G, W (c + 1) / G) of a
// line of length W, cut at step boundaries: a long sequence is spread over
// many CTAs and short ones share a CTA, whatever the mix of lengths. The CTAs
// that share a unit join their partial results (no CTA waits for another: the
// last one to finish joins them).
//
// All of this runs on every CTA before its first load, from a cold
// instruction cache, so it is kept small: 32-bit sums, few divisions, loops
// that stay loops. (An earlier form, with 64-bit divisions inlined, was 85 KB of
// code and took 7 us of a 14 us call; the softmax loop, too, was slowed down.)
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define EXATTN_HD __host__ __device__ __forceinline__
#else
#define EXATTN_HD inline
#endif

namespace exattn {

EXATTN_HD int smax(int a, int b) { return a > b ? a : b; }
EXATTN_HD int smin(int a, int b) { return a < b ? a : b; }

// What the line is made of; the same for every CTA of a launch. Costs are in
// steps of 128 rows (of keys, or of query heads times tokens), or 2^k of them
// where a call is so large that its sum would not fit 31 bits.
struct LineShape {
    int heads;      // K/V heads
    int unit_len;   // tokens (or keys) of one unit
    int step_len;   // keys (or tokens) of one step
    int causal;
    int by_key;     // 0: units over query tokens, steps over keys; 1: the other way round
    int weight;     // 128-row steps count weight / 2^shift of the keys (tokens) streamed;
    int shift;      //   weight 0: every unit counts the same
    int unit_cost;  // a unit's fixed cost
    int min_steps;  // a unit is not cut this close to its ends
    int min_part;   // the least a CTA takes of the line before units are cut
    uint32_t unit_mul, step_mul;  // x / len = x * mul >> shift for x < 2^31
    int unit_div, step_div;       //   (the shifts)
};

// A unit's fixed cost, in steps.
constexpr int kUnitSteps = 2;

// mul and shift of a division by len (1 .. 256): with 2^k >= len, mul =
// ceil(2^(31 + k) / len) fits 32 bits, and x * mul >> (31 + k) is exact for x <
// 2^31, as mul errs by less than 1 and x / 2^(31 + k) < 1 / len.
inline void fast_division(int len, uint32_t *mul, int *shift) {
    int k = 0;
    while ((1 << k) < len) ++k;
    *shift = 31 + k;
    *mul = static_cast<uint32_t>(((1ull << *shift) + len - 1) / len);
}
EXATTN_HD int divided(uint32_t x, uint32_t mul, int shift) {
    return static_cast<int>((static_cast<uint64_t>(x) * mul) >> shift);
}

// Units of one head of a sequence of sq query rows and sk keys.
EXATTN_HD int line_units(const LineShape &s, int sq, int sk) {
    return divided((s.by_key ? sk : sq) + s.unit_len - 1, s.unit_mul, s.unit_div);
}

// The steps [first, first + count) of unit u. With the causal mask query
// token i sees key j only if j <= i + sk - sq.
EXATTN_HD void line_steps(const LineShape &s, int sq, int sk, int u, int *first, int *count) {
    const int len = s.by_key ? sq : sk;  // what is streamed
    int lo = 0, hi = len;                // the part of it that the unit sees
    if (s.causal) {
        if (s.by_key)
            lo = smin(smax(u * s.unit_len - (sk - sq), 0), len);
        else
            hi = smax(smin((u + 1) * s.unit_len, sq) + sk - sq, 0);
    }
    const int a = divided(lo, s.step_mul, s.step_div);
    const int z = divided(hi + s.step_len - 1, s.step_mul, s.step_div);
    // (a unit over keys that no row sees starts at the end of the rows)
    *first = a;
    *count = lo < hi ? z - a : 0;
}

// Cost of the units before unit n of one head (n up to line_units()).
EXATTN_HD int line_before(const LineShape &s, int sq, int sk, int n) {
    const int off = sk - sq;
    int64_t sum;  // keys (tokens) streamed
    if (!s.causal) {
        sum = static_cast<int64_t>(n) * (s.by_key ? sq : sk);
    } else if (!s.by_key) {
        // unit u streams max(0, off + (u + 1) len) keys
        const int u0 = off < 0 ? smin(divided(-off, s.unit_mul, s.unit_div), n) : 0;
        const int64_t pairs = static_cast<int64_t>(n - u0) * (n + u0 + 1);  // / 2
        sum = static_cast<int64_t>(n - u0) * off + ((pairs * s.unit_len) >> 1);
    } else {
        // unit u streams sq tokens while 128 u <= off, then sk - 128 u
        const int u0 = off < 0 ? 0 : smin((off >> 7) + 1, n);
        const int64_t pairs = static_cast<int64_t>(n - u0) * (n + u0 - 1);
        sum = static_cast<int64_t>(u0) * sq + static_cast<int64_t>(n - u0) * sk - 64 * pairs;
    }
    return n * s.unit_cost + static_cast<int>((sum * s.weight) >> s.shift);
}

// Rows [a, z) of a sequence whose starts come from the device, moved into [0,
// total): whatever the array holds, they stay inside the tensor. False: the
// starts are out of order.
EXATTN_HD bool clamp_rows(int a, int z, int total, int *first, int *rows) {
    *first = smin(smax(a, 0), total);
    *rows = smin(smax(z, *first), total) - *first;
    return a <= z;
}

// Sums over the sequences. Starts in order give sequences that do not overlap,
// so that the sums stay below the bound that the host fitted the shape to;
// out of order, sequences could overlap and the 32-bit sums wrap, and with
// them every place on the line. kOutOfOrder as `longest` then says so (no unit
// is that long), and nothing is dealt out.
constexpr int kOutOfOrder = 0x7fffffff;
struct LineSum {
    int cost;     // with the heads
    int units;    // with the heads
    int longest;  // unit: the last one over query tokens, the first one over keys
};

EXATTN_HD void line_add(LineSum *t, const LineShape &s, int sq, int sk, bool ordered) {
    if (!ordered) t->longest = kOutOfOrder;
    const int n = line_units(s, sq, sk);
    if (n == 0) return;
    const int all = line_before(s, sq, sk, n);
    // (unsigned: out of order, they may wrap)
    t->cost = static_cast<int>(static_cast<uint32_t>(t->cost) + static_cast<uint32_t>(s.heads) * all);
    t->units = static_cast<int>(static_cast<uint32_t>(t->units) + static_cast<uint32_t>(s.heads) * n);
    t->longest = smax(t->longest, s.by_key ? line_before(s, sq, sk, 1) : all - line_before(s, sq, sk, n - 1));
}

// How the line is dealt: `parts` CTAs take a share each; part c begins at
// q c + r c / parts. Where every unit is short and there is a CTA for each,
// each takes one whole unit: every unit then counts 1 (weight 0).
struct LineDeal {
    int length, parts, q, r;
};

EXATTN_HD bool line_whole(const LineShape &s, const LineSum &t, int ctas) {
    return t.units <= ctas && t.longest <= 2 * s.min_part;
}

EXATTN_HD LineDeal line_deal(LineShape *s, const LineSum &t, int ctas) {
    LineDeal d{0, 0, 0, 0};
    if (t.longest == kOutOfOrder) return d;
    d.length = t.cost;
    d.parts = smin(ctas, smax(1, static_cast<int>(static_cast<uint32_t>(t.cost) / static_cast<uint32_t>(s->min_part))));
    if (line_whole(*s, t, ctas)) {
        s->weight = 0;
        s->unit_cost = 1;
        d.length = d.parts = t.units;
    }
    d.q = d.parts > 0 ? static_cast<int>(static_cast<uint32_t>(d.length) / static_cast<uint32_t>(d.parts)) : 0;
    d.r = d.length - d.q * d.parts;
    return d;
}

// (r c and parts are below 2^16 and 2^8: the quotient of floats, half a unit
// up, has the integer quotient's floor)
EXATTN_HD int part_begin(const LineDeal &d, int c) {
#if defined(__CUDA_ARCH__)
    return d.q * c + static_cast<int>(__fdividef(static_cast<float>(d.r * c) + 0.5f, static_cast<float>(d.parts)));
#else
    return d.q * c + d.r * c / d.parts;
#endif
}

// CTAs of the backward's key-tile kind, of ctas in all, from both kinds' lines.
// A key-tile step (four products) takes 1.15 times a query-tile step (three);
// with the units' fixed costs, short sequences have more of their time in query
// tiles (b1 s8192 h32/8 d128 causal: 1581 us with 80 of 152 for keys whatever
// the lengths, 1542 so). Each line counts 2^(shift - 7) steps as one, the two
// shifts can differ, and a unit's fixed cost then is a rounded one (1000
// sequences of 660 tokens, h32/8 d128 causal: 27.1 ms with the lines' costs
// compared as they are, 19.8 so). Where every unit can have a CTA to itself,
// each kind gets at least its units.
EXATTN_HD float line_steps_of(const LineShape &s, const LineSum &t) {
    return static_cast<float>(t.cost - t.units * s.unit_cost) * static_cast<float>(1u << (s.shift - 7)) +
           static_cast<float>(kUnitSteps) * static_cast<float>(t.units);
}
EXATTN_HD int key_ctas(const LineShape &q, const LineSum &qs, const LineShape &kv, const LineSum &kvs, int ctas) {
    const float wq = line_steps_of(q, qs), wkv = 1.15f * line_steps_of(kv, kvs), all = wq + wkv > 1.f ? wq + wkv : 1.f;
#if defined(__CUDA_ARCH__)
    int n = static_cast<int>(__fdividef(static_cast<float>(ctas) * wkv, all) + 0.5f);
#else
    int n = static_cast<int>(static_cast<float>(ctas) * wkv / all + 0.5f);
#endif
    if (qs.units + kvs.units <= ctas) n = smin(smax(n, kvs.units), ctas - qs.units);
    return smin(smax(n, 1), ctas - 1);
}

// A place x (counted from the unit's beginning) as a step of a unit of n
// steps and cost c. Cuts near the unit's ends move to the ends.
EXATTN_HD int place_step(const LineShape &s, int x, int c, int n) {
    const int y = x - s.unit_cost, all = c - s.unit_cost;
    if (y <= 0 || all <= 0) return 0;
    // (an approximate quotient: every CTA forms the same one)
    const float at = static_cast<float>(y) * static_cast<float>(n);
#if defined(__CUDA_ARCH__)
    const int t = smin(static_cast<int>(__fdividef(at, static_cast<float>(all)) + 0.5f), n);
#else
    const int t = smin(static_cast<int>(at / static_cast<float>(all) + 0.5f), n);
#endif
    if (n < 2 * s.min_steps) return 2 * t < n ? 0 : n;
    if (t < s.min_steps) return 0;
    return n - t < s.min_steps ? n : t;
}

// A place on the line: step `step` of `unit` of `head` of sequence `seq`.
// step == count of the unit means its end.
struct Place {
    int seq, head, unit, step;
};

// The place `rem` into the sequence's part of the line (0 <= rem < its cost).
// (The kernels try many units at once.)
inline Place place_in_seq(const LineShape &s, int seq, int sq, int sk, int rem) {
    Place p;
    p.seq = seq;
    const int n = line_units(s, sq, sk);
    const int per_head = line_before(s, sq, sk, n);
    p.head = rem / per_head;
    rem -= p.head * per_head;
    p.unit = 0;  // the last unit that begins at or before rem
    while (p.unit + 1 < n && line_before(s, sq, sk, p.unit + 1) <= rem) ++p.unit;
    int first, count;
    line_steps(s, sq, sk, p.unit, &first, &count);
    const int u0 = line_before(s, sq, sk, p.unit);
    p.step = place_step(s, rem - u0, line_before(s, sq, sk, p.unit + 1) - u0, count);
    return p;
}

// Whether part c begins inside a unit that begins at x0, costs `cost` and has n
// steps, away from its ends: where it cuts it. The parts that share a unit are
// the one before the first cut, and one per cut (part 0 begins at 0, where the
// line begins: it cuts nothing, so there is one before).
EXATTN_HD bool part_cuts(const LineShape &s, const LineDeal &d, int c, int x0, int cost, int n) {
    const int x = part_begin(d, c) - x0;
    if (x <= 0 || x >= cost) return false;
    const int t = place_step(s, x, cost, n);
    return t > 0 && t < n;
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
    int x0, cost, steps;  // of a cut unit: its place on the line and its steps, for part_cuts()
};

// A part's units in order, from place p to place e (seq == b: the line's end).
// x, units: the lengths and units per head of p's sequence, before which
// seq_x0 of the line lie. len(i): a sequence's lengths; emit(range): false
// ends the walk.
template <class Len, class Emit>
EXATTN_HD void walk_part(const LineShape &s, int b, Place p, const Place &e, SeqLen x, int units, int seq_x0,
                         Len len, Emit emit) {
    bool fresh = false;  // p.seq's lengths are still to be read
#pragma unroll 1
    for (;;) {
        if (p.seq >= b) return;
        if (fresh) {
            x = len(p.seq);
            units = line_units(s, x.sq, x.sk);
            fresh = false;
        }
        if (p.unit < units) {
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
                r.slot = p.step == 0 && stop == count ? -1 : p.step > 0 ? 0 : 1;
                r.x0 = r.cost = r.steps = 0;
                if (r.slot >= 0) {
                    const int u0 = line_before(s, x.sq, x.sk, p.unit);
                    r.x0 = seq_x0 + p.head * line_before(s, x.sq, x.sk, units) + u0;
                    r.cost = line_before(s, x.sq, x.sk, p.unit + 1) - u0;
                    r.steps = count;
                }
                if (!emit(r)) return;
            }
            if (last) return;
            p.step = 0;
            if (++p.unit < units) continue;
            p.unit = 0;
            if (++p.head < s.heads) continue;
        }
        p.head = 0;
        seq_x0 += s.heads * line_before(s, x.sq, x.sk, units);
        ++p.seq;
        fresh = true;
    }
}

}  // namespace exattn
