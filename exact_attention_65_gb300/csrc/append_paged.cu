// New rows into a paged K/V cache with their rotation on the way
// (attn_paged_append: 16-bit pages; attn_paged_append_q4: pages of 4 bits), and
// rows out of a 4-bit cache (attn_paged_read_q4).
#include <cuda_runtime.h>

#include "packed.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace exattn {
namespace {

constexpr int kAppendThreads = 256;

// Eight values of 16 bits as four pairs of fp32, and back.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, uint64_t (&y)[4]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (BF16) {
            y[j] = f2_make(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u));
        } else {
            const float2 f = h2_float2(x[j]);
            y[j] = f2_make(f.x, f.y);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const uint64_t (&y)[4]) {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float lo, hi;
        f2_split(y[j], lo, hi);
        x[j] = BF16 ? cvt_pack_bf16(lo, hi) : cvt_pack_f16(lo, hi);
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// ------------------------------------------------------------ append
// Rotation: a pair (a, b) of a token's row at position p becomes (a cos - b sin,
// b cos + a sin) with the table's cos and sin of p and of the pair, in fp32,
// rounded once to the output's type.
//
// A copy with some arithmetic in it: bound by HBM if the arithmetic stays out
// of the way. So a thread holds 16 channels of a row, both halves of 8 pairs
// (16391 tokens of h32 on 8 heads, d128, 412 MB: 72 us, 5.7 TB/s, 86% of the copy
// bandwidth; with 8 channels a thread, the pairs' other halves from another lane, 91
// us and 146 instructions a warp for each 512 bytes): chunks i
// and i + rot / 16 of 8 channels, or, with neighbouring channels paired and
// behind the rotated part, two chunks side by side. Each value is loaded once and
// q may be rotated in place. A token's rows, h of q, then h_kv of k and as many
// of v, are dealt to `per_token` groups of lanes, and the table's values are
// loaded once for all rows of a thread. Loads of rows do not wait for position and
// slot.
template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 16, GROUPS = kAppendThreads / LPR;  // lanes of a row; rows at once
    constexpr int CHUNKS = D / 8;                               // of a row
    constexpr int ROWS = 2;                                     // of q that are loaded together
    const int i = threadIdx.x % LPR, group = threadIdx.x / LPR, lane = threadIdx.x & 31;
    const int sub = group & (a.per_token - 1);  // its place among the token's groups
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (GROUPS >> a.per_token_log2) + (group >> a.per_token_log2);
    const bool there = t < a.tokens;
    const int half = a.rot >> 4;  // chunks of half the rotated part
    const bool turns = i < half, split = turns && !a.interleaved;
    // this thread's chunks
    const int c0 = split ? i : 2 * i, c1 = split ? i + half : 2 * i + 1;

    int64_t pos = -1, to = -1;
    if (there) {
        pos = __ldg(a.positions + t);
        to = __ldg(a.slot_map + t);
    }
    struct Row {
        uint4 x, y;
    };
    auto load = [&](const uint4 *row, bool have) {
        Row r{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (have) {
            r.x = __ldcs(row + c0);
            r.y = __ldcs(row + c1);
        }
        return r;
    };
    const uint4 *q = a.q + t * a.q_stride, *k = a.k + t * a.k_stride, *v = a.v + t * a.v_stride;
    auto load_q = [&](int r) { return load(q + r * CHUNKS, there && r < a.h); };
    auto load_kv = [&](int r) {
        return load(r < a.h_kv ? k + r * CHUNKS : v + (r - a.h_kv) * CHUNKS, there && r < 2 * a.h_kv);
    };
    Row w[ROWS], kv = load_kv(sub);
#pragma unroll
    for (int n = 0; n < ROWS; ++n) w[n] = load_q(n * a.per_token + sub);

    // a position that the table does not have: nothing is written for the token
    const bool live = pos >= 0 && pos < a.max_positions;
    const bool stored = live && to >= 0 && to < a.slots;
    uint64_t cs[4], sn[4];  // of pairs 8 i .. 8 i + 7
    if (live && turns) {
        const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + pos * a.rot) + 2 * i;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float4 x = __ldg(row + n), y = __ldg(row + 2 * half + n);
            cs[2 * n] = f2_make(x.x, x.y), cs[2 * n + 1] = f2_make(x.z, x.w);
            sn[2 * n] = f2_make(y.x, y.y), sn[2 * n + 1] = f2_make(y.z, y.w);
        }
    }
    // x and y are the thread's two chunks
    auto turn = [&](uint64_t(&x)[4], uint64_t(&y)[4]) {
        if (!a.interleaved) {
            // a = x, b = y, eight of each
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t p = f2_mul(y[j], sn[j]), r = f2_mul(x[j], sn[j]);
                x[j] = f2_fma(x[j], cs[j], f2_neg(p));
                y[j] = f2_fma(y[j], cs[j], r);
            }
        } else {
            // (a, b) are neighbours: pairs 0-3 in x, 4-7 in y
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float c[2], s[2], lo, hi;
                f2_split(cs[j], c[0], c[1]);
                f2_split(sn[j], s[0], s[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint64_t &z = j < 2 ? x[2 * j + e] : y[2 * (j - 2) + e];
                    f2_split(z, lo, hi);
                    z = f2_fma(z, f2_make(c[e], c[e]), f2_mul(f2_make(hi, lo), f2_make(-s[e], s[e])));
                }
            }
        }
    };

    // ---- queries (what does not turn is copied bit by bit)
    uint4 *q_out = a.q_out + t * a.q_out_stride;
#pragma unroll 1
    for (int r0 = sub; r0 < a.h; r0 += ROWS * a.per_token) {
        if (r0 != sub) {
#pragma unroll
            for (int n = 0; n < ROWS; ++n) w[n] = load_q(r0 + n * a.per_token);
        }
#pragma unroll
        for (int n = 0; n < ROWS; ++n) {
            const int r = r0 + n * a.per_token;
            if (!live || r >= a.h) continue;
            if (turns) {
                uint64_t x[4], y[4];
                unpack8<BF16>(w[n].x, x);
                unpack8<BF16>(w[n].y, y);
                turn(x, y);
                w[n] = Row{pack8<BF16>(x), pack8<BF16>(y)};
            }
            q_out[r * CHUNKS + c0] = w[n].x;
            q_out[r * CHUNKS + c1] = w[n].y;
        }
    }

    // ---- keys and values
    if constexpr (!Q4) {
#pragma unroll 1
        for (int r = sub; r < 2 * a.h_kv; r += a.per_token) {
            if (r != sub) kv = load_kv(r);
            if (!stored) continue;
            const bool is_k = r < a.h_kv;
            if (is_k && turns) {
                uint64_t x[4], y[4];
                unpack8<BF16>(kv.x, x);
                unpack8<BF16>(kv.y, y);
                turn(x, y);
                kv = Row{pack8<BF16>(x), pack8<BF16>(y)};
            }
            uint4 *row = static_cast<uint4 *>(is_k ? a.k_pages : a.v_pages) +
                         (to * a.h_kv + (is_k ? r : r - a.h_kv)) * CHUNKS;
            row[c0] = kv.x;
            row[c1] = kv.y;
        }
    } else {
        int64_t page = 0, at_row = 0;  // of the token's slot
        if (stored) {
            page = a.slots <= 0xffffffffLL ? static_cast<uint32_t>(to) / static_cast<uint32_t>(a.page_size)
                                           : to / a.page_size;
            at_row = to - page * a.page_size;
        }
        // The 16 channels of a group are chunks 2 n and 2 n + 1: where the other
        // one of this thread's c0 and c1 is (which lane of the row, and which of its two)
        auto where = [&](int c, int *from, int *second) {
            const int o = c ^ 1;
            const bool in_first = !a.interleaved && o < half, in_second = !a.interleaved && !in_first && o < 2 * half;
            *from = lane - i + (in_first ? o : in_second ? o - half : o >> 1);
            *second = in_first ? 0 : in_second ? 1 : o & 1;
        };
        int from0, from1, second0, second1;
        where(c0, &from0, &second0);
        where(c1, &from1, &second1);
#pragma unroll 1
        for (int r0 = 0; r0 < 2 * a.h_kv; r0 += a.per_token) {  // (whole warps: they exchange)
            const int r = r0 + sub;
            if (r0 > 0) kv = load_kv(r);
            const bool is_k = r < a.h_kv;
            uint64_t z[2][4];
            unpack8<BF16>(kv.x, z[0]);
            unpack8<BF16>(kv.y, z[1]);
            if (is_k && turns && live) turn(z[0], z[1]);
            // each chunk's largest magnitude, infinite where a value is not finite
            float f[2][8], m[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                m[n] = 0.f;
                bool finite = true;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f2_split(z[n][j], f[n][2 * j], f[n][2 * j + 1]);
                    m[n] = max3f(m[n], fabsf(f[n][2 * j]), fabsf(f[n][2 * j + 1]));
                    // (infinity - infinity, NaN - NaN are NaN)
                    finite = finite && f[n][2 * j] - f[n][2 * j] == 0.f && f[n][2 * j + 1] - f[n][2 * j + 1] == 0.f;
                }
                if (!finite) m[n] = INFINITY;
            }
            const float a0 = __shfl_sync(0xffffffffu, m[0], from0), b0 = __shfl_sync(0xffffffffu, m[1], from0);
            const float a1 = __shfl_sync(0xffffffffu, m[0], from1), b1 = __shfl_sync(0xffffffffu, m[1], from1);
            m[0] = fmaxf(m[0], second0 ? b0 : a0);
            m[1] = fmaxf(m[1], second1 ? b1 : a1);
            if (!stored || r >= 2 * a.h_kv) continue;
            const float scale = is_k ? a.k_scale : a.v_scale, six = is_k ? a.k_six : a.v_six;
            uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) +
                            (page * a.h_kv + (is_k ? r : r - a.h_kv)) * a.block;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t sb = m[n] == INFINITY ? 0x7fu : q4_scale_byte(__fdiv_rn(m[n], six));
                const float unit = h2_float2(q4_scales_f16(sb)).x * scale;
                // x / unit, corrected once: exact where x is a border between two codes,
                // so that ties go to the even one. Its magnitude is at most 6 times 17 / 16
                // where the scale is a normal number, and below 9 where it is not (m / six
                // just below 1.5 2^-9 rounds to 2^-9): the conversion to codes saturates.
                // The largest scale bounds nothing, and there x is limited first.
                const float inv = unit > 0.f ? __frcp_rn(unit) : 0.f;
                if (sb == 0x7eu) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[n][j] = fminf(fmaxf(f[n][j], -8.f * unit), 8.f * unit);
                }
                const uint64_t inv2 = f2_make(inv, inv), minus2 = f2_make(-unit, -unit);
                uint32_t word = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t y = f2_make(f[n][2 * j], f[n][2 * j + 1]);
                    const uint64_t u = f2_mul(y, inv2);
                    float lo, hi;
                    f2_split(f2_fma(f2_fma(u, minus2, y), inv2, u), lo, hi);
                    word |= q4_code_byte(lo, hi) << (8 * j);
                }
                const int c = n ? c1 : c0;
                reinterpret_cast<uint32_t *>(pool)[at_row * CHUNKS + c] = word;
                if ((c & 1) == 0) pool[a.codes + at_row * (CHUNKS / 2) + (c >> 1)] = sb;
            }
        }
    }
}

// ------------------------------------------------------------ read
// A group of 16 channels of K and of V a thread: 8 bytes of codes and a scale
// in, 32 bytes out (one store where rows begin at multiples of 32 bytes).
constexpr int kReadThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadQ4Args a) {
    const int groups = a.h_kv << a.gpr_log2;  // of a row
    const int64_t n = a.tokens * groups;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kReadThreads + threadIdx.x;
    if (i >= n) return;
    const int64_t t = n <= 0xffffffffLL ? static_cast<uint32_t>(i) / static_cast<uint32_t>(groups) : i / groups;
    const int g = static_cast<int>(i - t * groups);
    const int hd = g >> a.gpr_log2, c = g & ((1 << a.gpr_log2) - 1);
    const int64_t from = __ldg(a.slot_map + t);
    uint2 code[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
    uint32_t sb[2] = {0u, 0u};
    if (from >= 0 && from < a.slots) {
        const int64_t page = a.slots <= 0xffffffffLL
                                 ? static_cast<uint32_t>(from) / static_cast<uint32_t>(a.page_size)
                                 : from / a.page_size;
        const int64_t row = (from - page * a.page_size) << a.gpr_log2;
        const int64_t base = (page * a.h_kv + hd) * a.block;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t *pool = (kv ? a.v_pages : a.k_pages) + base;
            code[kv] = __ldg(reinterpret_cast<const uint2 *>(pool) + row + c);
            sb[kv] = __ldg(pool + a.codes + row + c);
        }
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint32_t s2 = q4_scales_f16(sb[kv] | sb[kv] << 8);
        const float scale = kv ? a.v_scale : a.k_scale;
        uint32_t o[8], x[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            q4_codes_f16(w ? code[kv].y : code[kv].x, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = h2_float2(h2_mul(x[j], s2));
                o[4 * w + j] = BF16 ? cvt_pack_bf16(f.x * scale, f.y * scale) : cvt_pack_f16(f.x * scale, f.y * scale);
            }
        }
        uint4 *dst = (kv ? a.v + t * a.v_stride : a.k + t * a.k_stride) + 2 * g;
        if (a.wide) {
            st_global_v8(dst, o);
        } else {
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

template <int D, bool BF16>
void launch_d(const AppendArgs &a, bool q4, unsigned blocks, cudaStream_t stream) {
    if (q4)
        append_kernel<D, BF16, true><<<blocks, kAppendThreads, 0, stream>>>(a);
    else
        append_kernel<D, BF16, false><<<blocks, kAppendThreads, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &args, int d, bool bf16, bool q4, cudaStream_t stream) {
    AppendArgs a = args;
    // groups of lanes to a token: as few stay idle as a power of two allows
    const int groups = kAppendThreads / (d / 16), rows = a.h < 2 * a.h_kv ? a.h : 2 * a.h_kv;
    a.per_token_log2 = log2_of(rows < groups ? rows : groups);
    if ((1 << a.per_token_log2) > rows) --a.per_token_log2;
    a.per_token = 1 << a.per_token_log2;
    const int tpb = groups >> a.per_token_log2;
    const unsigned n = static_cast<unsigned>((a.tokens + tpb - 1) / tpb);
    switch (d) {
        case 16: bf16 ? launch_d<16, true>(a, q4, n, stream) : launch_d<16, false>(a, q4, n, stream); break;
        case 32: bf16 ? launch_d<32, true>(a, q4, n, stream) : launch_d<32, false>(a, q4, n, stream); break;
        case 64: bf16 ? launch_d<64, true>(a, q4, n, stream) : launch_d<64, false>(a, q4, n, stream); break;
        case 128: bf16 ? launch_d<128, true>(a, q4, n, stream) : launch_d<128, false>(a, q4, n, stream); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

cudaError_t launch_read_q4(const ReadQ4Args &args, int d, bool bf16, cudaStream_t stream) {
    ReadQ4Args a = args;
    a.gpr_log2 = log2_of(d / 16);
    a.wide = 1;
    for (const void *p : {a.k, a.v})
        if (reinterpret_cast<uintptr_t>(p) % 32 != 0) a.wide = 0;
    if ((a.k_stride | a.v_stride) % 2 != 0) a.wide = 0;
    const int64_t n = a.tokens * (static_cast<int64_t>(a.h_kv) << a.gpr_log2);
    const unsigned blocks = static_cast<unsigned>((n + kReadThreads - 1) / kReadThreads);
    if (bf16)
        read_kernel<true><<<blocks, kReadThreads, 0, stream>>>(a);
    else
        read_kernel<false><<<blocks, kReadThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace exattn
