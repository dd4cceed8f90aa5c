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

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &w, float (&y)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = BF16 ? make_float2(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xffff0000u))
                              : h2_float2(x[j]);
        y[2 * j] = f.x;
        y[2 * j + 1] = f.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = BF16 ? cvt_pack_bf16(y[2 * j], y[2 * j + 1]) : cvt_pack_f16(y[2 * j], y[2 * j + 1]);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// ------------------------------------------------------------ append
// Rotation: a pair (a, b) of a token's row at position p becomes (a cos - b sin,
// b cos + a sin) with the table's cos and sin of p and of the pair. Products and
// their sum are rounded one by one in fp32, the result once to the output's type.
//
// A thread holds 8 channels of a row (16 bytes), so d / 8 neighbouring lanes hold
// the row and the other half of a pair comes from a lane of the same warp
// (or, with neighbouring channels paired, from the thread itself): each value
// is loaded once, and q may be rotated in place. The rows of a token, first h
// of q, then h_kv of k and as many of v, are dealt to `per_token` groups of lanes,
// so that the table's values are loaded once and used for every row that a
// thread takes. Loads of rows do not wait for position and slot.
//
// Two lanes hold the 16 channels of a group that share a 4-bit scale.
template <int D, bool BF16, bool Q4>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    constexpr int LPR = D / 8, GROUPS = kAppendThreads / LPR;  // lanes of a row; rows at once
    constexpr int ROWS = 2;                                    // a thread's rows that are loaded together
    const int c = threadIdx.x % LPR, group = threadIdx.x / LPR, lane = threadIdx.x & 31;
    const int sub = group & (a.per_token - 1);  // its place among the token's groups
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (GROUPS >> a.per_token_log2) + (group >> a.per_token_log2);
    const bool there = t < a.tokens;
    const int half = a.rot >> 4;  // chunks of 8 channels of half the rotated part
    const bool turns = c < 2 * half, first = c < half;
    const int partner = a.interleaved || !turns ? lane : first ? lane + half : lane - half;

    int64_t pos = -1, to = -1;
    if (there) {
        pos = __ldg(a.positions + t);
        to = __ldg(a.slot_map + t);
    }
    const uint4 *q = a.q + t * a.q_stride + c, *k = a.k + t * a.k_stride + c, *v = a.v + t * a.v_stride + c;
    uint4 w[ROWS], wk = make_uint4(0u, 0u, 0u, 0u);
    auto load_q = [&](int r0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = r0 + i * a.per_token + sub;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            if (there && r < a.h) w[i] = __ldcs(q + r * LPR);
        }
    };
    auto load_kv = [&](int r0) {
        const int r = r0 + sub;
        if (there && r < 2 * a.h_kv) wk = __ldcs(r < a.h_kv ? k + r * LPR : v + (r - a.h_kv) * LPR);
    };
    load_q(0);
    load_kv(0);

    // a position that the table does not have: nothing is written for the token
    const bool live = pos >= 0 && pos < a.max_positions;
    const bool stored = live && to >= 0 && to < a.slots;
    float cs[8], sn[8];  // a y of the other's sign: y cs + other sn
    if (live && turns) {
        const float *row = a.cos_sin + pos * a.rot;
        if (a.interleaved) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(row + 4 * c));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(row + 8 * half + 4 * c));
            cs[0] = cs[1] = x.x, cs[2] = cs[3] = x.y, cs[4] = cs[5] = x.z, cs[6] = cs[7] = x.w;
            sn[0] = -y.x, sn[1] = y.x, sn[2] = -y.y, sn[3] = y.y;
            sn[4] = -y.z, sn[5] = y.z, sn[6] = -y.w, sn[7] = y.w;
        } else {
            const float *at = row + 8 * (first ? c : c - half);
            const float sign = first ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(at) + i);
                const float4 y = __ldg(reinterpret_cast<const float4 *>(at + 8 * half) + i);
                cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                sn[4 * i] = sign * y.x, sn[4 * i + 1] = sign * y.y;
                sn[4 * i + 2] = sign * y.z, sn[4 * i + 3] = sign * y.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
    }
    // y turned (all lanes of a warp take part); turn: this row does
    auto rotate = [&](const uint4 &x, bool turn, float(&y)[8]) {
        unpack8<BF16>(x, y);
        float z[8];
        if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = y[j ^ 1];
        } else {
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, x.x, partner);
            o.y = __shfl_sync(0xffffffffu, x.y, partner);
            o.z = __shfl_sync(0xffffffffu, x.z, partner);
            o.w = __shfl_sync(0xffffffffu, x.w, partner);
            unpack8<BF16>(o, z);
        }
        if (turn) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(__fmul_rn(y[j], cs[j]), __fmul_rn(z[j], sn[j]));
        }
    };

    // ---- queries
    uint4 *q_out = a.q_out + t * a.q_out_stride + c;
#pragma unroll 1
    for (int r0 = 0; r0 < a.h; r0 += ROWS * a.per_token) {
        if (r0 > 0) load_q(r0);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (r0 + i * a.per_token >= a.h) break;  // (the same for the whole block)
            const int r = r0 + i * a.per_token + sub;
            float y[8];
            rotate(w[i], turns, y);
            // (what does not turn is copied bit by bit)
            if (live && r < a.h) q_out[r * LPR] = turns ? pack8<BF16>(y) : w[i];
        }
    }

    // ---- keys and values
    int64_t page = 0, at_row = 0;  // of the token's slot
    if (Q4 && stored) {
        page = a.slots <= 0xffffffffLL ? static_cast<uint32_t>(to) / static_cast<uint32_t>(a.page_size) : to / a.page_size;
        at_row = to - page * a.page_size;
    }
#pragma unroll 1
    for (int r0 = 0; r0 < 2 * a.h_kv; r0 += a.per_token) {
        if (r0 > 0) load_kv(r0);
        const int r = r0 + sub;
        const bool is_k = r < a.h_kv, row = stored && r < 2 * a.h_kv;
        const int hd = is_k ? r : r - a.h_kv;
        float y[8];
        rotate(wk, turns && is_k, y);
        if constexpr (!Q4) {
            uint4 *pool = static_cast<uint4 *>(is_k ? a.k_pages : a.v_pages);
            if (row) pool[(to * a.h_kv + hd) * LPR + c] = turns && is_k ? pack8<BF16>(y) : wk;
        } else {
            // the group's largest magnitude, infinite where a value is not finite
            float m = 0.f;
            bool finite = true;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m = fmaxf(m, fabsf(y[j]));
                finite = finite && fabsf(y[j]) <= 3.402823466e+38f;
            }
            if (!finite) m = INFINITY;
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            if (!row) continue;
            const uint32_t sb = m == INFINITY ? 0x7fu : q4_scale_byte(__fdiv_rn(m, is_k ? a.k_six : a.v_six));
            const float unit = h2_float2(q4_scales_f16(sb)).x * (is_k ? a.k_scale : a.v_scale);
            // y / unit, corrected once: exact where y is a border between two codes,
            // so that ties go to the even one. (At most 6 times 17 / 16 unless
            // the scale is at its largest.)
            const float inv = unit > 0.f ? __frcp_rn(unit) : 0.f;
            if (sb == 0x7eu) {
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fminf(fmaxf(y[j], -8.f * unit), 8.f * unit);
            }
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float u[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float q0 = y[j + e] * inv;
                    u[e] = __fmaf_rn(__fmaf_rn(-q0, unit, y[j + e]), inv, q0);
                }
                word |= q4_code_byte(u[0], u[1]) << (4 * j);
            }
            uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + (page * a.h_kv + hd) * a.block;
            reinterpret_cast<uint32_t *>(pool)[at_row * LPR + c] = word;
            if ((c & 1) == 0) pool[a.codes + at_row * (LPR / 2) + (c >> 1)] = sb;
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
    // as many groups of lanes to a token as it has rows of q, or of k and v
    const int groups = kAppendThreads / (d / 8), rows = a.h > 2 * a.h_kv ? a.h : 2 * a.h_kv;
    a.per_token_log2 = log2_of(rows < groups ? rows : groups);
    if ((1 << a.per_token_log2) > groups) --a.per_token_log2;
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
