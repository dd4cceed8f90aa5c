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
constexpr int kAppendRows = 4;  // rows of a thread that are loaded together

__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return h2_float2(w);
}

// ------------------------------------------------------------ append
// Rotation: a pair (a, b) of a token's row at position p becomes (a cos - b sin,
// b cos + a sin) with the table's cos and sin of p and of the pair. Products and
// their sum are rounded one by one in fp32, the result once to the output's type.
//
// A thread holds 8 channels of a row (16 bytes), so d / 8 neighbouring lanes hold
// the row and the other half of a pair comes from a lane of the same warp
// (or, with neighbouring channels paired, from the thread itself): each value
// is loaded once, and q may be rotated in place. The rows of a token (h of q,
// h_kv of k and of v) are dealt to `per_token` groups of lanes, so that the
// table's values are loaded once and used for every row that a thread takes.
//
// Two lanes hold the 16 channels of a group that share a 4-bit scale.
template <bool BF16, bool Q4>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    const int lpr = a.d >> 3;                            // lanes of a row: 2 .. 16
    const int slot = threadIdx.x >> a.lpr_log2;          // this row group
    const int c = threadIdx.x & (lpr - 1);               // this thread's 8 channels of the row
    const int sub = slot & (a.per_token - 1);            // its place among the token's groups
    const int tokens_per_block = (kAppendThreads >> a.lpr_log2) >> a.per_token_log2;
    const int rows = a.h + 2 * a.h_kv;
    const int half = a.rot >> 4;                         // chunks of 8 channels of half the rotated part
    const bool turns = c < (a.rot >> 3);
    const bool first = c < half;                         // (a of the pairs (a, b))
    const int lane = threadIdx.x & 31;
    const int partner = a.interleaved || !turns ? lane : first ? lane + half : lane - half;

    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block; t0 < a.tokens;
         t0 += static_cast<int64_t>(gridDim.x) * tokens_per_block) {
        const int64_t t = t0 + (slot >> a.per_token_log2);
        int64_t pos = -1, to = -1;
        if (t < a.tokens) {
            pos = __ldg(a.positions + t);
            to = __ldg(a.slot_map + t);
        }
        // a position that the table does not have: nothing is written for the token
        const bool live = pos >= 0 && pos < a.max_positions;
        const bool stored = live && to >= 0 && to < a.slots;
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i] = 1.f;
            sn[i] = 0.f;
        }
        if (live && turns) {
            const float *row = a.cos_sin + pos * a.rot;
            if (a.interleaved) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(row + 4 * c));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(row + (a.rot >> 1) + 4 * c));
                cs[0] = cs[1] = x.x, cs[2] = cs[3] = x.y, cs[4] = cs[5] = x.z, cs[6] = cs[7] = x.w;
                sn[0] = -y.x, sn[1] = y.x, sn[2] = -y.y, sn[3] = y.y;
                sn[4] = -y.z, sn[5] = y.z, sn[6] = -y.w, sn[7] = y.w;
            } else {
                const float *at = row + 8 * (first ? c : c - half);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(at) + i);
                    const float4 y = __ldg(reinterpret_cast<const float4 *>(at + (a.rot >> 1)) + i);
                    cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
                    const float sign = first ? -1.f : 1.f;
                    sn[4 * i] = sign * y.x, sn[4 * i + 1] = sign * y.y;
                    sn[4 * i + 2] = sign * y.z, sn[4 * i + 3] = sign * y.w;
                }
            }
        }
        // where the token's row of a pool's first head lies, in 16-byte words (16 bits) or bytes
        int64_t page = 0, at_row = 0;
        if (Q4 && stored) {
            if (a.slots <= 0xffffffffLL) {
                page = static_cast<uint32_t>(to) / static_cast<uint32_t>(a.page_size);
            } else {
                page = to / a.page_size;
            }
            at_row = to - page * a.page_size;
        }
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += kAppendRows * a.per_token) {
            uint4 w[kAppendRows];
#pragma unroll
            for (int i = 0; i < kAppendRows; ++i) {
                const int r = r0 + i * a.per_token + sub;
                w[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < a.h) {
                    if (live) w[i] = __ldcs(a.q + t * a.q_stride + r * lpr + c);
                } else if (r < a.h + a.h_kv) {
                    if (stored) w[i] = __ldcs(a.k + t * a.k_stride + (r - a.h) * lpr + c);
                } else if (r < rows) {
                    if (stored) w[i] = __ldcs(a.v + t * a.v_stride + (r - a.h - a.h_kv) * lpr + c);
                }
            }
#pragma unroll
            for (int i = 0; i < kAppendRows; ++i) {
                if (r0 + i * a.per_token >= rows) break;  // (the same for the whole block)
                const int r = r0 + i * a.per_token + sub;
                uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 own = unpack16(x[j], BF16);
                    y[2 * j] = own.x;
                    y[2 * j + 1] = own.y;
                }
                float z[8];
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = y[j ^ 1];
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 other = unpack16(__shfl_sync(0xffffffffu, x[j], partner), BF16);
                        z[2 * j] = other.x;
                        z[2 * j + 1] = other.y;
                    }
                }
                if (turns && r < a.h + a.h_kv) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(__fmul_rn(y[j], cs[j]), __fmul_rn(z[j], sn[j]));
                }
                if constexpr (Q4) {
                    // amax of the group, and whether all of it is finite
                    float m = 0.f;
                    bool finite = true;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        m = fmaxf(m, fabsf(y[j]));
                        finite = finite && fabsf(y[j]) <= 3.402823466e+38f;
                    }
                    if (!finite) m = INFINITY;
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    if (r >= a.h) {
                        if (stored && r < rows) {
                            const bool is_k = r < a.h + a.h_kv;
                            const float scale = is_k ? a.k_scale : a.v_scale;
                            const float six = is_k ? a.k_six : a.v_six;
                            const uint32_t sb = m == INFINITY ? 0x7fu : q4_scale_byte(__fdiv_rn(m, six));
                            const float unit = h2_float2(q4_scales_f16(sb)).x * scale;
                            // x / unit, corrected once: exact where x is a border between
                            // two codes, so that ties go to the even one
                            const float inv = unit > 0.f ? __frcp_rn(unit) : 0.f;
                            uint32_t word = 0;
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                float u[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float q0 = y[j + e] * inv;
                                    const float q1 = __fmaf_rn(__fmaf_rn(-q0, unit, y[j + e]), inv, q0);
                                    u[e] = fabsf(q0) < 8.f ? q1 : q0;
                                }
                                word |= q4_code_byte(u[0], u[1]) << (4 * j);
                            }
                            const int hd = is_k ? r - a.h : r - a.h - a.h_kv;
                            uint8_t *pool = static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) +
                                            (page * a.h_kv + hd) * a.block;
                            reinterpret_cast<uint32_t *>(pool)[at_row * lpr + c] = word;
                            if ((c & 1) == 0) pool[a.codes + at_row * (lpr >> 1) + (c >> 1)] = sb;
                        }
                        continue;
                    }
                }
                uint4 o;
                if (BF16) {
                    o = make_uint4(cvt_pack_bf16(y[0], y[1]), cvt_pack_bf16(y[2], y[3]), cvt_pack_bf16(y[4], y[5]),
                                   cvt_pack_bf16(y[6], y[7]));
                } else {
                    o = make_uint4(cvt_pack_f16(y[0], y[1]), cvt_pack_f16(y[2], y[3]), cvt_pack_f16(y[4], y[5]),
                                   cvt_pack_f16(y[6], y[7]));
                }
                // what does not turn is copied bit by bit
                if (!turns || r >= a.h + a.h_kv) o = w[i];
                if (r < a.h) {
                    if (live) a.q_out[t * a.q_out_stride + r * lpr + c] = o;
                } else if (!Q4 && stored && r < rows) {
                    const int hd = r < a.h + a.h_kv ? r - a.h : r - a.h - a.h_kv;
                    uint4 *pool = static_cast<uint4 *>(r < a.h + a.h_kv ? a.k_pages : a.v_pages);
                    pool[(to * a.h_kv + hd) * lpr + c] = o;
                }
            }
        }
    }
}

// ------------------------------------------------------------ read
// A group of 16 channels a thread: 8 bytes of codes and a scale in, 32 bytes
// out, of K and of V of a token.
constexpr int kReadThreads = 256;

template <bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadQ4Args a) {
    const int groups = a.h_kv << a.gpr_log2;  // of a row
    const int64_t n = a.tokens * groups;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kReadThreads + threadIdx.x;
    if (i >= n) return;
    int64_t t;
    if (n <= 0xffffffffLL)
        t = static_cast<uint32_t>(i) / static_cast<uint32_t>(groups);
    else
        t = i / groups;
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
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

}  // namespace

cudaError_t launch_append(const AppendArgs &args, bool bf16, bool q4, int num_sms, cudaStream_t stream) {
    AppendArgs a = args;
    a.lpr_log2 = log2_of(a.d / 8);
    const int groups = kAppendThreads >> a.lpr_log2, rows = a.h + 2 * a.h_kv;
    a.per_token_log2 = log2_of(rows < groups ? rows : groups);
    a.per_token = 1 << a.per_token_log2;
    const int tpb = groups >> a.per_token_log2;
    int64_t blocks = (a.tokens + tpb - 1) / tpb;
    if (blocks > 64ll * num_sms) blocks = 64ll * num_sms;
    const unsigned n = static_cast<unsigned>(blocks);
    if (q4)
        bf16 ? append_kernel<true, true><<<n, kAppendThreads, 0, stream>>>(a)
             : append_kernel<false, true><<<n, kAppendThreads, 0, stream>>>(a);
    else
        bf16 ? append_kernel<true, false><<<n, kAppendThreads, 0, stream>>>(a)
             : append_kernel<false, false><<<n, kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_read_q4(const ReadQ4Args &args, bool bf16, cudaStream_t stream) {
    ReadQ4Args a = args;
    a.gpr_log2 = log2_of(a.d / 16);
    const int64_t n = a.tokens * (static_cast<int64_t>(a.h_kv) << a.gpr_log2);
    const unsigned blocks = static_cast<unsigned>((n + kReadThreads - 1) / kReadThreads);
    if (bf16)
        read_kernel<true><<<blocks, kReadThreads, 0, stream>>>(a);
    else
        read_kernel<false><<<blocks, kReadThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace exattn
