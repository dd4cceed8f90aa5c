// A few new rows of each request over a cache held in 4 bits
// (attn_chunk_paged_q4: all requests where none is said to have more than 16 rows to
// a K/V head; in other batches those with up to 8, or a token of up to 16).
//
// The mathematics is the forward's: S = scale Q K^T, an online softmax, O = P V,
// and per key 1.125 bytes of K and V a channel are read once. What bounds it is
// the way from those bytes to the tensor core: at the copy bandwidth an SM gets
// 128 channels of K and V of 16 keys every 100 cycles, 4,096 codes to be
// widened. So the codes go from HBM into a warp's own ring in shared memory
// (bulk copies, two or four for 16 keys) and from there straight into registers
// in the order in which mma.sync wants its operand; nothing widened is written
// back.
//
// S^T = K Q^T and O^T = V^T P^T: keys (channels) are the 16 rows of the left
// operand, query rows the 8 columns of the right one, so that 1 to 8 rows fill
// the product (tcgen05's least tile is 64 rows, and its operands lie in shared
// memory). The order of channels within a product, and of keys, is free:
//   K  lane (g, t) holds D / 4 neighbouring channels of keys k(g) and k(g + 8):
//      a byte of codes is a pair of channels, as the operand wants them
//   V  lane (g, t) holds D / 8 neighbouring channels of keys k(2t), k(2t + 1),
//      k(2t + 8), k(2t + 9); the operand wants pairs of keys, so the codes of two
//      keys are merged into bytes of two before they are widened
//   k(r) = r ^ (r >> 2 & 1): reads of K meet no bank twice, those of V at most
//      twice (at D = 128)
//   P  the C fragment of S^T, rounded to fp16 and transposed 8 by 8 (movmatrix)
// A code times its scale is exact in fp16 (q4.cuh). bf16 queries are brought into
// fp16 with a power of two a row (largest value in [2^14, 2^15): nothing above
// 2^-31 of it is rounded), which goes into the softmax's scale.
//
// Every warp is on its own: the line of work (packed_sched.h) is dealt to warps,
// each takes its share of a unit's keys from its first tile to its last, and
// ranges of a cut unit leave normalised fp32 O_i and LSE_i (log2) in the
// workspace. The range that finishes last joins them in the order of the keys,
// so the result does not depend on who that is; those of a CTA's warps are joined
// in shared memory first, and where more than kJoin are left, groups of so many.
// (With a CTA's warps sharing every unit and meeting at its end, 64 requests of 200
// to 8192 keys took 83 us, a fifth of it waiting for one another; so 66.)
//
// Measured, h32/8 d128 with 16-key pages: 64 requests of 4096 keys 73 us, of 8192
// 126, by the difference 5.7 TB/s, 86% of the copy bandwidth; the start takes 8 us
// (to the first tiles of every warp) and uneven ends with the joins some 10. A warp
// executes 316 instructions for 16 keys, 128 of them for widening, with the ALU pipe,
// half of which they need, at 50%: what is left is the latency of their chains, which
// 16 warps do not hide. Tried: 18 and 20 warps with fewer registers and a tile at a
// time (4.0 TB/s), S of one slot beside O of the last (4.7), the softmax's scale
// folded into one multiplication (the same).
#include "packed.h"
#include "packed_dev.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace exattn {
namespace {

constexpr float kShift = 6.0f;  // P is 2^6 times the softmax's, at most 2^14
constexpr int kJoin = 10;       // results joined at once

template <int D, int NT>
struct DecGeom {
    static constexpr int ROWS = 8 * NT;
    // registers decide: 128 a thread for 16 warps an SM, 168 for 12 (D = 128 spills 40
    // to 52 bytes with 8 rows, in the joins only; with 16 rows 224, 196 without the
    // joins, and D = 64 52 to 76, 40 without)
    static constexpr int WARPS = decode_q4_warps(ROWS), CTAS = decode_q4_ctas(ROWS);
    static constexpr int J = D / 16;                    // products of 16 channels
    static constexpr int CODE_BYTES = 16 * q4_code_bytes(D);    // of a tile of K or V
    static constexpr int SCALE_BYTES = 16 * q4_scale_bytes(D);
    static constexpr int OFF_KS = CODE_BYTES, OFF_V = OFF_KS + SCALE_BYTES, OFF_VS = OFF_V + CODE_BYTES;
    static constexpr int STAGE = OFF_VS + SCALE_BYTES;  // a tile: 16 keys
    // tiles that a warp takes at once, as many as registers allow (64 requests of 8192
    // keys, h16/4 d64: 55 us with 2, 52 with 4)
    static constexpr int B = D == 128 ? 2 : 4;
    static constexpr int DEPTH = D == 128 ? 3 : 2;      // slots of B tiles of a warp's ring
    static constexpr int RING = (DEPTH * B * STAGE + 127) / 128 * 128;  // bytes
    static constexpr int OFF_BAR = WARPS * RING;       // [WARPS, DEPTH] a slot has landed
    static constexpr int OFF_SUM = OFF_BAR + WARPS * DEPTH * 8;
    static constexpr int OFF_MISC = OFF_SUM + WARPS * 12;
    static constexpr int SMEM_BYTES = OFF_MISC + 16 + WARPS * 4;  // abort, arrivals of the CTA's warps
    static_assert(RING >= ROWS * (D + 1) * 4, "a ring holds a range's results");
    static_assert(STAGE % 16 == 0 && (SMEM_BYTES + 1024) * CTAS <= 228 * 1024, "shared memory budget");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Words of shared memory.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}

// c += a b: a 16 x 16 (rows), b 16 x 8 (columns), fp16, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// The key in its tile that row r of the products stands for.
__device__ __forceinline__ int key_of(int r) { return r ^ (r >> 2 & 1); }

// As arrive_last(), by a warp whose results are written. Lane 0 counts for all
// of them: the barriers order the other lanes' stores before its fence, and its
// second fence before their loads (a shuffle alone orders no memory).
__device__ __forceinline__ bool warp_arrives_last(uint32_t *counter, uint32_t call, int n) {
    __syncwarp();
    int last = 0;
    if ((threadIdx.x & 31) == 0) {
        __threadfence();
        last = arrive_last(counter, call, n);
        __threadfence();
    }
    last = __shfl_sync(0xffffffffu, last, 0);
    __syncwarp();
    return last != 0;
}

// The same among a CTA's warps, for results in shared memory.
__device__ __forceinline__ bool warp_arrives_last_in_cta(int *counter, int n) {
    __syncwarp();
    int old = 0;
    if ((threadIdx.x & 31) == 0) {
        __threadfence_block();
        old = atomicAdd(counter, 1);
        __threadfence_block();
    }
    old = __shfl_sync(0xffffffffu, old, 0);
    __syncwarp();
    return old == n - 1;
}

// A lane's codes of one key for S: D / 4 channels, a word for 8.
template <int D>
__device__ __forceinline__ void load_k(uint32_t stage, int key, int t, uint32_t (&w)[(D + 31) / 32]) {
    if constexpr (D == 128) {
        const uint4 x = lds128(stage + key * 64 + t * 16);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (D == 64) {
        const uint2 x = lds64(stage + key * 32 + t * 8);
        w[0] = x.x, w[1] = x.y;
    } else if constexpr (D == 32) {
        w[0] = lds32(stage + key * 16 + t * 4);
    } else {
        w[0] = lds16(stage + key * 8 + t * 2);
    }
}

// ... and its scales: of channels t D / 4 on, in both halves each.
template <int D>
__device__ __forceinline__ void load_ks(uint32_t scales, int key, int t, uint32_t (&s)[D == 128 ? 2 : 1]) {
    if constexpr (D == 128) {
        const uint32_t x = q4_scales_f16(lds16(scales + key * 8 + t * 2));
        s[0] = __byte_perm(x, 0, 0x1010);
        s[1] = __byte_perm(x, 0, 0x3232);
    } else {
        const uint32_t x = lds8(scales + (D == 64 ? key * 4 + t : D == 32 ? key * 2 + (t >> 1) : key));
        s[0] = q4_scales_f16(x | x << 8);
    }
}

// A lane's codes of one key for O: D / 8 channels.
template <int D>
__device__ __forceinline__ void load_v(uint32_t stage, int key, int g, uint32_t (&w)[(D + 63) / 64]) {
    if constexpr (D == 128) {
        const uint2 x = lds64(stage + key * 64 + g * 8);
        w[0] = x.x, w[1] = x.y;
    } else if constexpr (D == 64) {
        w[0] = lds32(stage + key * 32 + g * 4);
    } else if constexpr (D == 32) {
        w[0] = lds16(stage + key * 16 + g * 2);
    } else {
        w[0] = lds8(stage + key * 8 + g);
    }
}
template <int D>
__device__ __forceinline__ uint32_t load_vs(uint32_t scales, int key, int g) {
    return lds8(scales + (D == 128 ? key * 8 + g : D == 64 ? key * 4 + (g >> 1) : D == 32 ? key * 2 + (g >> 2) : key));
}

// A warp's ring: slots on their way, and the next one to be taken.
struct TileRing {
    int get = 0, put = 0, pending = 0;
    uint32_t phase = 0;  // of the slot `get`
};

// Where a range of a cut unit leaves its results: its unit's part `i` of those
// from CTA part `first` on.
__device__ __forceinline__ int64_t part_place(int first, int i) {
    return 2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0);
}

// The parts that share a cut unit, and the first of them (by the warp that has
// one of them, so that there is a cut to be found).
__device__ __forceinline__ void who_shares(const LineShape &s, const LineDeal &d, const UnitRange &r, int *first,
                                           int *nparts) {
    const int lane = threadIdx.x & 31;
    int lo, hi;
    parts_inside(d, r.x0, r.cost, &lo, &hi);
    int a = lo, z = hi;
    uint32_t in = 0;
#pragma unroll 1
    for (; a <= hi; a += 32) {
        in = __ballot_sync(0xffffffffu, a + lane <= hi && part_cuts<true>(s, d, a + lane, r.x0, r.cost, r.steps));
        if (in != 0) break;
    }
    a += in != 0 ? __ffs(in) - 1 : 0;
#pragma unroll 1
    for (; z >= lo; z -= 32) {
        in = __ballot_sync(0xffffffffu, z - lane >= lo && part_cuts<true>(s, d, z - lane, r.x0, r.cost, r.steps));
        if (in != 0) break;
    }
    z -= in != 0 ? __ffs(in) - 1 : 0;
    *first = a - 1;
    *nparts = z - a + 2;
}

// A range of a unit: its tiles, and its results. False: a wait ran out.
template <int D, bool BF16, int NT>
__device__ __forceinline__ bool take_range(const UnitRange &r, const SeqInfo &seq, const LineShape &shape,
                                           const LineDeal &deal, int part, uint8_t *smem, uint32_t ring,
                                           uint32_t landed, TileRing &q, const PackArgs &a, const WaitGuard &guard) {
    using G = DecGeom<D, NT>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tok0 = r.unit * a.tile_tokens;
    // the range's tiles, and the end of its keys
    const int first = r.step0 * 2, end = min((r.step0 + r.nstep) * 2, (seq.sk + 15) >> 4);
    const int limit = min(seq.sk, 16 * end);

    // ---- fetching: lane i knows the page of tile i of 32, and the next 32's;
    // lanes below B fetch a slot's tiles
    const int32_t *table = a.block_table + static_cast<int64_t>(r.seq) * a.max_pages;
    int page = 0, row = 0, page2 = 0, row2 = 0, issued = first;
    auto look_up = [&](int tile, int *pg, int *rw) {
        if (tile + lane < end) {
            const int p = divided(static_cast<uint32_t>(tile + lane), a.page_mul, a.page_div);
            *rw = 16 * (tile + lane) - p * a.page_size;
            *pg = __ldg(table + p);
        }
    };
    auto refill = [&] {
#pragma unroll 1
        while (q.pending < G::DEPTH && issued < end) {
            const int at = issued - first & 31;
            if (at == 0 && issued != first) {
                page = page2;
                row = row2;
                look_up(issued + 32, &page2, &row2);
            }
            const int src = at + (lane & (G::B - 1));
            const int pg = __shfl_sync(0xffffffffu, page, src), rw = __shfl_sync(0xffffffffu, row, src);
            if (lane < G::B) {
                const uint32_t bar = landed + 8u * q.put;
                if (issued + lane < end) {
                    // (a page of all heads is less than 2^31 bytes)
                    const uint8_t *kp = a.k4 + r.head * a.block4 +
                                        static_cast<uint64_t>(static_cast<uint32_t>(min(max(pg, 0), a.num_pages - 1))) *
                                            a.page_bytes;
                    const uint8_t *vp = kp + (a.v4 - a.k4);
                    const uint32_t dst = ring + (q.put * G::B + lane) * G::STAGE;
                    mbar_arrive_expect_tx(bar, G::STAGE);
                    if (a.page_size == 16) {  // the page's scales follow its codes
                        bulk_load(dst, kp, G::OFF_V, bar);
                        bulk_load(dst + G::OFF_V, vp, G::OFF_V, bar);
                    } else {
                        const int codes = rw * q4_code_bytes(D);
                        const int scales = a.page_size * q4_code_bytes(D) + rw * q4_scale_bytes(D);
                        bulk_load(dst, kp + codes, G::CODE_BYTES, bar);
                        bulk_load(dst + G::OFF_KS, kp + scales, G::SCALE_BYTES, bar);
                        bulk_load(dst + G::OFF_V, vp + codes, G::CODE_BYTES, bar);
                        bulk_load(dst + G::OFF_VS, vp + scales, G::SCALE_BYTES, bar);
                    }
                } else {
                    mbar_arrive(bar);  // (the second tile is not there)
                }
            }
            issued += G::B;
            if (++q.put == G::DEPTH) q.put = 0;
            ++q.pending;
        }
    };
    look_up(first, &page, &row);
    look_up(first + 32, &page2, &row2);
    if (!(a.flags & kFlagSkipLoads)) refill();
    int first_part = 0, nparts = 1;  // of a cut unit
    if (r.slot >= 0) who_shares(shape, deal, r, &first_part, &nparts);

    // ---- queries: row n of the products is token n / group, head n % group
    uint32_t qf[NT][2 * G::J];
    float c[NT][2];       // the softmax's scale of queries 2t and 2t + 1
    int all_see = limit;  // keys that every row sees
    // keys of the range that row n sees
    auto row_sees = [&](int n) {
        const int tok = tok0 + ((n * a.group_inv) >> 16);
        return a.causal && tok < seq.sq ? min(limit, tok + seq.sk - seq.sq + 1) : limit;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = 8 * nt + g, rt = (n * a.group_inv) >> 16;
#pragma unroll
        for (int i = 0; i < 2 * G::J; ++i) qf[nt][i] = 0u;
        if (rt < a.tile_tokens && tok0 + rt < seq.sq) {
            const uint16_t *src = static_cast<const uint16_t *>(a.q) +
                                  (static_cast<int64_t>(seq.q0) + tok0 + rt) * a.q_stride +
                                  (r.head * a.group + n - rt * a.group) * D + t * (D / 4);
            if constexpr (D >= 32) {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src) + i);
                    qf[nt][4 * i] = y.x, qf[nt][4 * i + 1] = y.y, qf[nt][4 * i + 2] = y.z, qf[nt][4 * i + 3] = y.w;
                }
            } else {
                const uint2 y = __ldg(reinterpret_cast<const uint2 *>(src));
                qf[nt][0] = y.x, qf[nt][1] = y.y;
            }
        }
        float factor = 1.0f;
        if constexpr (BF16) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * G::J; ++i)
                top = max3f(top, fabsf(__uint_as_float(qf[nt][i] << 16)),
                            fabsf(__uint_as_float(qf[nt][i] & 0xffff0000u)));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^e and 2^-e as bits: e = the exponent of the largest value less 14
            const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14, -112);
            factor = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 2 * G::J; ++i)
                qf[nt][i] = cvt_pack_f16(__uint_as_float(qf[nt][i] << 16) * inv,
                                         __uint_as_float(qf[nt][i] & 0xffff0000u) * inv);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            c[nt][e] = a.scale_log2 * __shfl_sync(0xffffffffu, factor, (2 * t + e) * 4);
            all_see = min(all_see, row_sees(8 * nt + 2 * t + e));
        }
    }
    all_see = __reduce_min_sync(0xffffffffu, all_see);

    float o[NT][G::J][4], m[NT][2], neg[NT][2], l[NT][2];
    auto clear = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < G::J; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][j][i] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                neg[nt][e] = 0.f;  // kShift - m, of use once m is finite
                l[nt][e] = 0.f;
            }
        }
    };
    clear();
    {
        // S^T = K Q^T of the tiles in a slot
        auto scores = [&](uint32_t stage, float(&s)[G::B][NT][4]) {
#pragma unroll
            for (int b = 0; b < G::B; ++b) {
                const uint32_t at = stage + b * G::STAGE;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[b][nt][i] = 0.f;
                uint32_t w0[(D + 31) / 32], w1[(D + 31) / 32], s0[D == 128 ? 2 : 1], s1[D == 128 ? 2 : 1];
                const int k0 = key_of(g), k1 = k0 + 8;
                load_k<D>(at, k0, t, w0);
                load_k<D>(at, k1, t, w1);
                load_ks<D>(at + G::OFF_KS, k0, t, s0);
                load_ks<D>(at + G::OFF_KS, k1, t, s1);
#pragma unroll
                for (int i = 0; i < (D + 31) / 32; ++i) {
                    uint32_t x0[4], x1[4];
                    q4_codes_f16(w0[i], x0);
                    q4_codes_f16(w1[i], x1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x0[e] = h2_mul(x0[e], s0[D == 128 ? i / 2 : 0]);
                        x1[e] = h2_mul(x1[e], s1[D == 128 ? i / 2 : 0]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(s[b][nt], x0[0], x1[0], x0[1], x1[1], qf[nt][4 * i % (2 * G::J)],
                                 qf[nt][(4 * i + 1) % (2 * G::J)]);
                        if (D > 16)
                            mma16816(s[b][nt], x0[2], x1[2], x0[3], x1[3], qf[nt][(4 * i + 2) % (2 * G::J)],
                                     qf[nt][(4 * i + 3) % (2 * G::J)]);
                    }
                }
            }
        };
        // P of the tiles from `tile` on, whose S is given, with the running max and sum
        uint32_t p[G::B][NT][2];
        auto softmax = [&](int tile, float(&s)[G::B][NT][4]) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4 * G::B; ++i) s[i >> 2][nt][i & 3] *= c[nt][i & 1];
            if (16 * (tile + (G::B - 1)) + 16 > all_see) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int sees = row_sees(8 * nt + 2 * t + e) - 16 * tile - key_of(g);
#pragma unroll
                        for (int i = 0; i < 2 * G::B; ++i)
                            if (16 * (i >> 1) + 8 * (i & 1) >= sees) s[i >> 1][nt][2 * (i & 1) + e] = -INFINITY;
                    }
            }
            float top[NT][2];
            bool need = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
#pragma unroll
                    for (int b = 1; b < G::B; ++b) top[nt][e] = max3f(top[nt][e], s[b][nt][e], s[b][nt][e + 2]);
                    need = need || top[nt][e] > m[nt][e] + 8.0f;
                }
            // The reference max moves when a tile exceeds it by more than 8 (log2)
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[nt][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        if (x > m[nt][e] + 8.0f) {
                            const float alpha = fast_exp2(m[nt][e] - x);
                            m[nt][e] = x;
                            neg[nt][e] = kShift - x;
                            l[nt][e] *= alpha;
#pragma unroll
                            for (int j = 0; j < G::J; ++j) {
                                o[nt][j][e] *= alpha;
                                o[nt][j][e + 2] *= alpha;
                            }
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4 * G::B; ++i) {
                    float &x = s[i >> 2][nt][i & 3];
                    x = fast_exp2(x + neg[nt][i & 1]);
                    l[nt][i & 1] += x;
                }
#pragma unroll
                for (int i = 0; i < 2 * G::B; ++i)
                    p[i >> 1][nt][i & 1] =
                        transpose8x8(cvt_pack_f16(s[i >> 1][nt][2 * (i & 1)], s[i >> 1][nt][2 * (i & 1) + 1]));
            }
        };
        // O^T += V^T P^T of the tiles in a slot
        auto values = [&](int tile, uint32_t stage) {
            // Scales are not negative, and a NaN (a key whose value is no number, or
            // what lies behind the sequence) counts as 0 here: its product with a P
            // of 0 would be NaN
            uint32_t bad = 0;
#pragma unroll
            for (int b = 0; b < G::B; ++b) {
                const uint32_t at = stage + b * G::STAGE + G::OFF_V;
                uint32_t lo[2][(D + 63) / 64], hi[2][(D + 63) / 64], sv[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w0[(D + 63) / 64], w1[(D + 63) / 64];
                    const int k0 = key_of(2 * t) + 8 * half, k1 = key_of(2 * t + 1) + 8 * half;
                    load_v<D>(at, k0, g, w0);
                    load_v<D>(at, k1, g, w1);
                    const uint32_t read = q4_scales_f16(load_vs<D>(at + G::CODE_BYTES, k0, g) |
                                                        load_vs<D>(at + G::CODE_BYTES, k1, g) << 8);
                    sv[half] = h2_max0(read);
                    bad |= read ^ sv[half];
#pragma unroll
                    for (int i = 0; i < (D + 63) / 64; ++i) {
                        lo[half][i] = (w0[i] & 0x0f0f0f0fu) | ((w1[i] << 4) & 0xf0f0f0f0u);
                        hi[half][i] = ((w0[i] >> 4) & 0x0f0f0f0fu) | (w1[i] & 0xf0f0f0f0u);
                    }
                }
#pragma unroll
                for (int i = 0; i < (D + 63) / 64; ++i) {
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    q4_codes_f16(lo[0][i], a0);
                    q4_codes_f16(hi[0][i], a1);
                    q4_codes_f16(lo[1][i], a2);
                    q4_codes_f16(hi[1][i], a3);
#pragma unroll
                    for (int e = 0; e < (D < 64 ? D / 16 : 4); ++e) {
                        a0[e] = h2_mul(a0[e], sv[0]);
                        a1[e] = h2_mul(a1[e], sv[0]);
                        a2[e] = h2_mul(a2[e], sv[1]);
                        a3[e] = h2_mul(a3[e], sv[1]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[nt][4 * i + e], a0[e], a1[e], a2[e], a3[e], p[b][nt][0], p[b][nt][1]);
                    }
                }
            }
            if (__any_sync(0xffffffffu, bad != 0)) {
                // the rows that see such a key come out as NaN
#pragma unroll 1
                for (int b = 0; b < G::B; ++b) {
                    int lowest = 16;  // the first one of the tile
#pragma unroll 1
                    for (int i = lane; i < G::SCALE_BYTES; i += 32)
                        if ((lds8(stage + b * G::STAGE + G::OFF_VS + i) & 0x7fu) == 0x7fu)
                            lowest = min(lowest, i / q4_scale_bytes(D));
                    lowest = __reduce_min_sync(0xffffffffu, lowest) + 16 * (tile + b);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (lowest < min(row_sees(8 * nt + 2 * t + e), 16 * (tile + b) + 16))
                                l[nt][e] = __int_as_float(0x7fffffff);
                }
            }
        };
#pragma unroll 1
        for (int tile = first; tile < end; tile += G::B) {
            const uint32_t bar = landed + 8u * q.get;
            if (!__all_sync(0xffffffffu, mbar_try_wait(bar, q.phase)) &&
                !__all_sync(0xffffffffu, await(bar, q.phase, guard, 5)))
                return false;
            const uint32_t stage = ring + q.get * (G::B * G::STAGE);
            float s[G::B][NT][4];
            scores(stage, s);
            softmax(tile, s);
            values(tile, stage);
            __syncwarp();
            if (++q.get == G::DEPTH) {
                q.get = 0;
                q.phase ^= 1u;
            }
            --q.pending;
            refill();
        }
    }

    // ---- results: O / l and the LSE (log2) of each row; 0 and -inf of one without a key
    float lse2[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        }
    auto finish = [&](float scale, float shift) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                // (l is NaN where a NaN came in)
                const bool none = l[nt][e] == 0.f;
                const float inv = none ? 0.f : scale / l[nt][e];
#pragma unroll
                for (int j = 0; j < G::J; ++j) {
                    o[nt][j][e] = none ? 0.f : o[nt][j][e] * inv;
                    o[nt][j][e + 2] = none ? 0.f : o[nt][j][e + 2] * inv;
                }
                lse2[nt][e] = none ? -INFINITY : m[nt][e] + __log2f(l[nt][e]) - shift;
            }
    };
    finish(a.v_scale4, kShift);
    // to O and LSE: a lane has D / 8 neighbouring channels of its queries
    auto write = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * nt + 2 * t + e, rt = (n * a.group_inv) >> 16;
                if (rt >= a.tile_tokens || tok0 + rt >= seq.sq) continue;
                const int64_t tok = static_cast<int64_t>(seq.q0) + tok0 + rt;
                const int head = r.head * a.group + n - rt * a.group;
                uint16_t *dst = static_cast<uint16_t *>(a.o) + (tok * a.h + head) * D + g * (D / 8);
                uint32_t w[G::J];
#pragma unroll
                for (int j = 0; j < G::J; ++j)
                    w[j] = BF16 ? cvt_pack_bf16(o[nt][j][e], o[nt][j][e + 2]) : cvt_pack_f16(o[nt][j][e], o[nt][j][e + 2]);
                if constexpr (D >= 64) {
#pragma unroll
                    for (int j = 0; j < G::J; j += 4)
                        reinterpret_cast<uint4 *>(dst)[j / 4] = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                } else if constexpr (D == 32) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
                } else {
                    *reinterpret_cast<uint32_t *>(dst) = w[0];
                }
                if (g == 0) a.lse[static_cast<int64_t>(head) * a.total_q + tok] = lse2[nt][e] * 0.69314718055994530942f;
            }
    };
    if (r.slot < 0) {
        write();
        return true;
    }

    // ---- a cut unit. Results lie in memory as the lanes hold them: O_i [NT, 2,
    // J, 32 lanes, 2] and LSE_i [ROWS].
    constexpr int V = G::J > 1 ? 2 : 1;  // products whose values a lane moves at once
    auto leave = [&](float *o_to, float *lse_to) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float *dst = o_to + (nt * 2 + e) * (G::J * 64) + lane * (2 * V);
#pragma unroll
                for (int j = 0; j < G::J; j += V) {
                    if constexpr (V == 2)
                        *reinterpret_cast<float4 *>(dst + j * 64) =
                            make_float4(o[nt][j][e], o[nt][j][e + 2], o[nt][j + 1][e], o[nt][j + 1][e + 2]);
                    else
                        *reinterpret_cast<float2 *>(dst + j * 64) = make_float2(o[nt][j][e], o[nt][j][e + 2]);
                }
                if (g == 0) lse_to[8 * nt + 2 * t + e] = lse2[nt][e];
            }
    };
    // Joins n results, place(i, &o, &lse) says where the i-th lies: with M the
    // largest LSE_i, l = sum_i 2^(LSE_i - M), O = sum_i 2^(LSE_i - M) O_i / l, LSE =
    // M + log2 l. P at a time, as registers allow: bound by the latency of loads
    // from L2.
    constexpr int P = D == 128 ? 2 : 4;
    auto gather = [&](int n, auto place, auto load) {
        clear();
#pragma unroll 1
        for (int i = 0; i < n; i += P) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float v[P][2][G::J][2], lse[P][2];
#pragma unroll
                for (int b = 0; b < P; ++b) {
                    const float *o_from, *lse_from;
                    place(min(i + b, n - 1), &o_from, &lse_from);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        lse[b][e] = load(lse_from + 8 * nt + 2 * t + e);
                        const float *src = o_from + (nt * 2 + e) * (G::J * 64) + lane * (2 * V);
#pragma unroll
                        for (int j = 0; j < G::J; j += V) {
                            if constexpr (V == 2) {
                                const float4 y = load(reinterpret_cast<const float4 *>(src + j * 64));
                                v[b][e][j][0] = y.x, v[b][e][j][1] = y.y;
                                v[b][e][j + 1][0] = y.z, v[b][e][j + 1][1] = y.w;
                            } else {
                                const float2 y = load(reinterpret_cast<const float2 *>(src + j * 64));
                                v[b][e][j][0] = y.x, v[b][e][j][1] = y.y;
                            }
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < P; ++b)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = i + b < n ? lse[b][e] : -INFINITY;
                        const float top = fmaxf(m[nt][e], x);
                        const float fo = m[nt][e] == -INFINITY ? 0.f : fast_exp2(m[nt][e] - top);
                        // (-inf: nothing to add; a NaN stays one)
                        const float fn = x == -INFINITY ? 0.f : fast_exp2(x - top);
                        m[nt][e] = top;
                        l[nt][e] = l[nt][e] * fo + fn;
#pragma unroll
                        for (int j = 0; j < G::J; ++j) {
                            o[nt][j][e] = o[nt][j][e] * fo + v[b][e][j][0] * fn;
                            o[nt][j][e + 2] = o[nt][j][e + 2] * fo + v[b][e][j][1] * fn;
                        }
                    }
            }
        }
        finish(1.0f, 0.f);
    };
    // The CTA's warps whose shares end inside the unit have no more work: they
    // leave their results in their rings, and the last one to come joins them.
    // Entries of the unit's list: one for each CTA so, and its last part.
    const int cta = part / G::WARPS, cta0 = first_part / G::WARPS, last = first_part + nparts - 1;
    const int entries = (last - 1) / G::WARPS - cta0 + 2;
    if (part != last) {
        const int from = max(first_part, cta * G::WARPS), to = min(last - 1, cta * G::WARPS + G::WARPS - 1);
        if (from < to) {
            float *room = reinterpret_cast<float *>(smem + (part % G::WARPS) * G::RING);
            leave(room, room + G::ROWS * D);
            if (!warp_arrives_last_in_cta(reinterpret_cast<int *>(smem + G::OFF_MISC + 16) + from % G::WARPS,
                                          to - from + 1))
                return true;
            gather(to - from + 1, [&](int i, const float **o_from, const float **lse_from) {
                *o_from = reinterpret_cast<const float *>(smem + ((from + i) % G::WARPS) * G::RING);
                *lse_from = *o_from + G::ROWS * D;
            }, [](const auto *p) { return *p; });
        }
    }
    // where entry i of the unit lies: at the place of its first part
    auto place = [&](int i) {
        return part_place(first_part, i == entries - 1 ? nparts - 1 : max((cta0 + i) * G::WARPS - first_part, 0));
    };
    auto leave_entry = [&](int i) { leave(a.o_part + place(i) * (G::ROWS * D), a.lse_part + place(i) * G::ROWS); };
    auto gather_entries = [&](int i0, int every, int n) {
        gather(n, [&](int i, const float **o_from, const float **lse_from) {
            const int64_t at = place(i0 + i * every);
            *o_from = a.o_part + at * (G::ROWS * D);
            *lse_from = a.lse_part + at * G::ROWS;
        }, [](const auto *p) { return __ldcg(p); });
    };
    const int mine = part == last ? entries - 1 : cta - cta0, group = mine / kJoin * kJoin;
    const int members = min(kJoin, entries - group);
    leave_entry(mine);
    if (!warp_arrives_last(a.arrivals + place(group), a.call, members)) return true;
    gather_entries(group, 1, members);
    if (entries > kJoin) {
        leave_entry(group);
        const int groups = (entries + kJoin - 1) / kJoin;
        if (!warp_arrives_last(a.arrivals + 2 * deal.parts + first_part, a.call, groups)) return true;
        gather_entries(0, kJoin, groups);
    }
    write();
    return true;
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(DecGeom<D, NT>::WARPS * 32, DecGeom<D, NT>::CTAS) decode_q4_kernel(const PackArgs a) {
    using G = DecGeom<D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_MISC);
    LineSum *sums = reinterpret_cast<LineSum *>(smem + G::OFF_SUM);
    griddep_launch_dependents();  // (the chunks' kernel touches nothing of this one's)
    if (threadIdx.x == 0) {
        for (int i = 0; i < G::WARPS * G::DEPTH; ++i) mbar_init(sbase + G::OFF_BAR + 8u * i, G::B);
        *abort_flag = 0u;
        for (int i = 0; i < G::WARPS; ++i) reinterpret_cast<int *>(smem + G::OFF_MISC + 16)[i] = 0;
        fence_mbar_init();
    }
    if (a.seqs.b > 32) line_sum_warps<2, true>(a.seqs, a.line, sums, a.filter);  // (fewer: find_part does it alone)
    __syncthreads();
    const WaitGuard g{abort_flag, a.status, kKernFwd};
    const uint32_t ring = sbase + warp * G::RING, landed = sbase + G::OFF_BAR + 8u * (warp * G::DEPTH);
    const int part = blockIdx.x * G::WARPS + warp;
    LineShape shape = a.line;
    LineDeal deal;
    PartPlace at = find_part<2, true, true>(
        a.seqs, shape, [&] { return line_total(sums, G::WARPS); }, part, gridDim.x * G::WARPS, &deal, a.filter);
    TileRing q;
    walk_part(
        shape, a.seqs.b, at.p, at.e, at.p_len, at.p_units, at.p_x0,
        [&](int i) {
            at.cur = seq_info<true>(a.seqs, i, nullptr, a.filter);
            return SeqLen{at.cur.sq, at.cur.sk};
        },
        [&](const UnitRange &r) {
            return take_range<D, BF16, NT>(r, at.cur, shape, deal, part, smem, ring, landed, q, a, g);
        });
    // Never leave the CTA with a copy still landing (after a wait that ran out)
    WaitGuard drain = g;
    uint32_t no_abort = 0;
    drain.abort = &no_abort;
#pragma unroll 1
    for (; q.pending > 0; --q.pending) {
        await(landed + 8u * q.get, q.phase, drain, 10);
        if (++q.get == G::DEPTH) {
            q.get = 0;
            q.phase ^= 1u;
        }
    }
}

template <int D, bool BF16, int NT>
cudaError_t launch_t(const PackArgs &a, cudaStream_t stream) {
    using G = DecGeom<D, NT>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(decode_q4_kernel<D, BF16, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 G::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    decode_q4_kernel<D, BF16, NT><<<a.ctas, G::WARPS * 32, G::SMEM_BYTES, stream>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(bool bf16, bool two, const PackArgs &a, cudaStream_t stream) {
    if (two) return bf16 ? launch_t<D, true, 2>(a, stream) : launch_t<D, false, 2>(a, stream);
    return bf16 ? launch_t<D, true, 1>(a, stream) : launch_t<D, false, 1>(a, stream);
}

}  // namespace

cudaError_t launch_decode_q4(int d, bool bf16, int rows, const PackArgs &a, cudaStream_t stream) {
    const bool two = rows == 16;
    switch (d) {
        case 16: return launch_d<16>(bf16, two, a, stream);
        case 32: return launch_d<32>(bf16, two, a, stream);
        case 64: return launch_d<64>(bf16, two, a, stream);
        case 128: return launch_d<128>(bf16, two, a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace exattn
