// A few new rows of each request over a cache held in 4 bits
// (attn_chunk_paged_q4 where no request has more than 16 rows to a K/V head).
//
// The mathematics is the forward's: S = scale Q K^T, an online softmax, O = P V,
// and per key 1.125 bytes of K and V a channel are read once. What bounds it is
// the way from those bytes to the tensor core: at the copy bandwidth an SM gets
// 128 channels of K and V of 16 keys every 100 cycles, 4,096 codes to be
// widened. So the codes go from HBM into a warp's own ring in shared memory
// (cp.async, 16 bytes a lane) and from there straight into registers in the
// order in which mma.sync wants its operand; nothing widened is written back.
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
//   k(r) = r ^ (r >> 2 & 1), and 16-byte chunks swapped by bit 1 of the key (D =
//      128), so that neither read meets a bank twice
//   P  the C fragment of S^T, rounded to fp16 and transposed 8 by 8 (movmatrix)
// A code times its scale is exact in fp16 (q4.cuh). bf16 queries are brought into
// fp16 with a power of two a row (largest value in [2^14, 2^15): nothing above
// 2^-31 of it is rounded), which goes into the softmax's scale.
//
// Warps share nothing on the way: each takes every W-th tile of 16 keys of the
// unit with a softmax of its own, and prefetches across units. They meet at a
// unit's end. Units are dealt to CTAs as in fwd_packed.cuh; a cut unit's ranges
// are joined by the one that finishes last, in the order of the keys.
#include "packed.h"
#include "packed_dev.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace exattn {
namespace {

constexpr float kShift = 6.0f;  // P is 2^6 times the softmax's, at most 2^14

template <int D, int NT>
struct DecGeom {
    static constexpr int W = NT == 1 ? 7 : 11;          // warps that compute (with the scheduler, 4 or 3 to a quarter SM)
    static constexpr int CTAS = NT == 1 ? 2 : 1;        // of an SM
    static constexpr int THREADS = (W + 1) * 32;
    static constexpr int ROWS = 8 * NT;
    static constexpr int J = D / 16;                    // products of 16 channels
    static constexpr int CODE_BYTES = 16 * q4_code_bytes(D);    // of a tile of K or V
    static constexpr int SCALE_BYTES = 16 * q4_scale_bytes(D);
    static constexpr int OFF_KS = CODE_BYTES, OFF_V = OFF_KS + SCALE_BYTES, OFF_VS = OFF_V + CODE_BYTES;
    static constexpr int STAGE = OFF_VS + SCALE_BYTES;
    static constexpr int DEPTH = D == 128 ? 5 : 8;      // tiles of a warp's ring
    static constexpr int FRAGS = NT * J * 2;            // float2 of a lane's O
    static constexpr int OFF_PART = W * DEPTH * STAGE;
    static constexpr int OFF_ML = OFF_PART + W * FRAGS * 32 * 8;
    static constexpr int OFF_BAR = OFF_ML + W * ROWS * 8;
    static constexpr int BAR_MF = 0;
    static constexpr int BAR_ME = BAR_MF + kMsgSlots;
    static constexpr int BAR_MS = BAR_ME + kMsgSlots;
    static constexpr int BAR_A = BAR_MS + kMsgSlots;  // warps meet
    static constexpr int BAR_B = BAR_A + 1;           // a unit's parts have been read
    static constexpr int NUM_BARS = BAR_B + 1;
    static constexpr int OFF_MSG = (OFF_BAR + NUM_BARS * 8 + 15) & ~15;
    static constexpr int OFF_SUM = OFF_MSG + kMsgSlots * 64;
    static constexpr int OFF_MISC = OFF_SUM + (W + 1) * 12;
    static constexpr int SMEM_BYTES = OFF_MISC + 16;
    static_assert(STAGE % 16 == 0 && (SMEM_BYTES + 1024) * CTAS <= 228 * 1024, "shared memory budget");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
    asm volatile(
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

// The key in its tile that row r of the products stands for, and where chunk c
// (16 bytes) of a key's codes lies among the tile's.
__device__ __forceinline__ int key_of(int r) { return r ^ (r >> 2 & 1); }
template <int D>
__device__ __forceinline__ int chunk_at(int key, int c) {
    return D == 128 ? key * 4 + (c ^ (key & 2)) : D == 64 ? key * 2 + c : key;
}

// As arrive_last(), for more than 255 CTAs: (call's low 22 bits << 10 | arrivals).
__device__ __forceinline__ bool arrive_last_of_many(uint32_t *counter, uint32_t call, int n) {
    call &= 0x3fffffu;
    uint32_t old = *reinterpret_cast<volatile uint32_t *>(counter), seen;
    do {
        seen = old;
        old = atomicCAS(counter, seen, ((seen >> 10) == call ? seen : call << 10) + 1);
    } while (old != seen);
    const bool last = ((seen >> 10) == call ? seen & 0x3ffu : 0u) + 1 == static_cast<uint32_t>(n);
    if (last) atomicExch(counter, 0u);
    return last;
}

// The tiles that a warp fetches, in the order in which it will take them:
// where the next one lies, its page looked up ahead.
template <int D, int NT>
struct Fetch {
    using G = DecGeom<D, NT>;
    int n = 0, tile = 0, end = 0;  // the next message; the next tile and the end of its unit's
    int head = 0, page = 0, row = 0;
    const int32_t *table = nullptr;

    // Finds the next tile, in a later unit where this one's are over. False:
    // no unit there yet, or the message would lie in the slot of one that this
    // warp, at unit `now`, has not freed. Never waits.
    __device__ __forceinline__ bool next(int now, int w, const UnitMsg *msgs, uint32_t full, const PackArgs &a) {
        while (tile >= end) {
            const int s = n % kMsgSlots;
            if (n - now >= kMsgSlots || !__all_sync(0xffffffffu, mbar_test_wait(full + 8u * s, n / kMsgSlots & 1)))
                return false;
            const volatile UnitMsg *x = msgs + s;
            if (x->live == 0) return false;
            ++n;
            tile = x->step0 * 8 + w;
            end = min((x->step0 + x->nstep) * 8, (x->sk + 15) >> 4);
            head = x->head;
            table = a.block_table + static_cast<int64_t>(x->seq) * a.max_pages;
            look_up(a);
        }
        return true;
    }
    __device__ __forceinline__ void look_up(const PackArgs &a) {
        if (tile < end) {
            const int p = divided(static_cast<uint32_t>(tile), a.page_mul, a.page_div);
            row = 16 * tile - p * a.page_size;
            page = __ldg(table + p);
        }
    }
    // Fetches the tile that next() found, and goes on to the one after it.
    __device__ __forceinline__ void issue(uint32_t stage, const PackArgs &a) {
        {
            const int lane = threadIdx.x & 31;
            const int64_t block =
                (static_cast<int64_t>(min(max(page, 0), a.num_pages - 1)) * a.line.heads + head) * a.block4;
            const int64_t codes = block + row * q4_code_bytes(D);
            const int64_t scales = block + a.page_size * q4_code_bytes(D) + row * q4_scale_bytes(D);
            constexpr int CH = G::CODE_BYTES / 16, SCH = G::SCALE_BYTES / 16, CPK = CH / 16 > 0 ? CH / 16 : 1;
#pragma unroll
            for (int i0 = 0; i0 < CH; i0 += 32) {
                const int i = i0 + lane;
                if (CH % 32 == 0 || i < CH) {
                    const uint32_t at = stage + 16 * (D >= 64 ? chunk_at<D>(i / CPK, i % CPK) : i);
                    cp_async16(at, a.k4 + codes + 16 * i);
                    cp_async16(at + G::OFF_V, a.v4 + codes + 16 * i);
                }
            }
            if (lane < SCH)
                cp_async16(stage + G::OFF_KS + 16 * lane, a.k4 + scales + 16 * lane);
            else if (lane >= 16 && lane < 16 + SCH)
                cp_async16(stage + G::OFF_VS + 16 * (lane - 16), a.v4 + scales + 16 * (lane - 16));
        }
        cp_async_commit();
        tile += G::W;
        look_up(a);
    }
};

// A lane's codes of one key for S: D / 4 channels, a word for 8.
template <int D>
__device__ __forceinline__ void load_k(uint32_t stage, int key, int t, uint32_t (&w)[(D + 31) / 32]) {
    if constexpr (D == 128) {
        const uint4 x = lds128(stage + 16 * chunk_at<D>(key, t));
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
        const uint2 x = lds64(stage + 16 * chunk_at<D>(key, g >> 1) + 8 * (g & 1));
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

template <int D, bool BF16, int NT>
__device__ __forceinline__ void decode_warp(uint8_t *smem, uint32_t sbase, int w, const UnitMsg *msgs,
                                            const PackArgs &a, const WaitGuard &guard) {
    using G = DecGeom<D, NT>;
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = sbase + w * G::DEPTH * G::STAGE;
    float2 *parts = reinterpret_cast<float2 *>(smem + G::OFF_PART);
    float2 *ml = reinterpret_cast<float2 *>(smem + G::OFF_ML);
    volatile int *joiner = reinterpret_cast<volatile int *>(smem + G::OFF_MISC + 8);

    Fetch<D, NT> f;
    int get = 0, put = 0, pending = 0;  // ring slots, and tiles on their way
    // as many tiles on their way as the ring holds
    auto refill = [&](int now) {
#pragma unroll 1
        while (pending < G::DEPTH && f.next(now, w, msgs, bar(G::BAR_MF), a)) {
            f.issue(ring + put * G::STAGE, a);
            if (++put == G::DEPTH) put = 0;
            ++pending;
        }
    };
    int met = 0, parts_read = 0;  // phases of the meetings

#pragma unroll 1
    for (int n = 0;; ++n) {
        const volatile UnitMsg *x = wait_unit(n, msgs, bar(G::BAR_MF), guard, 17);
        if (x == nullptr) break;
        refill(n);
        const int sk = x->sk, sq = x->sq, tok0 = x->tok0, kv_head = x->head;
        const int64_t q0 = x->q0;
        // ---- the unit's queries: row n of the products is token n / group, head n % group
        uint32_t qf[NT][2 * G::J];
        float c[NT][2];    // the softmax's scale of queries 2t and 2t + 1
        int sees[NT][2];   // keys that they see
        int all_see = sk;  // keys that every row sees
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = 8 * nt + g, rt = (row * a.group_inv) >> 16;
            const bool used = rt < a.tile_tokens && tok0 + rt < sq;
#pragma unroll
            for (int i = 0; i < 2 * G::J; ++i) qf[nt][i] = 0u;
            if (used) {
                const uint16_t *src = static_cast<const uint16_t *>(a.q) + (q0 + tok0 + rt) * a.q_stride +
                                      (kv_head * a.group + row - rt * a.group) * D + t * (D / 4);
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
                const int r = 8 * nt + 2 * t + e, tok = tok0 + ((r * a.group_inv) >> 16);
                sees[nt][e] = a.causal && tok < sq ? min(sk, tok + sk - sq + 1) : sk;
                all_see = min(all_see, sees[nt][e]);
            }
        }
        all_see = __reduce_min_sync(0xffffffffu, all_see);

        float o[NT][G::J][4], m[NT][2], neg[NT][2], l[NT][2];
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

        const int end = min((x->step0 + x->nstep) * 8, (sk + 15) >> 4);
#pragma unroll 1
        for (int tile = x->step0 * 8 + w; tile < end; tile += G::W) {
            // (this unit's message is there: its next tile is on its way, or can be fetched)
            if (pending == G::DEPTH) {
                cp_async_wait<G::DEPTH - 1>();
            } else {
                if (pending == 0) refill(n);
                cp_async_wait<0>();
            }
            __syncwarp();
            const uint32_t stage = ring + get * G::STAGE;
            // ---- S^T = K Q^T
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
            {
                uint32_t w0[(D + 31) / 32], w1[(D + 31) / 32], s0[D == 128 ? 2 : 1], s1[D == 128 ? 2 : 1];
                const int k0 = key_of(g), k1 = k0 + 8;
                load_k<D>(stage, k0, t, w0);
                load_k<D>(stage, k1, t, w1);
                load_ks<D>(stage + G::OFF_KS, k0, t, s0);
                load_ks<D>(stage + G::OFF_KS, k1, t, s1);
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
                        mma16816(s[nt], x0[0], x1[0], x0[1], x1[1], qf[nt][4 * i % (2 * G::J)],
                                 qf[nt][(4 * i + 1) % (2 * G::J)]);
                        if (D > 16)
                            mma16816(s[nt], x0[2], x1[2], x0[3], x1[3], qf[nt][(4 * i + 2) % (2 * G::J)],
                                     qf[nt][(4 * i + 3) % (2 * G::J)]);
                    }
                }
            }
            // ---- softmax
            uint32_t p[NT][2];
            const bool ragged = 16 * tile + 16 > all_see;
            bool need = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] *= c[nt][i & 1];
                if (ragged) {
                    const int k0 = 16 * tile + key_of(g);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k0 + 8 * (i >> 1) >= sees[nt][i & 1]) s[nt][i] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) need = need || fmaxf(s[nt][e], s[nt][e + 2]) > m[nt][e] + 8.0f;
            }
            // The reference max moves when a tile exceeds it by more than 8 (log2)
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[nt][e], s[nt][e + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        if (top > m[nt][e] + 8.0f) {
                            const float alpha = fast_exp2(m[nt][e] - top);
                            m[nt][e] = top;
                            neg[nt][e] = kShift - top;
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
                for (int i = 0; i < 4; ++i) {
                    s[nt][i] = fast_exp2(s[nt][i] + neg[nt][i & 1]);
                    l[nt][i & 1] += s[nt][i];
                }
                p[nt][0] = transpose8x8(cvt_pack_f16(s[nt][0], s[nt][1]));
                p[nt][1] = transpose8x8(cvt_pack_f16(s[nt][2], s[nt][3]));
            }
            // ---- O^T += V^T P^T
            {
                uint32_t lo[2][(D + 63) / 64], hi[2][(D + 63) / 64], sv[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t w0[(D + 63) / 64], w1[(D + 63) / 64];
                    const int k0 = key_of(2 * t) + 8 * half, k1 = key_of(2 * t + 1) + 8 * half;
                    load_v<D>(stage + G::OFF_V, k0, g, w0);
                    load_v<D>(stage + G::OFF_V, k1, g, w1);
                    sv[half] = q4_scales_f16(load_vs<D>(stage + G::OFF_VS, k0, g) |
                                             load_vs<D>(stage + G::OFF_VS, k1, g) << 8);
                    // (a stale scale may be NaN)
                    if (16 * tile + k0 >= sk) sv[half] &= 0xffff0000u;
                    if (16 * tile + k1 >= sk) sv[half] &= 0x0000ffffu;
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
                            mma16816(o[nt][4 * i + e], a0[e], a1[e], a2[e], a3[e], p[nt][0], p[nt][1]);
                    }
                }
            }
            __syncwarp();
            if (++get == G::DEPTH) get = 0;
            --pending;
            refill(n);
        }

        // ---- the warps' results of the unit together
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
            }
        if (n > 0) {  // the last unit's parts have been read
            const bool ok = await(bar(G::BAR_B), parts_read & 1, guard, 19);
            ++parts_read;
            if (!__all_sync(0xffffffffu, ok)) return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < G::J; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    parts[(w * G::FRAGS + (nt * 2 + e) * G::J + j) * 32 + lane] =
                        make_float2(o[nt][j][e], o[nt][j][e + 2]);
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    ml[w * G::ROWS + 8 * nt + 2 * t + e] = make_float2(m[nt][e], l[nt][e]);
            }
        }
        if (!meet(bar(G::BAR_A), met, guard)) return;
        const int part_slot = x->slot;
        const int64_t mine = 2 * static_cast<int64_t>(blockIdx.x) + max(part_slot, 0);
        // Writes row r's channels of product j (this lane's pair), or the row's LSE
        auto write = [&](int r, int j, float2 v) {
            const int rt = (r * a.group_inv) >> 16;
            if (rt < a.tile_tokens && tok0 + rt < sq) {
                const int64_t at = ((q0 + tok0 + rt) * a.h + kv_head * a.group + r - rt * a.group) * D;
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.o) + at + g * (D / 8) + 2 * j) =
                    BF16 ? cvt_pack_bf16(v.x, v.y) : cvt_pack_f16(v.x, v.y);
            }
        };
        auto write_lse = [&](int r, float lse2) {
            const int rt = (r * a.group_inv) >> 16;
            if (rt < a.tile_tokens && tok0 + rt < sq)
                a.lse[static_cast<int64_t>(kv_head * a.group + r - rt * a.group) * a.total_q + q0 + tok0 + rt] =
                    lse2 * 0.69314718055994530942f;
        };
#pragma unroll 1
        for (int ne = 0; ne < 2 * NT; ++ne) {
            const int r = 8 * (ne >> 1) + 2 * t + (ne & 1);
            float top = -INFINITY, sum = 0.f, weight[G::W];
#pragma unroll
            for (int i = 0; i < G::W; ++i) top = fmaxf(top, ml[i * G::ROWS + r].x);
#pragma unroll
            for (int i = 0; i < G::W; ++i) {
                const float2 y = ml[i * G::ROWS + r];
                weight[i] = y.x == -INFINITY ? 0.f : fast_exp2(y.x - top);
                sum += y.y * weight[i];
            }
            // (a row without a key has no maximum; a NaN stays one)
            const bool none = top == -INFINITY && sum == 0.f;
            const float inv = none ? 0.f : a.v_scale4 / sum;
#pragma unroll 1
            for (int j = w; j < G::J; j += G::W) {
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < G::W; ++i) {
                    const float2 y = parts[(i * G::FRAGS + ne * G::J + j) * 32 + lane];
                    v.x += y.x * weight[i];
                    v.y += y.y * weight[i];
                }
                v = none ? make_float2(0.f, 0.f) : make_float2(v.x * inv, v.y * inv);
                if (part_slot >= 0)
                    reinterpret_cast<float2 *>(a.o_part)[(mine * G::FRAGS + ne * G::J + j) * 32 + lane] = v;
                else
                    write(r, j, v);
            }
            if (w == 0 && g == 0) {
                const float lse2 = none ? -INFINITY : top + __log2f(sum) - kShift;
                if (part_slot >= 0)
                    a.lse_part[mine * G::ROWS + r] = lse2;
                else
                    write_lse(r, lse2);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(G::BAR_B));
        if (part_slot >= 0) {
            // A cut unit: the range that arrives last joins them all
            const bool ok = await(bar(G::BAR_MS + n % kMsgSlots), (n / kMsgSlots) & 1, guard, 23);
            if (!__all_sync(0xffffffffu, ok)) return;
            const int first = x->first_part, nparts = x->nparts;
            __threadfence();
            if (!meet(bar(G::BAR_A), met, guard)) return;
            if (w == 0 && lane == 0) {
                *joiner = arrive_last_of_many(a.arrivals + first, a.call, nparts);
                __threadfence();
            }
            if (!meet(bar(G::BAR_A), met, guard)) return;
            if (*joiner) {
                __threadfence();
#pragma unroll 1
                for (int ne = 0; ne < 2 * NT; ++ne) {
                    const int r = 8 * (ne >> 1) + 2 * t + (ne & 1);
                    constexpr int P = 8;  // ranges at once: bound by the latency of L2
#pragma unroll 1
                    for (int j = w; j < G::J; j += G::W) {
                        float top = -INFINITY, sum = 0.f;
                        float2 v = make_float2(0.f, 0.f);
#pragma unroll 1
                        for (int p0 = 0; p0 < nparts; p0 += P) {
                            float lp[P];
                            float2 op[P];
#pragma unroll
                            for (int i = 0; i < P; ++i) {
                                lp[i] = -INFINITY;
                                op[i] = make_float2(0.f, 0.f);
                                if (p0 + i < nparts) {
                                    const int64_t at = 2 * static_cast<int64_t>(first + p0 + i) + (p0 + i == 0 ? 1 : 0);
                                    lp[i] = __ldcg(a.lse_part + at * G::ROWS + r);
                                    op[i] = __ldcg(reinterpret_cast<const float2 *>(a.o_part) +
                                                   (at * G::FRAGS + ne * G::J + j) * 32 + lane);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < P; ++i) {
                                const float mn = fmaxf(top, lp[i]);
                                const float fo = top == -INFINITY ? 0.f : fast_exp2(top - mn);
                                const float fn = lp[i] == -INFINITY ? 0.f : fast_exp2(lp[i] - mn);
                                top = mn;
                                sum = sum * fo + fn;
                                v.x = v.x * fo + op[i].x * fn;
                                v.y = v.y * fo + op[i].y * fn;
                            }
                        }
                        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
                        write(r, j, make_float2(v.x * inv, v.y * inv));
                        if (j == 0 && g == 0) write_lse(r, sum == 0.f ? -INFINITY : top + __log2f(sum));
                    }
                }
            }
        }
        free_unit(n, bar(G::BAR_ME));
    }
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(DecGeom<D, NT>::THREADS, DecGeom<D, NT>::CTAS) decode_q4_kernel(const PackArgs a) {
    using G = DecGeom<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
    const int warp = threadIdx.x >> 5;
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(smem + G::OFF_MISC);
    UnitMsg *msgs = reinterpret_cast<UnitMsg *>(smem + G::OFF_MSG);
    LineSum *sums = reinterpret_cast<LineSum *>(smem + G::OFF_SUM);
    if (threadIdx.x == 0) {
        for (int i = 0; i < G::NUM_BARS; ++i)
            mbar_init(bar(i), (i >= G::BAR_ME && i < G::BAR_MS) || i >= G::BAR_A ? G::W : 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (a.seqs.b > 32) line_sum_warps<0>(a.seqs, a.line, sums);
    __syncthreads();
    const WaitGuard g{abort_flag, a.status, kKernFwd};
    if (warp < G::W) {
        decode_warp<D, BF16, NT>(smem, sbase, warp, msgs, a, g);
        cp_async_wait<0>();  // never leave the CTA with a copy still landing
    } else if (!(a.flags & kFlagSkipLoads))
        post_units<0>(
            a.seqs, a.line, [&] { return line_total(sums, G::W + 1); }, msgs, bar(G::BAR_MF), bar(G::BAR_ME),
            bar(G::BAR_MS), g, 18, blockIdx.x, gridDim.x);
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
    decode_q4_kernel<D, BF16, NT><<<a.ctas, G::THREADS, G::SMEM_BYTES, stream>>>(a);
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
